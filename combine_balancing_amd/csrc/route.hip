// The router's expert choice and its gradient: logits [T,E] become the
// topk_ids and scores that the plan, the remap, the combine and the expert
// layer take.
//
// Forward, per token (l widened exactly; an expert whose logit is -inf or
// NaN is absent):
//   s = softmax(l) over the experts present, or sigmoid(l)
//   c = l without a bias, s + bias with one; c = -inf is never taken
//   with n_group > 1, only the topk_group groups of the largest value are
//   kept: a group's value is its largest c without a bias, the sum of its
//   two largest with one
//   ids = the K largest c, descending; ties go to the lower id
//   w = s[ids], renormalised to sum 1 if asked, times `scale`
// A choice next to a border must not hang on how s was rounded, so c is
// formed in fp64, and groups are compared in it; experts are compared on the
// upper 42 bits of c's mantissa, whose lower bits carry the expert's id.
#include <algorithm>
#include <type_traits>

#include "rows.h"

namespace mep {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / kWave;
constexpr int kRouteMaxE = 1024;
constexpr int kRouteMaxK = 64;  // one lane per chosen expert
constexpr int kRouteMaxGroups = 64;
constexpr int kRouteManyTokens = 4096;
constexpr int kRouteMaxT = 1 << 26;  // a launch holds fewer than 2^32 threads, up to 64 a token
constexpr double kRenormEps = 1e-20;  // sigmoid scores may all round to zero

template <typename T>
__device__ __forceinline__ float widen(T v);
template <>
__device__ __forceinline__ float widen<float>(float v) { return v; }
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t v) {  // bf16 bits
    return __uint_as_float((uint32_t)v << 16);
}
template <>
__device__ __forceinline__ float widen<_Float16>(_Float16 v) { return (float)v; }

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float v) {
    return (uint16_t)bf16x2_bits(v, 0.0f);
}
template <>
__device__ __forceinline__ _Float16 narrow<_Float16>(float v) { return (_Float16)v; }

// A logit as it is used: +inf counts as the largest finite value, NaN as -inf.
__device__ __forceinline__ float clean(float l) {
    return l > -INFINITY ? fminf(l, 3.402823466e38f) : -INFINITY;
}

__device__ __forceinline__ double wave_max_d(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = fmax(v, __shfl_xor(v, m, kWave));
    return v;
}

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
    return v;
}

// exp(x) for x <= 0 within about 2^-50 (0 below -800): 2^n times the Taylor
// series of the remainder r = x - n ln 2, |r| <= ln(2) / 2, to the 13th power
// (the next term is under 5e-18). ln 2 is taken in two parts, the first with
// 40 fraction bits, so that n times it is exact.
__device__ __forceinline__ double exp_neg(double x) {
    x = fmax(x, -800.0);
    const double n = rint(x * 1.4426950408889634);
    double r = __builtin_fma(n, -0.6931471805601177, x);
    r = __builtin_fma(n, 1.7239444525614835e-13, r);
    double p = 1.0 / 6227020800.0;
    auto next = [&](double c) {
        asm("" : "+s"(c));  // a scalar operand of the fma, not two moves into its target first
        p = __builtin_fma(p, r, c);
    };
    next(1.0 / 479001600.0);
    next(1.0 / 39916800.0);
    next(1.0 / 3628800.0);
    next(1.0 / 362880.0);
    next(1.0 / 40320.0);
    next(1.0 / 5040.0);
    next(1.0 / 720.0);
    next(1.0 / 120.0);
    next(1.0 / 24.0);
    next(1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}

// 1 / d for 1 <= d <= 2: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double reciprocal(double d) {
    double y = __builtin_amdgcn_rcp(d);
    y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
    return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}

__device__ __forceinline__ double sigmoid(float l) {
    const double x = exp_neg(-fabs((double)l));
    const double y = reciprocal(1.0 + x);
    return l >= 0.0f ? y : x * y;
}

// Exchange of a double over the L lanes (16, 32 or 64) of a token: within 16
// by row rotations (no LDS), further by shuffles.
template <int CTRL>
__device__ __forceinline__ double row_move(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, 0xf, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, 0xf, 0xf, false);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

template <int L, class F>
__device__ __forceinline__ double lanes_reduce(double v, F f) {
    v = f(v, row_move<0x128>(v));  // row_ror 8, 4, 2, 1
    v = f(v, row_move<0x124>(v));
    v = f(v, row_move<0x122>(v));
    v = f(v, row_move<0x121>(v));
    if (L >= 32) v = f(v, __shfl_xor(v, 16, kWave));
    if (L >= 64) v = f(v, __shfl_xor(v, 32, kWave));
    return v;
}
template <int L>
__device__ __forceinline__ double lanes_max(double v) {
    return lanes_reduce<L>(v, [](double a, double b) { return fmax(a, b); });
}
template <int L>
__device__ __forceinline__ double lanes_sum(double v) {
    return lanes_reduce<L>(v, [](double a, double b) { return a + b; });
}

// Logits in one load of a lane's V: 16 bytes where they divide V, else 4.
template <typename LT, int V>
constexpr int kLaneVec = V % (16 / (int)sizeof(LT)) == 0 ? 16 / (int)sizeof(LT) : 4;

constexpr double kNone = -1e300;  // an expert that cannot be taken (c is above -1e39)

// Batcher's merge exchange, largest first; 63 exchanges for 16 values.
template <int V>
__device__ __forceinline__ void sort_down(double (&c)[V]) {
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int a = 0; a < V - k; ++a)
                if (a >= k % p && (a - k % p) / k % 2 == 0 && a / (2 * p) == (a + k) / (2 * p)) {
                    const double x = c[a], y = c[a + k];
                    c[a] = fmax(x, y);
                    c[a + k] = fmin(x, y);
                }
}

// L lanes per token; lane i of them holds experts i * V .. i * V + V - 1.
// Needs E <= L * V, K <= L, and whole lanes per group.
//
// Each lane sorts its V values; then the chosen are taken one by one: the
// largest of the lanes' first values, and the lane that has it moves the rest
// of its list up. The id in a value's lowest 10 bits (complemented where the
// value is positive) makes all values different and equal c go to the lower
// id, so maxima and minima are all it takes. 64 / L tokens share a wave: the
// exchange over the lanes then serves several tokens. Bound by the issue of
// instructions, most in 64 bits (about 1700 a wave of 4 tokens of 256 experts):
// 32768 tokens over 256 experts in 8 groups, bias, sigmoid, 8 taken: 28 us, of
// which the scores are 40 %. A maximum over the lane's 16 unsorted values and a
// strike for each of the chosen: 34 us; one token a wave: 117 us.
template <typename LT, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void route_lanes(
    const LT* __restrict__ logits, const float* __restrict__ bias, int sig, int wide, int n_group,
    int topk_group, int renorm, float scale, int* __restrict__ ids, float* __restrict__ scores,
    int T, int E, int K) {
    constexpr int kTokens = kRouteThreads / L;
    const int lane = lane_id(), i = lane & (L - 1), base = lane & ~(L - 1);
    const int t_raw = blockIdx.x * kTokens + threadIdx.x / L;
    const int t = min(t_raw, T - 1);  // lanes past T work on a real row, store nothing
    const LT* row = logits + (size_t)t * E;

    float l[V];
    if (wide) {  // rows and lanes start on whole vectors, E is a multiple of V
        constexpr int M = kLaneVec<LT, V>;
        typedef LT vec __attribute__((ext_vector_type(M)));
#pragma unroll
        for (int v = 0; v < V; v += M) {
            const vec w = *(const vec*)(row + min(i * V, E - V) + v);
#pragma unroll
            for (int k = 0; k < M; ++k) l[v + k] = widen<LT>(w[k]);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) l[v] = widen<LT>(row[min(i * V + v, E - 1)]);
    }
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        l[v] = i * V + v < E ? clean(l[v]) : -INFINITY;
        top = fmaxf(top, l[v]);
    }
    double z = 1.0;  // 1 / sum of the softmax
    if (!sig) {
        top = (float)lanes_max<L>(top);
        if (bias || !renorm) {
            double part = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v)
                part += l[v] > -INFINITY ? exp_neg((double)l[v] - (double)top) : 0.0;
            part = lanes_sum<L>(part);
            z = part > 0.0 ? 1.0 / part : 0.0;
        }
    }

    double c[V];
    // one loop for each form: a branch an expert kept the sixteen chains of
    // an exponential from running side by side
    auto fill = [&](auto f) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            c[v] = f(v) + 0.0;  // -0 counts as 0
            if (!(l[v] > -INFINITY && c[v] > kNone)) c[v] = kNone;  // absent, or such a bias
            c[v] = fmin(c[v], 1e300);
        }
    };
    auto added = [&](int v) { return (double)bias[min(i * V + v, E - 1)]; };
    if (!bias)
        fill([&](int v) { return (double)l[v]; });
    else if (sig)
        fill([&](int v) { return sigmoid(l[v]) + added(v); });
    else
        fill([&](int v) { return exp_neg((double)l[v] - (double)top) * z + added(v); });

    if (n_group > 1) {
        double a = kNone, b = kNone;  // the two largest of the lane, then of the group
#pragma unroll
        for (int v = 0; v < V; ++v) {
            b = fmax(b, fmin(a, c[v]));
            a = fmax(a, c[v]);
        }
        const int per = E / n_group / V;  // lanes of a group
        const int mine = i / per, first = base + min(mine, n_group - 1) * per;
        double ga = kNone, gb = kNone;
        for (int j = 0; j < per; ++j) {
            const double oa = __shfl(a, first + j, kWave), ob = __shfl(b, first + j, kWave);
            gb = fmax(fmax(gb, ob), fmin(ga, oa));
            ga = fmax(ga, oa);
        }
        const double gv = bias && gb > kNone ? ga + gb : ga;
        int rank = 0;
        for (int j = 0; j < n_group; ++j) {
            const double o = __shfl(gv, base + j * per, kWave);
            rank += o > gv || (o == gv && j < mine);
        }
        if (rank >= topk_group) {
#pragma unroll
            for (int v = 0; v < V; ++v) c[v] = kNone;
        }
    }

#pragma unroll
    for (int v = 0; v < V; ++v) {  // the id in the lowest bits
        const uint64_t u = __builtin_bit_cast(uint64_t, c[v]);
        const uint32_t flip = ~(uint32_t)((int64_t)u >> 63) & (kRouteMaxE - 1);
        c[v] = __builtin_bit_cast(double, (u & ~(uint64_t)(kRouteMaxE - 1)) |
                                              ((uint32_t)(i * V + v) ^ flip));
    }
    sort_down<V>(c);
    int my_id = -1;
    auto take = [&](auto depth) {
        constexpr int D = decltype(depth)::value;
        for (int k = 0; k < K; ++k) {
            const double best = lanes_max<L>(c[0]);
            const uint32_t low = (uint32_t)__builtin_bit_cast(uint64_t, best) & (kRouteMaxE - 1);
            const int id = (int)(best < 0.0 ? low : low ^ (kRouteMaxE - 1));
            if (i == k && best > 0.5 * kNone) my_id = id;
            const bool mine = c[0] == best;
#pragma unroll
            for (int v = 0; v + 1 < D; ++v) c[v] = mine ? c[v + 1] : c[v];
            c[D - 1] = mine ? kNone : c[D - 1];
        }
    };
    if (V > 8 && K <= 8)  // a lane gives at most K
        take(std::integral_constant<int, std::min(V, 8)>{});
    else
        take(std::integral_constant<int, V>{});

    const float my_l = my_id >= 0 ? clean(widen<LT>(row[my_id])) : -INFINITY;
    double s = 0.0;
    if (sig) {
        s = my_id >= 0 ? sigmoid(my_l) : 0.0;
        if (renorm) s = s / (lanes_sum<L>(s) + kRenormEps);
    } else if (renorm) {  // the softmax of the chosen
        const double m = lanes_max<L>(my_id >= 0 ? (double)my_l : kNone);
        s = my_id >= 0 ? exp_neg((double)my_l - m) : 0.0;
        const double d = lanes_sum<L>(s);
        s = d > 0.0 ? s / d : 0.0;
    } else {
        s = my_id >= 0 ? exp_neg((double)my_l - (double)top) * z : 0.0;
    }
    if (t_raw < T && i < K) {
        ids[(size_t)t * K + i] = my_id;
        scores[(size_t)t * K + i] = (float)(s * (double)scale);
    }
}

// Any shape: one wave per token; lane i holds experts i, i + 64, ... (V of
// them). For groups that do not consist of whole lanes of route_lanes.
template <typename LT, int V, bool SIGMOID>
__global__ __launch_bounds__(kRouteThreads) void route_rows(
    const LT* __restrict__ logits, const float* __restrict__ bias, int n_group, int topk_group,
    int renorm, float scale, int* __restrict__ ids, float* __restrict__ scores, int T, int E,
    int K) {
    __shared__ double s_c[kRouteWaves][kRouteMaxE];
    const int lane = lane_id();
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x) / kWave;
    const int t_raw = blockIdx.x * kRouteWaves + w;
    const int t = min(t_raw, T - 1);  // waves past T work on a real row, store nothing

    float l[V];
    double c[V];
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * kWave + lane;
        l[v] = e < E ? clean(widen(logits[(size_t)t * E + min(e, E - 1)])) : -INFINITY;
        top = fmaxf(top, l[v]);
    }
    top = (float)wave_max_d(top);
    double z = 1.0;
    if constexpr (!SIGMOID) {
        double part = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            part += l[v] > -INFINITY ? exp((double)l[v] - (double)top) : 0.0;
        z = wave_sum_d(part);
    }
    auto score = [&](float x) {
        return SIGMOID ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top) / z;
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * kWave + lane;
        c[v] = -INFINITY;
        if (l[v] > -INFINITY) c[v] = bias ? score(l[v]) + (double)bias[e] : (double)l[v];
        if (!(c[v] > -INFINITY)) c[v] = -INFINITY;  // a NaN bias
    }

    if (n_group > 1) {
        const int per = E / n_group;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * kWave + lane < E) s_c[w][v * kWave + lane] = c[v];
        __syncthreads();
        double a = -INFINITY, b = -INFINITY;  // the group's two largest
        if (lane < n_group)
            for (int i = 0; i < per; ++i) {
                const double x = s_c[w][lane * per + i];
                b = fmax(b, fmin(a, x));
                a = fmax(a, x);
            }
        const double gv = bias && b > -INFINITY ? a + b : a;
        int rank = 0;
        for (int j = 0; j < n_group; ++j) {
            const double o = __shfl(gv, j, kWave);
            rank += o > gv || (o == gv && j < lane);
        }
        const uint64_t keep = __ballot(lane < n_group && rank < topk_group);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = min(v * kWave + lane, E - 1);
            if (!((keep >> (e / per)) & 1)) c[v] = -INFINITY;
        }
    }

    int my_id = -1;
    float my_l = -INFINITY;
    for (int k = 0; k < K; ++k) {
        double best = -INFINITY;
        int at = 0x7fffffff;
        float bl = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c[v] > best) { best = c[v]; at = v * kWave + lane; bl = l[v]; }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) {
            const double ob = __shfl_xor(best, m, kWave);
            const int oa = __shfl_xor(at, m, kWave);
            const float ol = __shfl_xor(bl, m, kWave);
            if (ob > best || (ob == best && oa < at)) { best = ob; at = oa; bl = ol; }
        }
        if (!(best > -INFINITY)) break;  // none left: the rest stay -1
        if (lane == k) { my_id = at; my_l = bl; }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (at == v * kWave + lane) c[v] = -INFINITY;
    }

    double s = 0.0;
    if (my_id >= 0) {
        // a renormalised softmax is the softmax of the chosen
        s = !SIGMOID && renorm ? exp((double)my_l - (double)top) : score(my_l);
    }
    if (renorm) {
        if (!SIGMOID) {
            const double m = wave_max_d(my_id >= 0 ? (double)my_l : -INFINITY);
            s = my_id >= 0 ? exp((double)my_l - m) : 0.0;
            const double d = wave_sum_d(s);
            s = d > 0.0 ? s / d : 0.0;
        } else {
            s = s / (wave_sum_d(s) + kRenormEps);
        }
    }
    if (t_raw < T && lane < K) {
        ids[(size_t)t * K + lane] = my_id;
        scores[(size_t)t * K + lane] = (float)(s * (double)scale);
    }
}

// Gradient of the scores with respect to the logits. With d = dscores:
//   g = scale * d[j], renormalised: (g_j - sum_i g_i w_i) / (sum s + eps)
//   sigmoid           dl[j] = g_j s_j (1 - s_j) at the chosen, 0 elsewhere
//   softmax renorm    dl[j] = w_j (g_j - sum_i g_i w_i) at the chosen
//   softmax           dl[e] = s_e ((chosen: g_e) - sum_i g_i s_i) everywhere
//
// L lanes per token; lane j < K has the j-th chosen expert, and in the last
// form each lane E / L experts. The row is put together in LDS, where the
// chosen land by id, and leaves in 16-byte stores. Only the last form reads
// whole rows; the others read the chosen logits, which still touches most
// of a row's lines, so all are bound by reading and writing the rows once:
// 9.2 us for 32768 tokens of 256 experts, sigmoid, fp32, 7.5 TB/s (some of it
// from the caches). Several tokens a wave: one token a wave spent its life in
// the chain ids, logits, sums, 27.7 us.
template <typename LT, int L>
__global__ __launch_bounds__(kRouteThreads) void route_grad_lanes(
    const LT* __restrict__ logits, const int* __restrict__ ids, const float* __restrict__ dscores,
    int sig, int renorm, float scale, LT* __restrict__ dlogits, int wide, int T, int E, int K) {
    constexpr int kTokens = kRouteThreads / L;
    extern __shared__ float s_rows[];  // [kTokens][pitch]
    const int pitch = (E + 3) & ~3;
    const int lane = lane_id(), i = lane & (L - 1), base = lane & ~(L - 1);
    const int t_raw = blockIdx.x * kTokens + threadIdx.x / L;
    const int t = min(t_raw, T - 1);  // lanes past T work on a real row, store nothing
    const LT* row = logits + (size_t)t * E;
    float* out = s_rows + (threadIdx.x / L) * pitch;

    int id = i < K ? ids[(size_t)t * K + i] : -1;
    double g = i < K ? (double)dscores[(size_t)t * K + i] * (double)scale : 0.0;
    if ((unsigned)id >= (unsigned)E) id = -1;
    const float lj = id >= 0 ? clean(widen<LT>(row[id])) : -INFINITY;
    const bool live = lj > -INFINITY;
    if (!live) g = 0.0;
    const bool dense = !sig && !renorm;

    double dl;  // of the chosen
    if (dense) {
        float m = -INFINITY;
        for (int e = i; e < E; e += L) m = fmaxf(m, clean(widen<LT>(row[e])));
        const double top = lanes_max<L>(m);
        double z = 0.0;
        for (int e = i; e < E; e += L) {
            const float l = clean(widen<LT>(row[e]));
            z += l > -INFINITY ? exp_neg((double)l - top) : 0.0;
        }
        z = lanes_sum<L>(z);
        const double r = z > 0.0 ? 1.0 / z : 0.0;
        const double s = live ? exp_neg((double)lj - top) * r : 0.0;
        const double dot = lanes_sum<L>(g * s);
        double twice = 0.0;  // an id given again adds its g
        for (int k = 0; k < K; ++k) {
            const double o = __shfl(g, base + k, kWave);
            if (__shfl(id, base + k, kWave) == id) twice += o;
        }
        dl = s * (twice - dot);
        for (int e = i; e < E; e += L) {
            const float l = clean(widen<LT>(row[e]));
            out[e] = l > -INFINITY ? (float)(-dot * (exp_neg((double)l - top) * r)) : 0.0f;
        }
    } else {
        if (sig) {
            const double x = live ? exp_neg(-fabs((double)lj)) : 0.0;  // s(1-s) = x / (1+x)^2
            const double y = reciprocal(1.0 + x);
            const double s = live ? (lj >= 0.0f ? y : x * y) : 0.0;
            if (renorm) {
                const double d = lanes_sum<L>(s) + kRenormEps;
                g = (g - lanes_sum<L>(g * (s / d))) / d;
            }
            dl = live ? g * (x * y * y) : 0.0;
        } else {
            const double m = lanes_max<L>(live ? (double)lj : kNone);
            const double x = live ? exp_neg((double)lj - m) : 0.0;
            const double d = lanes_sum<L>(x);
            const double w = d > 0.0 ? x / d : 0.0;
            dl = w * (g - lanes_sum<L>(g * w));
        }
        double all = 0.0;  // in k order: an id given again adds up
        for (int k = 0; k < K; ++k) {
            const double o = __shfl(dl, base + k, kWave);
            if (__shfl(id, base + k, kWave) == id) all += o;
        }
        dl = all;
        for (int e = i * 4; e < pitch; e += L * 4)
            *(rows::f32x4*)(out + e) = rows::f32x4{0, 0, 0, 0};
    }
    // a token's lanes lie in one wave, whose LDS operations stay in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (live) out[id] = (float)dl;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (t_raw >= T) return;
    LT* dst = dlogits + (size_t)t * E;
    if (wide) {
        constexpr int N = 16 / sizeof(LT);
        typedef LT vec __attribute__((ext_vector_type(N)));
        for (int e = i * N; e < E; e += L * N) {
            vec v;
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = narrow<LT>(out[e + k]);
            __builtin_nontemporal_store(v, (vec*)(dst + e));
        }
    } else {
        for (int e = i; e < E; e += L) dst[e] = narrow<LT>(out[e]);
    }
}

template <typename LT, int V>
void launch_route(hipStream_t s, bool sig, const void* logits, const float* bias, int ng, int tg,
                  int renorm, float scale, int* ids, float* scores, int T, int E, int K) {
    const dim3 g((T + kRouteWaves - 1) / kRouteWaves), b(kRouteThreads);
    if (sig)
        hipLaunchKernelGGL((route_rows<LT, V, true>), g, b, 0, s, (const LT*)logits, bias, ng, tg,
                           renorm, scale, ids, scores, T, E, K);
    else
        hipLaunchKernelGGL((route_rows<LT, V, false>), g, b, 0, s, (const LT*)logits, bias, ng, tg,
                           renorm, scale, ids, scores, T, E, K);
}

template <typename LT, int L, int V>
bool try_lanes(hipStream_t s, bool sig, const void* logits, const float* bias, int ng, int tg,
               int renorm, float scale, int* ids, float* scores, int T, int E, int K) {
    if (E > L * V || K > L || (ng > 1 && (E / ng) % V != 0)) return false;
    static_assert(V % kLaneVec<LT, V> == 0, "whole vectors per lane");
    constexpr size_t kVec = kLaneVec<LT, V> * sizeof(LT);
    const int wide = E % V == 0 && (E * sizeof(LT)) % kVec == 0 && (uintptr_t)logits % kVec == 0;
    constexpr int kTokens = kRouteThreads / L;
    hipLaunchKernelGGL((route_lanes<LT, L, V>), dim3((T + kTokens - 1) / kTokens),
                       dim3(kRouteThreads), 0, s, (const LT*)logits, bias, sig ? 1 : 0, wide, ng,
                       tg, renorm, scale, ids, scores, T, E, K);
    return true;
}

template <typename LT>
void dispatch_route(hipStream_t s, bool sig, const void* logits, const float* bias, int ng, int tg,
                    int renorm, float scale, int* ids, float* scores, int T, int E, int K) {
#define MEP_TRY(L, V)                                                                          \
    if (try_lanes<LT, L, V>(s, sig, logits, bias, ng, tg, renorm, scale, ids, scores, T, E, K)) \
        return;
    if (T >= kRouteManyTokens) {
        MEP_TRY(16, 4)
        MEP_TRY(16, 8)
        MEP_TRY(16, 16)
        MEP_TRY(32, 4)
        MEP_TRY(32, 8)
        MEP_TRY(32, 12)
        MEP_TRY(32, 16)
    }
    MEP_TRY(64, 4)
    MEP_TRY(64, 8)
    MEP_TRY(64, 12)
    MEP_TRY(64, 16)
#undef MEP_TRY
    if (E <= 256)
        launch_route<LT, 4>(s, sig, logits, bias, ng, tg, renorm, scale, ids, scores, T, E, K);
    else if (E <= 512)
        launch_route<LT, 8>(s, sig, logits, bias, ng, tg, renorm, scale, ids, scores, T, E, K);
    else
        launch_route<LT, 16>(s, sig, logits, bias, ng, tg, renorm, scale, ids, scores, T, E, K);
}

template <typename LT, int L>
void launch_route_grad(hipStream_t s, bool sig, const void* logits, const int* ids,
                       const float* ds, int renorm, float scale, void* dl, int T, int E, int K) {
    constexpr int kTokens = kRouteThreads / L;
    const int wide = (E * sizeof(LT)) % 16 == 0 && (uintptr_t)dl % 16 == 0;
    hipLaunchKernelGGL((route_grad_lanes<LT, L>), dim3((T + kTokens - 1) / kTokens),
                       dim3(kRouteThreads), (size_t)kTokens * ((E + 3) & ~3) * 4, s,
                       (const LT*)logits, ids, ds, sig ? 1 : 0, renorm, scale, (LT*)dl, wide, T, E,
                       K);
}

// Whole waves for few tokens (a token's chain of steps is shorter), for many
// chosen, and for rows of which 16 tokens would not fit a work-group's LDS.
template <typename LT>
void dispatch_route_grad(hipStream_t s, bool sig, const void* logits, const int* ids,
                         const float* ds, int renorm, float scale, void* dl, int T, int E, int K) {
    if (T >= kRouteManyTokens && K <= 16 && E <= 512)
        launch_route_grad<LT, 16>(s, sig, logits, ids, ds, renorm, scale, dl, T, E, K);
    else
        launch_route_grad<LT, 64>(s, sig, logits, ids, ds, renorm, scale, dl, T, E, K);
}

bool known_dtype(int d) {
    return d == MEP_SCALE_F32 || d == MEP_SCALE_BF16 || d == MEP_SCALE_F16;
}

bool aligned_to(const void* p, int dtype) {
    return ((uintptr_t)p & (dtype == MEP_SCALE_F32 ? 3u : 1u)) == 0;
}

}  // namespace
}  // namespace mep

using namespace mep;

extern "C" int mep_route(int T, int E, int K, const void* logits, int logit_dtype,
                         const float* bias, int scoring, int n_group, int topk_group,
                         int renormalize, float scale, int32_t* topk_ids, float* scores,
                         void* stream) {
    if (T < 0 || T >= kRouteMaxT || E < 1 || E > kRouteMaxE || K < 1 || K > kRouteMaxK ||
        (long long)T * K >= (1ll << 31))
        return MEP_ERR_SHAPE;
    if (n_group < 1 || n_group > kRouteMaxGroups || E % n_group != 0 || topk_group < 1 ||
        topk_group > n_group || K > topk_group * (E / n_group) || !known_dtype(logit_dtype) ||
        (scoring != MEP_SCORE_SOFTMAX && scoring != MEP_SCORE_SIGMOID) ||
        !(scale > -3.0e38f && scale < 3.0e38f))
        return MEP_ERR_PARAM;
    if (T == 0) return MEP_OK;
    if (!logits || !topk_ids || !scores) return MEP_ERR_NULLPTR;
    if (!aligned_to(logits, logit_dtype)) return MEP_ERR_SHAPE;
    const bool sig = scoring == MEP_SCORE_SIGMOID;
    hipStream_t s = (hipStream_t)stream;
    int* ids = (int*)topk_ids;
    if (logit_dtype == MEP_SCALE_F32)
        dispatch_route<float>(s, sig, logits, bias, n_group, topk_group, renormalize, scale, ids, scores, T, E, K);
    else if (logit_dtype == MEP_SCALE_BF16)
        dispatch_route<uint16_t>(s, sig, logits, bias, n_group, topk_group, renormalize, scale, ids, scores, T, E, K);
    else
        dispatch_route<_Float16>(s, sig, logits, bias, n_group, topk_group, renormalize, scale, ids, scores, T, E, K);
    MEP_LAUNCH_CHECK();
    return MEP_OK;
}

extern "C" int mep_route_grad(int T, int E, int K, const void* logits, int logit_dtype,
                              const int32_t* topk_ids, const float* dscores, int scoring,
                              int renormalize, float scale, void* dlogits, void* stream) {
    if (T < 0 || T >= kRouteMaxT || E < 1 || E > kRouteMaxE || K < 1 || K > kRouteMaxK || K > E ||
        (long long)T * K >= (1ll << 31))
        return MEP_ERR_SHAPE;
    if (!known_dtype(logit_dtype) ||
        (scoring != MEP_SCORE_SOFTMAX && scoring != MEP_SCORE_SIGMOID) ||
        !(scale > -3.0e38f && scale < 3.0e38f))
        return MEP_ERR_PARAM;
    if (T == 0) return MEP_OK;
    if (!logits || !topk_ids || !dscores || !dlogits) return MEP_ERR_NULLPTR;
    if (!aligned_to(logits, logit_dtype) || !aligned_to(dlogits, logit_dtype))
        return MEP_ERR_SHAPE;
    const bool sig = scoring == MEP_SCORE_SIGMOID;
    hipStream_t s = (hipStream_t)stream;
    const int* ids = (const int*)topk_ids;
    if (logit_dtype == MEP_SCALE_F32)
        dispatch_route_grad<float>(s, sig, logits, ids, dscores, renormalize, scale, dlogits, T, E, K);
    else if (logit_dtype == MEP_SCALE_BF16)
        dispatch_route_grad<uint16_t>(s, sig, logits, ids, dscores, renormalize, scale, dlogits, T, E, K);
    else
        dispatch_route_grad<_Float16>(s, sig, logits, ids, dscores, renormalize, scale, dlogits, T, E, K);
    MEP_LAUNCH_CHECK();
    return MEP_OK;
}
