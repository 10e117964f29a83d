// Kernels of the experts' products for a few routes (gfx950, wave64): the
// routed product y = W[id] x and the two halves of the expert layer. The
// weights are read once per expert that any route reaches; everything else
// is small, so the kernels stream weights and are bound by HBM.
//
// Products run on the matrix cores (16x16x32 bf16 MFMA, fp32 sums): columns
// are routes, so a route's products never mix with another's and a NaN in
// one stays there. The MFMA wants lane l (i = l % 16, q = l / 16) to hold
// row i, inputs 8q..8q+7 of A and column i, the same inputs, of B. Loading
// 16 weight rows like that touches 64 bytes of a row per instruction, and
// such reads reached 5.4-6.0 TB/s where whole 128-byte lines reach 7.1. So
// an MFMA here takes 8 rows and 64 inputs: lanes i < 8 hold row i and the
// first 32 inputs, lanes i >= 8 row i - 8 and the other 32, and B likewise
// holds 8 routes, the first 32 inputs in columns 0-7 and the other 32 in
// columns 8-15. Of the 16x16 results the blocks (rows 0-7, columns 0-7) and
// (rows 8-15, columns 8-15) are the two halves of the wanted 8x8 sums, the
// other two mean nothing. Lane l's four results are rows 4q..4q+3 of column
// i; the second half of lane l's sum lies in lane l + 40. Up to 8 routes
// cost one MFMA per KiB of weights this way, and 16 columns are not half
// idle when few routes share an expert.
#pragma once

#include <utility>

#include "rows.h"

namespace mep {
namespace experts {

using rows::f32x4;
using rows::u32x4;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Register arrays that a lambda captures stay registers only if it is inlined.
#define MEP_INLINE __attribute__((always_inline))

// f(0), f(1), .. f(N - 1) with constant arguments, up to the first that
// returns true; whether one did.
template <class F, int... I>
__device__ __forceinline__ bool any_of(F f, std::integer_sequence<int, I...>) {
    return (f(std::integral_constant<int, I>{}) || ...);
}
template <int N, class F>
__device__ __forceinline__ bool any_of(F f) {
    return any_of(f, std::make_integer_sequence<int, N>{});
}

constexpr int kTile = 8;        // weight rows of one MFMA
constexpr int kStep = 64;       // inputs of one MFMA
constexpr int kCols = 8;        // routes of one MFMA
constexpr int kPackK = 256;     // inputs of one packed 4-bit block
constexpr int kMaxRoutes = 2048;
constexpr int kMaxExperts = 1024;
constexpr int kMaxLayerTokens = 128;
constexpr int kMaxWaves = 16;

// Routed list that the layer's first kernel leaves for its second.
struct Table {
    int n_slots;
    int expert[kMaxExperts];     // of slot s, ascending
    int offset[kMaxExperts + 1]; // of slot s in `route`
    uint16_t route[kMaxRoutes];  // grouped by expert, ascending inside
};

struct Weights {
    const u32x4* codes;
    const uint16_t* scales;  // bits of bf16 or fp16
    const uint8_t* zeros;
    int N, K;
    int KV;     // K / 8, inputs in vectors of 8
    int tiles;  // packed: ceil(N / 8)
    int KB;     // packed: ceil(K / 256)
};

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Loads from a buffer (its base and size in scalar registers) at a scalar
// offset plus a byte offset per lane: stepping through it costs no vector
// instruction, and a load past its end returns 0. `kNt` streams past the
// caches (weights are used once).
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr int kNt = 2;
constexpr uint32_t kPast = 0x80000000u;  // an offset past every buffer's end

__device__ __forceinline__ Buffer buffer_of(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, bytes, 0x00027000);
}
template <typename T, int AUX>
__device__ __forceinline__ T buffer_load(Buffer b, uint32_t lane_bytes, uint32_t bytes) {
    if constexpr (sizeof(T) == 16)
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b128(b, lane_bytes, bytes, AUX));
    else if constexpr (sizeof(T) == 8)
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b64(b, lane_bytes, bytes, AUX));
    else
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(b, lane_bytes, bytes, AUX));
}

// Vector (8 inputs) of a 64-input step that a lane holds: q, or q + 4 in the
// lanes of the second half.
__device__ __forceinline__ int lane_vec(int lane) { return (lane >> 4) + ((lane >> 3) & 1) * 4; }

// ---------------------------------------------------------------- weights
//
// A weight kind gives: kSteps (MFMA steps of one chunk), Ptr (where a lane's
// part of one 8-row tile starts), Reg (one chunk of it in registers), load,
// and mma (chunk times NB column blocks).

// WHOLE: K is a multiple of a chunk. Otherwise, in the chunk that K cuts, a
// lane's vectors past K lie in the next row and are loaded from past the
// buffer, as zeros; the selects this takes cost 4 us of 80 on 7168 inputs.
template <bool WHOLE>
struct Bf16Weights {
    static constexpr int kSteps = 2;
    static constexpr int kMaxHeld = 4;   // chunks of inputs that a wave can hold
    static constexpr bool kWide = true;  // whether expert_down takes four tiles at a time
    struct Reg {
        u32x4 a[kSteps];
    };
    struct Ptr {
        Buffer rows;
    };
    struct Lane {
        int left;  // vectors of the row from the lane's first on
        uint32_t bytes;
    };
    static __device__ __forceinline__ Lane lane_of(const Weights& w, int lane) {
        const int v = lane_vec(lane);
        return {w.KV - v, (uint32_t)((lane & 7) * w.KV + v) * 16u};
    }
    static __device__ __forceinline__ Ptr at(const Weights& w, int e, int row0) {
        const u32x4* p = w.codes + ((size_t)e * w.N + min(row0, w.N - kTile)) * w.KV;
        return {buffer_of(p, (uint32_t)(kTile * w.KV) * 16u)};
    }
    static __device__ __forceinline__ void load(Reg& r, const Ptr& p, const Lane& l, int c) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
            r.a[j] = buffer_load<u32x4, kNt>(
                p.rows,
                WHOLE || (c * kSteps + j) * 8 < l.left ? l.bytes + j * 128 : kPast,
                c * (kSteps * 128));
    }
    // acc += r x over the SN steps from S0 on.
    template <int S0, int SN, int NT, int NB>
    static __device__ __forceinline__ void mma(const Reg (&r)[NT], const u32x4 (&x)[NB][SN],
                                               f32x4 (&acc)[NT][NB]) {
#pragma unroll
        for (int j = 0; j < SN; ++j)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < NT; ++i) acc[i][b] = mfma(r[i].a[S0 + j], x[b][j], acc[i][b]);
    }
};

// 4-bit codes in the packed layout (pack4.hip): 1 KiB per 8 rows and 256
// inputs, 16 bytes per lane, one word per step; scales and zero points
// [tile][block][2 row quads][groups][4 rows], the order in which the
// accumulators' lanes need them (groups of 32: those of the steps' first
// halves, then those of the second, since lanes q >= 2 hold the latter).
//
// An int4 code q becomes the bf16 number 16 + q by or-ing it into the upper
// mantissa bits of 16 (a shift, and an and-or, per two codes). The constant
// is taken out of the sum again by a product of the same inputs with a
// constant row, -(16 + 8) for symmetric codes, whose result is the
// accumulator that the code product starts from:
// sum (16 + q) x - sum 24 x = sum (q - 8) x. With zero points the constant
// row is -16 and z of the row times sum x = -1/16 of that result is
// subtracted per row. All terms are exact products summed in fp32; 16 is the
// smallest power of two that keeps all sixteen codes in one binade, so the
// terms are at most 7 times larger than the result's. (With the code in the
// lowest mantissa bits the constant is 128: an fp32 output was 1.3e-6 from
// the exact one where 3e-7 is fp32's share.)
// A 4-bit float is converted by the hardware, two codes per instruction.
template <bool FP4, int G, bool ZP, bool F16>
struct PackedWeights {
    static constexpr int kSteps = 4;
    static constexpr int kMaxHeld = 2;
    static constexpr bool kWide = G == 128;
    static constexpr int SM = G == 128 ? 2 : 1;  // steps per scale
    static constexpr int GL = kSteps / SM;       // scales per lane, row and chunk
    static constexpr int GP = kPackK / G;        // groups per block
    struct Ptr {
        Buffer codes, scales, zeros;
    };
    struct Lane {
        uint32_t bytes, group;  // group: of the zero points, which take 1 byte a row
    };
    struct Reg {
        u32x4 a;
        uint32_t s[GL * 2];
        uint32_t z[ZP ? GL : 1];
    };
    static __device__ __forceinline__ Lane lane_of(const Weights&, int lane) {
        return {(uint32_t)lane * 16u,
                (uint32_t)(((lane >> 4) & 1) * GP + (G == 32 ? (lane >> 5) * GL : 0)) * 4u};
    }
    static __device__ __forceinline__ Ptr at(const Weights& w, int e, int row0) {
        const size_t tile = (size_t)e * w.tiles + min(row0 / kTile, w.tiles - 1);
        const size_t g = tile * w.KB * (8 * GP);
        const uint32_t n = (uint32_t)w.KB * (8 * GP);
        Ptr p;
        p.codes = buffer_of(w.codes + tile * w.KB * 64, (uint32_t)w.KB * 1024u);
        p.scales = buffer_of(w.scales + g, n * 2u);
        if constexpr (ZP) p.zeros = buffer_of(w.zeros + g, n);
        return p;
    }
    static __device__ __forceinline__ void load(Reg& r, const Ptr& p, const Lane& l, int c) {
        r.a = buffer_load<u32x4, kNt>(p.codes, l.bytes, c * 1024);
#pragma unroll
        for (int i = 0; i < GL / 2; ++i) {
            const u32x4 s = buffer_load<u32x4, 0>(p.scales, l.group * 2 + i * 16, c * (16 * GP));
#pragma unroll
            for (int k = 0; k < 4; ++k) r.s[i * 4 + k] = s[k];
            if constexpr (ZP) {
                const u32x2 z = buffer_load<u32x2, 0>(p.zeros, l.group + i * 8, c * (8 * GP));
                r.z[i * 2] = z[0];
                r.z[i * 2 + 1] = z[1];
            }
        }
    }
    static __device__ __forceinline__ float scale(uint32_t w, int hi) {
        if constexpr (F16) {
            const uint16_t b = (uint16_t)(hi ? w >> 16 : w);
            return (float)__builtin_bit_cast(_Float16, b);
        }
        return __uint_as_float(hi ? w & 0xffff0000u : w << 16);
    }
    // k16: 16.0 twice. Given in a vector register, so that the mask (a
    // scalar) and it fit one v_and_or_b32; as two constants they took two
    // instructions.
    static __device__ __forceinline__ uint32_t offset_bits() {
        uint32_t k16 = 0x41804180u;
        asm("" : "+v"(k16));
        return k16;
    }
    static __device__ __forceinline__ u32x4 decode(uint32_t d, uint32_t k16) {
        u32x4 o;
        if constexpr (FP4) {
            o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 0));
            o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 1));
            o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 2));
            o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 3));
        } else {
            o[0] = (d & 0x00780078u) | k16;
            o[1] = ((d >> 4) & 0x00780078u) | k16;
            o[2] = ((d >> 8) & 0x00780078u) | k16;
            o[3] = (__builtin_amdgcn_alignbit(d, d, 12) & 0x00780078u) | k16;
        }
        return o;
    }
    template <int S0, int SN, int NT, int NB>
    static __device__ __forceinline__ void mma(const Reg (&r)[NT], const u32x4 (&x)[NB][SN],
                                               f32x4 (&acc)[NT][NB]) {
        static_assert(S0 % SM == 0 && SN % SM == 0, "whole groups");
        constexpr uint32_t kOff = ZP ? 0xc180c180u : 0xc1c0c1c0u;  // -16, -24
        const u32x4 off = {kOff, kOff, kOff, kOff};
        const uint32_t k16 = offset_bits();
#pragma unroll
        for (int g = S0 / SM; g < (S0 + SN) / SM; ++g) {
            f32x4 x0[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                x0[b] = f32x4{0, 0, 0, 0};
                if constexpr (!FP4) {
#pragma unroll
                    for (int j = 0; j < SM; ++j) x0[b] = mfma(off, x[b][g * SM + j - S0], x0[b]);
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                f32x4 c[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) c[b] = x0[b];
#pragma unroll
                for (int j = 0; j < SM; ++j) {
                    const u32x4 a = decode(r[i].a[g * SM + j], k16);
#pragma unroll
                    for (int b = 0; b < NB; ++b) c[b] = mfma(a, x[b][g * SM + j - S0], c[b]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float s = scale(r[i].s[g * 2 + k / 2], k & 1);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float v = c[b][k];
                        if constexpr (ZP) {
                            const float z = (float)((r[i].z[g] >> (8 * k)) & 0xffu) * (1.0f / 16);
                            v = __builtin_fmaf(z, x0[b][k], v);
                        }
                        acc[i][b][k] = __builtin_fmaf(s, v, acc[i][b][k]);
                    }
                }
            }
        }
    }
};

// ----------------------------------------------------------------- inputs

// A route's inputs as bf16 terms to be summed: one for bf16 rows read as they
// are; for the layer's h (fp32) each term is the rest of the ones before,
// rounded (two terms lose at most 2^-17 of the value, three at most 2^-25),
// stored per 8 values as 16 bytes of each term. Two terms serve a bf16
// output (its own rounding is 2^-8), three an fp32 one: with two, an fp32
// output measured 2.7e-6 from the exact result where 2.5e-7 is fp32's share.
// The terms of a route take columns of their own, kRoutes routes to a block
// of 8 columns: column c holds term c / kRoutes of route c % kRoutes. An
// expert rarely sees more than a few of a decode step's routes, so these
// columns would mostly stand empty, and the terms then cost no product and
// no load of their own. Inputs past K count as zero. The lanes of a column
// past the last route (or term) read a real one; their column is not used.
template <int TERMS>
struct Input {
    static constexpr int kRoutes = TERMS == 1 ? 8 : TERMS == 2 ? 4 : 2;
    int left;        // vectors of the row from the lane's first on
    uint32_t bytes;  // where the lane's first vector of the route's row lies
    __device__ __forceinline__ void row(int r, int KV, int lane) {
        const uint32_t term = min((lane & 7) / kRoutes, TERMS - 1);
        left = KV - lane_vec(lane);
        bytes = (((uint32_t)r * KV + lane_vec(lane)) * TERMS + term) * 16u;
    }
    // Chunk c in chunks of STEPS steps; WHOLE: rows are whole chunks.
    template <bool WHOLE, int STEPS>
    __device__ __forceinline__ void load(u32x4 (&x)[STEPS], Buffer b, int c) const {
#pragma unroll
        for (int j = 0; j < STEPS; ++j)
            x[j] = buffer_load<u32x4, 0>(
                b, WHOLE || (c * STEPS + j) * 8 < left ? bytes + j * (128 * TERMS) : kPast,
                c * (STEPS * 128 * TERMS));
    }
    // The wanted sum of a lane i < kRoutes, q < 2: both halves of the inputs
    // and all terms.
    static __device__ __forceinline__ float total(float v, int lane) {
        v = v + __shfl(v, (lane + 40) & 63, kWave);
        float o = v;
#pragma unroll
        for (int t = 1; t < TERMS; ++t) o = o + __shfl(v, (lane + t * kRoutes) & 63, kWave);
        return o;
    }
};

// Inputs of a row of h, padded with zeros.
__host__ __device__ __forceinline__ int padded(int I) { return (I + kPackK - 1) / kPackK * kPackK; }

template <class W>
__host__ __device__ __forceinline__ int chunks(int K) {
    return (K + W::kSteps * kStep - 1) / (W::kSteps * kStep);
}

// acc[i][b] += tile i of the weights times column block b over chunks
// [lo, hi), the loads of the next D - 1 chunks in flight while one is used.
// The loop has no branch around its loads: where two paths with and without
// loads meet, the compiler waits for all of them before the next use, which
// undoes the prefetch. So past the end the last chunk is loaded again.
template <class W, int D, int TERMS, int NT, int NB>
__device__ __forceinline__ void stream(const Weights& w, const typename W::Ptr (&wp)[NT],
                                       Buffer xb, const Input<TERMS> (&xp)[NB], int lo, int hi,
                                       int lane, f32x4 (&acc)[NT][NB]) {
    if (lo >= hi) return;
    typename W::Reg r[D][NT];
    u32x4 x[D][NB][W::kSteps];
    const typename W::Lane l = W::lane_of(w, lane);
    auto load = [&](int d, int c) MEP_INLINE {
        c = min(c, hi - 1);
#pragma unroll
        for (int i = 0; i < NT; ++i) W::load(r[d][i], wp[i], l, c);
#pragma unroll
        for (int b = 0; b < NB; ++b) xp[b].template load<false>(x[d][b], xb, c);
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) load(d, lo + d);
    for (int c = lo;;) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            load((d + D - 1) % D, c + D - 1);
            W::template mma<0, W::kSteps, NT, NB>(r[d], x[d], acc);
            if (++c >= hi) return;
        }
    }
}

// --------------------------------------------------- products per expert

struct RowsArgs {
    const u32x4* x;      // input rows, K inputs each
    int div;             // route r reads row r / div
    const int* ids;      // [n], or NULL: every route goes to matrix 0
    const uint8_t* mask; // [n] or NULL
    int n, first, E;
    Weights w;
    // product
    void* out;           // [n, N] bf16 or fp32
    int out_f32;
    // first half of the layer
    u32x4* h;            // [n][padded(I) / 8][terms]
    int I, terms;
    Table* table;
};

// Up to 64 routes, one per lane: every wave finds experts and routes by
// itself in registers, with no barrier (the decode of a few tokens is mostly
// waiting). Experts are ordered by their first route.
struct FewRoutes {
    int id;          // this lane's expert, or -1
    uint64_t peers;  // the lanes of that expert
    int first;       // the lowest of them (64 where id is -1)

    static __device__ __forceinline__ FewRoutes read(const int* ids, const uint8_t* mask, int n,
                                                     int first_id, int E) {
        FewRoutes f;
        const int lane = lane_id();
        f.id = -1;
        if (lane < n) {
            // in 64 bits: an id far outside may not wrap into the range
            const long long v = (long long)ids[lane] - first_id;
            if (v >= 0 && v < E && !(mask && mask[lane] == 0)) f.id = (int)v;
        }
        f.peers = match_peers<kKeyBits>(f.id, f.id >= 0);
        f.first = f.id >= 0 ? (int)__builtin_ctzll(f.peers) : kWave;
        return f;
    }
    // Jobs of `per` routes: a lane that is its expert's first gets the number
    // of its expert's jobs, other lanes 0.
    __device__ __forceinline__ int jobs(int per) const {
        return first == lane_id() ? (__popcll(peers) + per - 1) / per : 0;
    }
    // This route's place in a list ordered by (expert's first route, route).
    __device__ __forceinline__ int place() const {
        const int ends = wave_inclusive_sum(first == lane_id() ? __popcll(peers) : 0);
        return __shfl(ends, first & (kWave - 1), kWave) - __popcll(peers) + count_below(peers);
    }
};

// The experts that any route reaches, jobs of up to 8 of an expert's routes,
// and an expert's routes in route order. All threads of the work-group take
// part in each call.
struct Finder {
    int16_t id[kMaxRoutes];
    uint16_t list[kMaxRoutes];
    uint16_t routes[kMaxExperts];  // of each expert
    uint16_t job[kMaxRoutes];      // its expert; a job's place among its expert's
    uint8_t pass[kMaxRoutes];      // jobs, 8 routes each
    int count[kMaxWaves], less[kMaxWaves], slots, jobs;

    // Reads the ids; returns the number of jobs.
    __device__ __forceinline__ int begin(const RowsArgs& a, FewRoutes& few) {
        const int tid = threadIdx.x;
        if (a.n <= kWave) {
            few = FewRoutes::read(a.ids, a.mask, a.n, a.first, a.E);
            return __builtin_amdgcn_readlane(wave_inclusive_sum(few.jobs(kCols)), kWave - 1);
        }
        // counted in pairs of 16 bits: no more than 2048 routes
        uint32_t* pairs = (uint32_t*)routes;
        for (int i = tid; i < kMaxExperts / 2; i += blockDim.x) pairs[i] = 0u;
        lds_barrier();
        for (int i = tid; i < a.n; i += blockDim.x) {
            // in 64 bits: an id far outside may not wrap into the range
            const long long v = (long long)a.ids[i] - a.first;
            const bool live = v >= 0 && v < a.E && !(a.mask && a.mask[i] == 0);
            id[i] = (int16_t)(live ? (int)v : -1);
            if (live) atomicAdd(&pairs[v >> 1], 1u << (16 * (v & 1)));
        }
        lds_barrier();
        if (tid < kWave) {
            int js = 0, ss = 0;
            for (int e0 = 0; e0 < a.E; e0 += kWave) {
                const int e = e0 + tid;
                const int c = e < a.E ? routes[e] : 0;
                const int mine = (c + kCols - 1) / kCols;
                const int inc = wave_inclusive_sum(mine);
                for (int k = 0; k < mine; ++k) {
                    job[js + inc - mine + k] = (uint16_t)e;
                    pass[js + inc - mine + k] = (uint8_t)k;
                }
                js += __builtin_amdgcn_readlane(inc, kWave - 1);
                ss += __popcll(__ballot(c > 0));
            }
            if (tid == 0) {
                slots = ss;
                jobs = js;
            }
        }
        lds_barrier();
        return __builtin_amdgcn_readfirstlane(jobs);
    }

    // Expert of a job, and the job's first place among that expert's routes.
    __device__ __forceinline__ int expert_of(const RowsArgs& a, const FewRoutes& few, int j,
                                             int* c0) const {
        if (a.n <= kWave) {
            const int mine = few.jobs(kCols), to = wave_inclusive_sum(mine);
            const int at = (int)__builtin_ctzll(__ballot(j < to && j >= to - mine));
            *c0 = (j - (__builtin_amdgcn_readlane(to, at) - __builtin_amdgcn_readlane(mine, at))) *
                  kCols;
            return __builtin_amdgcn_readlane(few.id, at);
        }
        *c0 = __builtin_amdgcn_readfirstlane(pass[j]) * kCols;
        return __builtin_amdgcn_readfirstlane(job[j]);
    }

    // `list` = the routes of expert e; returns their count. *off: routes of
    // lower experts.
    __device__ __forceinline__ int find(const RowsArgs& a, const FewRoutes& few, int e,
                                        int* off_out) {
        const int lane = lane_id();
        *off_out = 0;
        if (a.n <= kWave) {  // each wave writes the same list
            const uint64_t m = __ballot(few.id == e);
            if (few.id == e) list[count_below(m)] = (uint16_t)lane;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            return __popcll(m);
        }
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x) / kWave;
        const int nw = blockDim.x / kWave;
        // each wave takes a range of whole 64-route rounds
        const int rounds = (a.n + kWave - 1) / kWave;
        const int r0 = rounds * wave / nw, r1 = rounds * (wave + 1) / nw;
        int c = 0, l = 0;
        for (int r = r0; r < r1; ++r) {
            const int i = r * kWave + lane;
            const int v = i < a.n ? id[i] : -1;
            c += __popcll(__ballot(v == e));
            l += __popcll(__ballot(v >= 0 && v < e));
        }
        if (lane == 0) {
            count[wave] = c;
            less[wave] = l;
        }
        lds_barrier();
        int base = 0, off = 0;
        for (int w = 0; w < nw; ++w) {
            if (w < wave) base += count[w];
            off += less[w];
        }
        for (int r = r0; r < r1; ++r) {
            const int i = r * kWave + lane;
            const bool mine = i < a.n && id[i] == e;
            const uint64_t m = __ballot(mine);
            if (mine) list[base + count_below(m)] = (uint16_t)i;
            base += __popcll(m);
        }
        lds_barrier();
        *off_out = off;
        return __builtin_amdgcn_readfirstlane(routes[e]);
    }

    // What the layer's second kernel reads where there are more than 64
    // routes: the slots, from work-group 0, and an expert's routes, from the
    // work-group that has its first rows.
    __device__ __forceinline__ void write_slots(Table* t) const {
        if (blockIdx.x != 0 || blockIdx.y != 0 || blockIdx.z != 0 || threadIdx.x >= kWave) return;
        const int lane = lane_id();
        int s0 = 0, off = 0;
        for (int e0 = 0; e0 < kMaxExperts; e0 += kWave) {
            const int c = routes[e0 + lane];
            const uint64_t m = __ballot(c > 0);
            const int inc = wave_inclusive_sum(c);
            if (c > 0) {
                const int s = s0 + count_below(m);
                t->expert[s] = e0 + lane;
                t->offset[s] = off + inc - c;
            }
            s0 += __popcll(m);
            off += __builtin_amdgcn_readlane(inc, kWave - 1);
        }
        if (lane == 0) {
            t->n_slots = s0;
            t->offset[s0] = off;
        }
    }
    // (and the zeros that pad its routes' rows of h)
    __device__ __forceinline__ void write_routes(const RowsArgs& a, int off, int cnt) const {
        if (a.n > kWave)
            for (int i = threadIdx.x; i < cnt; i += blockDim.x) a.table->route[off + i] = list[i];
        const int row = padded(a.I) / 8 * a.terms, from = a.I / 8 * a.terms, pad = row - from;
        for (int i = threadIdx.x; i < cnt * pad; i += blockDim.x)
            a.h[(size_t)list[i / pad] * row + from + i % pad] = u32x4{0, 0, 0, 0};
    }
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// Four results of a route (rows row..row+3), from the sums over all inputs.
template <bool LAYER>
__device__ __forceinline__ void store_rows(const RowsArgs& a, int r, int row, f32x4 v, f32x4 up) {
    if constexpr (LAYER) {
        if (row >= a.I) return;
        float h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = silu(v[k]) * up[k];
        u32x2* dst = (u32x2*)(a.h + ((size_t)r * (padded(a.I) / 8) + row / 8) * a.terms) + (row % 8) / 4;
        for (int n = 0; n < a.terms; ++n) {
            const u32x2 o = {bf16x2_bits(h[0], h[1]), bf16x2_bits(h[2], h[3])};
            dst[2 * n] = o;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float t = __uint_as_float(k & 1 ? o[k / 2] & 0xffff0000u : o[k / 2] << 16);
                // an infinite or NaN term has no rest
                h[k] = fabsf(t) < INFINITY ? h[k] - t : 0.0f;
            }
        }
    } else {
        const size_t at = (size_t)r * a.w.N + row;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (row + k >= a.w.N) break;
            if (a.out_f32)
                ((float*)a.out)[at + k] = v[k];
            else
                ((uint16_t*)a.out)[at + k] = (uint16_t)bf16x2_bits(v[k], 0.0f);
        }
    }
}

// First row of tile i of a group of NT tiles (LAYER: half of them gate rows,
// half the up rows that belong to them).
template <bool LAYER, int NT>
__device__ __forceinline__ int tile_row(const RowsArgs& a, int group, int i) {
    if constexpr (LAYER) return (i / (NT / 2)) * a.I + (group * (NT / 2) + i % (NT / 2)) * kTile;
    return (group * NT + i) * kTile;
}

// Products for few routes an expert: a work-group's waves split the inputs,
// XC chunks each, and hold their part of up to 8 routes' inputs in
// registers; then only weights move. The work-groups share all (job, row
// group) pairs equally, to one pair, and go through theirs group by group:
// tiles are loaded NT - 1 ahead, and after a group's NT tiles the waves'
// sums meet in LDS, where one wave (another each time) adds them up in wave
// order and stores them while the others go on. Measured on H 7168, I 2048:
// one token's 8 bf16 experts 82 us (5.7 TB/s, a fixed 10 us of it start and
// end), 64 int4 experts of 32 tokens 185-190 us (5.1 TB/s, near the vector
// units' limit); 16 x 8 routes of 32 fp4 experts 7168x2048 56 us (4.7 TB/s;
// the registers hold three tiles ahead, six in flight spill and take 74).
template <class W, bool LAYER, int NT, int XC>
__global__ __launch_bounds__(kMaxWaves* kWave) void expert_rows_held(const RowsArgs a,
                                                                     int groups) {
    static_assert(NT == 2 || NT == 4, "two tiles are joined at once");
    __shared__ Finder s_find;
    extern __shared__ f32x4 s_part[];  // [2][nw][NT][32]
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x) / kWave;
    const int nw = blockDim.x / kWave;
    const int KC = chunks<W>(a.w.K);
    const int ck0 = wave * XC;
    const Buffer xb = buffer_of(a.x, (uint32_t)(a.n / a.div) * a.w.KV * 16u);
    const typename W::Lane l = W::lane_of(a.w, lane);
    const int i16 = lane & 15, q = lane >> 4;
    const bool wanted = (i16 < 8) == (q < 2);
    const int part = (q >> 1) * 16 + (q & 1) * 8 + (i16 & 7);

    FewRoutes few = {};
    const int total = a.ids ? s_find.begin(a, few) : (a.n + kCols - 1) / kCols;
    if constexpr (LAYER) {
        if (a.n > kWave) s_find.write_slots(a.table);
    }
    const long long items = (long long)total * groups;
    const long long end = items * (blockIdx.x + 1) / gridDim.x;
    int turn = 0, found = -1, cnt = a.n;
    for (long long at = items * blockIdx.x / gridDim.x; at < end;) {
        const int job = (int)(at / groups), g0 = (int)(at - (long long)job * groups);
        const int g1 = (int)min((long long)groups, g0 + end - at);
        at += g1 - g0;
        int e = 0, c0 = job * kCols;
        if (a.ids) {
            e = s_find.expert_of(a, few, job, &c0);
            if (e != found) {
                int off;
                if (found >= 0) lds_barrier();  // the last expert's list has been used
                cnt = s_find.find(a, few, e, &off);
                found = e;
                if constexpr (LAYER) {
                    if (g0 == 0 && c0 == 0) s_find.write_routes(a, off, cnt);
                }
            }
        }
        u32x4 x[XC][1][W::kSteps];
        typename W::Reg r[NT][XC][1];
        f32x4 acc[NT][1][1];
        Input<1> xp;
        const int jx = min(c0 + (lane & 7), cnt - 1);
        xp.row((a.ids ? s_find.list[jx] : jx) / a.div, a.w.KV, lane);
        any_of<XC>([&](auto j) MEP_INLINE {
            const int c = min(ck0 + j, KC - 1);
            xp.template load<false>(x[j][0], xb, c);
            return false;
        });
        auto load = [&](int g, auto i) MEP_INLINE {
            const typename W::Ptr p = W::at(a.w, e, tile_row<LAYER, NT>(a, g, i));
            any_of<XC>([&](auto j) MEP_INLINE {
                W::load(r[i][j][0], p, l, min(ck0 + j, KC - 1));
                return false;
            });
        };
        auto use = [&](auto i) MEP_INLINE {
            acc[i][0][0] = f32x4{0, 0, 0, 0};
            any_of<XC>([&](auto j) MEP_INLINE {
                if (ck0 + j < KC) {
                    W::template mma<0, W::kSteps, 1, 1>(r[i][j], x[j], acc[i]);
                }
                return false;
            });
        };
        auto join = [&](int g) MEP_INLINE {
            f32x4* buf = s_part + (turn & 1) * (nw * NT * 32);
            if (wanted) {
#pragma unroll
                for (int i = 0; i < NT; ++i) buf[(wave * NT + i) * 32 + part] = acc[i][0][0];
            }
            lds_barrier();
            // Lane: half of the inputs (bit 4), one of two tiles (bit 5). The
            // next write to this buffer comes two groups later, after a
            // barrier that this wave only reaches when it is done here.
            if (turn % nw == wave) {
#pragma unroll
                for (int u = 0; u < NT / 2; ++u) {
                    const int i = LAYER ? u + (lane >> 5) * (NT / 2) : u * 2 + (lane >> 5);
                    f32x4 v = {0, 0, 0, 0}, o;
                    for (int w = 0; w < nw; ++w) {
                        const f32x4 t = buf[(w * NT + i) * 32 + (lane & 31)];
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = v[k] + t[k];
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        v[k] = v[k] + __shfl(v[k], lane ^ 16, kWave);
                        o[k] = LAYER ? __shfl(v[k], lane ^ 32, kWave) : 0.0f;
                    }
                    const int j = c0 + (lane & 7);
                    const int row =
                        tile_row<LAYER, NT>(a, g, LAYER ? u : i) + ((lane >> 3) & 1) * 4;
                    if ((lane & 16) == 0 && (!LAYER || lane < 32) && j < cnt)
                        store_rows<LAYER>(a, a.ids ? s_find.list[j] : j, row, v, o);
                }
            }
            ++turn;
        };
        any_of<NT - 1>([&](auto i) MEP_INLINE {
            load(g0, i);
            return false;
        });
        for (int g = g0; g + 1 < g1; ++g) {
            any_of<NT>([&](auto i) MEP_INLINE {
                load(i == 0 ? g : g + 1, std::integral_constant<int, (i + NT - 1) % NT>{});
                use(i);
                return false;
            });
            join(g);
        }
        load(g1 - 1, std::integral_constant<int, NT - 1>{});
        any_of<NT>([&](auto i) MEP_INLINE {
            use(i);
            return false;
        });
        join(g1 - 1);
    }
}

// Products for more routes an expert: one work-group has RT tiles (LAYER: of
// the gate rows, and the same of the up rows) of one slot, NW waves
// splitting the inputs, and reads the inputs along with the weights, for up
// to 16 routes at a time; the passes of a crowded expert are shared among
// gridDim.z work-groups. Measured: the up and gate halves of a rank's 32 bf16
// experts (H 7168, I 2048; skewed ids reach most of them), 128 tokens, 233 us,
// the rate of a plain read; one int4 matrix of 4096x7168 and one token 7-8 us,
// of which 2 are its bytes and the rest the launch and three round trips.
template <class W, bool LAYER, int RT, int NB, int NW>
__device__ __forceinline__ void rows_pass(const RowsArgs& a, const Finder& find, f32x4* s_part,
                                          int e, int cnt, int c0, int row0, Buffer xb,
                                          bool again) {
    constexpr int NT = LAYER ? 2 * RT : RT;
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x) / kWave;
    const int KC = chunks<W>(a.w.K);
    const int i16 = lane & 15, q = lane >> 4;
    typename W::Ptr wp[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) wp[i] = W::at(a.w, e, (i / RT) * a.I + row0 + (i % RT) * kTile);
    f32x4 acc[NT][NB];
    Input<1> xp[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int j = min(c0 + b * kCols + (lane & 7), cnt - 1);
        xp[b].row((a.ids ? find.list[j] : j) / a.div, a.w.KV, lane);
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i][b] = f32x4{0, 0, 0, 0};
    }
    stream<W, 2, 1, NT, NB>(a.w, wp, xb, xp, KC * wave / NW, KC * (wave + 1) / NW, lane, acc);
    if (again) lds_barrier();  // the last pass's sums have been read
    // [wave][tile][block][32]
    if ((i16 < 8) == (q < 2)) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                s_part[((wave * NT + i) * NB + b) * 32 + (q >> 1) * 16 + (q & 1) * 8 + (i16 & 7)] =
                    acc[i][b];
    }
    lds_barrier();
    // 16 threads per (tile, block): 8 routes x 2 row quads
    for (int u = threadIdx.x; u < RT * NB * 16; u += NW * kWave) {
        const int i = u / (NB * 16), b = (u / 16) % NB, s = u & 15;
        const int j = c0 + b * kCols + (s & 7);
        if (j >= cnt) continue;
        f32x4 v = {0, 0, 0, 0}, up = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < NW; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 o = s_part[((w * NT + i) * NB + b) * 32 + h * 16 + s];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = v[k] + o[k];
                if constexpr (LAYER) {
                    const f32x4 t = s_part[((w * NT + RT + i) * NB + b) * 32 + h * 16 + s];
#pragma unroll
                    for (int k = 0; k < 4; ++k) up[k] = up[k] + t[k];
                }
            }
        store_rows<LAYER>(a, a.ids ? find.list[j] : j, row0 + i * kTile + (s >> 3) * 4, v, up);
    }
}

template <class W, bool LAYER, int RT, int NW>
__global__ __launch_bounds__(NW* kWave, 2) void expert_rows_read(const RowsArgs a) {
    __shared__ Finder s_find;
    __shared__ f32x4 s_part[NW * (LAYER ? 2 : 1) * RT * 2 * 32];
    const int row0 = blockIdx.x * (RT * kTile);
    int e = 0, cnt = a.n;
    if (a.ids) {
        FewRoutes few = {};
        s_find.begin(a, few);
        int slot = blockIdx.y;  // the slot-th expert reached
        if (a.n <= kWave) {
            uint64_t firsts = __ballot(few.first == lane_id());
            if (slot >= __popcll(firsts)) return;
            for (; slot > 0; --slot) firsts &= firsts - 1;
            e = __builtin_amdgcn_readlane(few.id, (int)__builtin_ctzll(firsts));
        } else {
            if constexpr (LAYER) s_find.write_slots(a.table);
            if (slot >= s_find.slots) return;
            for (int e0 = 0;; e0 += kWave) {
                const uint64_t m = __ballot(s_find.routes[e0 + lane_id()] > 0);
                const int here = __popcll(m);
                if (slot < here) {
                    const bool hit = ((m >> lane_id()) & 1) && count_below(m) == slot;
                    e = e0 + (int)__builtin_ctzll(__ballot(hit));
                    break;
                }
                slot -= here;
            }
        }
        int off;
        cnt = s_find.find(a, few, e, &off);
        if constexpr (LAYER) {
            if (blockIdx.x == 0 && blockIdx.z == 0) s_find.write_routes(a, off, cnt);
        }
    }
    const Buffer xb = buffer_of(a.x, (uint32_t)(a.n / a.div) * a.w.KV * 16u);
    const int c1 = blockIdx.z * 2 * kCols, step = gridDim.z * 2 * kCols;
    for (int c0 = c1; c0 < cnt; c0 += step) {
        if (cnt - c0 > kCols)
            rows_pass<W, LAYER, RT, 2, NW>(a, s_find, s_part, e, cnt, c0, row0, xb, c0 > c1);
        else
            rows_pass<W, LAYER, RT, 1, NW>(a, s_find, s_part, e, cnt, c0, row0, xb, c0 > c1);
    }
}

// ------------------------------------------------ second half of the layer

struct DownArgs {
    const u32x4* h;
    const Table* table;   // read where n > 64, otherwise:
    const int* ids;       // [T*K]
    const uint8_t* mask;  // [T*K] or NULL
    int first;
    const float* scores;  // [T*K]
    int T, K, n, E;
    Weights w;            // [E, H, I]
    uint16_t* out_bf16;   // [T, H], either may be NULL
    float* out_f32;
};

// A job: up to two column blocks of one expert's routes, from place `off` in
// the list on. Packed, as the second kernel keeps up to 2048 of them in LDS.
struct Job {
    uint32_t expert : 12, cnt : 8, off : 12;
};
static_assert(kMaxExperts < (1 << 12) && kMaxRoutes <= (1 << 12), "fields of Job");

// One work-group: RT 8-row tiles of the output for all tokens, its waves
// splitting the (job, chunk) steps of all experts reached in equal, unbroken
// ranges; a step's loads are issued one step ahead, across jobs. A wave adds
// score * product into its own [token][row] sums in LDS after each job it
// visits; the waves' sums are joined in wave order at the end. Every sum has
// a fixed order, so equal inputs give equal bits. Measured on 7168x2048: a
// rank's 32 bf16 experts, 128 tokens, 144 us; one token's 8 bf16 experts
// 40-45 us (5.2-5.9 TB/s); 64 int4 experts, 32 tokens, 138-141 us (3.4 TB/s:
// two waves a SIMD, whose tiles, scales and inputs fill the registers, do not
// cover the loads).
template <class W, int TERMS, int RT, int NW>
__global__ __launch_bounds__(NW* kWave, 2) void expert_down(const DownArgs a) {
    extern __shared__ f32x4 s_dyn[];
    __shared__ int s_jobs;
    constexpr int R4 = RT * 2;  // row quads
    constexpr int kRoutes = Input<TERMS>::kRoutes;
    const int tid = threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid) / kWave;
    f32x4* s_sum = s_dyn;                              // [NW][T][R4]
    Job* s_job = (Job*)(s_dyn + NW * a.T * R4);        // [n]
    float* s_score = (float*)(s_job + a.n);            // [n] by place in the list
    uint16_t* s_route = (uint16_t*)(s_score + a.n);    // [n]
    uint8_t* s_token = (uint8_t*)(s_route + a.n);      // [n]
    const int row0 = blockIdx.x * (RT * kTile);

    for (int i = tid; i < NW * a.T * R4; i += NW * kWave) s_sum[i] = f32x4{0, 0, 0, 0};
    if (a.n <= kWave) {
        // each wave writes the same tables
        const FewRoutes few = FewRoutes::read(a.ids, a.mask, a.n, a.first, a.E);
        const float score = a.scores[min(lane, a.n - 1)];
        const int at = few.place();
        if (few.id >= 0) {
            s_route[at] = (uint16_t)lane;
            s_score[at] = score;
            s_token[at] = (uint8_t)(lane / a.K);
        }
        const int mine = few.jobs(2 * kRoutes), to = wave_inclusive_sum(mine);
        for (int j = 0; j < mine; ++j)
            s_job[to - mine + j] = {
                (uint32_t)few.id,
                (uint32_t)min(2 * kRoutes, __popcll(few.peers) - j * 2 * kRoutes),
                (uint32_t)(at + j * 2 * kRoutes)};
        if (lane == kWave - 1) s_jobs = to;
    } else {
        // Loads that do not wait for each other: entries past the last slot
        // or route are read (they lie in the table) and not used.
        const int n_slots = a.table->n_slots, slots_max = min(a.n, a.E);
        for (int i = tid; i < a.n; i += NW * kWave) {
            const int r = min((int)a.table->route[i], a.n - 1);
            s_route[i] = (uint16_t)r;
            s_score[i] = a.scores[r];
            s_token[i] = (uint8_t)(r / a.K);
        }
        if (wave == 0) {
            int jobs = 0;
            for (int s0 = 0; s0 < slots_max; s0 += kWave) {
                const int s = min(s0 + lane, slots_max - 1);
                const int e = a.table->expert[s], off = a.table->offset[s];
                const int to_off = a.table->offset[s + 1];
                const int cnt = s0 + lane < n_slots ? to_off - off : 0;
                const int mine = (cnt + 2 * kRoutes - 1) / (2 * kRoutes);
                const int to = jobs + wave_inclusive_sum(mine);
                for (int j = 0; j < mine; ++j)
                    s_job[to - mine + j] = {
                        (uint32_t)e, (uint32_t)min(2 * kRoutes, cnt - j * 2 * kRoutes),
                        (uint32_t)(off + j * 2 * kRoutes)};
                jobs = __builtin_amdgcn_readlane(to, kWave - 1);
            }
            if (lane == 0) s_jobs = jobs;
        }
    }
    lds_barrier();

    const int KC = chunks<W>(a.w.K);
    const long long steps = (long long)__builtin_amdgcn_readfirstlane(s_jobs) * KC;
    const int lo = (int)(steps * wave / NW), hi = (int)(steps * (wave + 1) / NW);
    f32x4* sum = s_sum + (size_t)wave * a.T * R4;
    const int hv = padded(a.w.K) / 8;  // vectors of a row of h
    const Buffer hb = buffer_of(a.h, (uint32_t)a.n * hv * (TERMS * 16u));
    const typename W::Lane l = W::lane_of(a.w, lane);

    if (lo < hi) {
        // Weights are loaded a chunk ahead. The inputs, which come from the
        // caches, half a chunk ahead where a chunk is four steps: a whole one
        // of two blocks, twice, would take half the registers. For bf16's two
        // steps that is too late (186 us against 140 on a rank's 32 experts
        // and 128 tokens), and the registers are there for a whole chunk.
        constexpr bool kHalves = W::kSteps == 4;
        constexpr int HS = kHalves ? W::kSteps / 2 : W::kSteps;
        constexpr int HN = kHalves ? 2 : 1;
        typename W::Reg r[2][RT];
        u32x4 x[2][2][HS];  // [half, or chunk][block]
        f32x4 acc[RT][2];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = f32x4{0, 0, 0, 0};
        struct At {
            int job, chunk, two;
        };
        typename W::Ptr wp[RT];
        Input<TERMS> xp[2];
        auto open = [&](At& p) MEP_INLINE {  // points the loads at a job
            const Job j = s_job[p.job];
            const int e = __builtin_amdgcn_readfirstlane(j.expert);
            const int cnt = __builtin_amdgcn_readfirstlane(j.cnt);
#pragma unroll
            for (int i = 0; i < RT; ++i) wp[i] = W::at(a.w, e, row0 + i * kTile);
#pragma unroll
            for (int b = 0; b < 2; ++b)
                xp[b].row(s_route[(int)j.off + min(b * kRoutes + (lane & (kRoutes - 1)), cnt - 1)],
                          hv, lane);
            p.two = cnt > kRoutes;
        };
        auto load_w = [&](auto d, const At& p) MEP_INLINE {
#pragma unroll
            for (int i = 0; i < RT; ++i) W::load(r[d][i], wp[i], l, p.chunk);
        };
        auto load_x = [&](auto to, auto h, const At& p) MEP_INLINE {
            xp[0].template load<true>(x[to][0], hb, p.chunk * HN + h);
            if (p.two) xp[1].template load<true>(x[to][1], hb, p.chunk * HN + h);
        };
        auto fold = [&](int job) MEP_INLINE {  // adds a job's sums to its tokens'
            const Job j = s_job[job];
            const int cnt = __builtin_amdgcn_readfirstlane(j.cnt);
            any_of<2>([&](auto b) MEP_INLINE {
                const int c = b * kRoutes + (lane & (kRoutes - 1));
                bool todo = lane < 32 && (lane & 15) < kRoutes && c < cnt;
                const int tok = s_token[(int)j.off + min(c, cnt - 1)];
                const float sc = s_score[(int)j.off + min(c, cnt - 1)];
                f32x4 v[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i][k] = Input<TERMS>::total(acc[i][b][k], lane);
                // a token that names an expert twice has adjacent columns:
                // they are added one after the other
                while (__ballot(todo)) {
                    const int before = __shfl(todo ? tok : -1, max(lane - 1, 0), kWave);
                    if (todo && ((lane & 15) == 0 || before != tok)) {
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            f32x4* s = sum + tok * R4 + i * 2 + (lane >> 4);
                            f32x4 o = *s;
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[k] = __builtin_fmaf(sc, v[i][k], o[k]);
                            *s = o;
                        }
                        todo = false;
                    }
                }
                return cnt <= kRoutes;
            });
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = f32x4{0, 0, 0, 0};
        };
        // Both blocks are always multiplied (the second's inputs are stale
        // where a job has one, and its sums not used): a branch here costs
        // more than the matrix cores' time.
        auto use = [&](auto d, auto from, auto h) MEP_INLINE {
            W::template mma<h * HS, HS, RT, 2>(r[d], x[from], acc);
        };
        constexpr std::integral_constant<int, 0> k0{};
        constexpr std::integral_constant<int, 1> k1{};
        At cur = {lo / KC, lo % KC, 0};
        open(cur);
        load_w(k0, cur);
        load_x(k0, k0, cur);
        int s = lo;
        while (!any_of<2>([&](auto d) MEP_INLINE {
            if constexpr (kHalves) load_x(k1, k1, cur);
            if (s + 1 >= hi) {
                if constexpr (kHalves) {
                    use(d, k0, k0);
                    use(d, k1, k1);
                } else {
                    use(d, d, k0);
                }
                fold(cur.job);
                return true;
            }
            At nxt = {cur.job, cur.chunk + 1, cur.two};
            if (nxt.chunk == KC) {
                nxt = {cur.job + 1, 0, 0};
                open(nxt);
            }
            constexpr std::integral_constant<int, 1 - d> other{};
            load_w(other, nxt);
            if constexpr (kHalves) {
                use(d, k0, k0);
                load_x(k0, k0, nxt);
                use(d, k1, k1);
            } else {
                load_x(other, k0, nxt);
                use(d, d, k0);
            }
            if (nxt.chunk == 0) fold(cur.job);
            cur = nxt;
            ++s;
            return false;
        })) {
        }
    }
    lds_barrier();
    for (int u = tid; u < a.T * R4; u += NW * kWave) {
        const int t = u / R4, row = row0 + (u % R4) * 4;
        if (row >= a.w.N) continue;  // N is a multiple of 8: quads are whole
        f32x4 v = s_sum[u];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            const f32x4 o = s_sum[(size_t)w * a.T * R4 + u];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = v[k] + o[k];
        }
        const size_t o = (size_t)t * a.w.N + row;
        if (a.out_bf16)
            *(u32x2*)(a.out_bf16 + o) = u32x2{bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3])};
        if (a.out_f32) *(f32x4*)(a.out_f32 + o) = v;
    }
}

// ----------------------------------------------------------------- launch

constexpr int kCus = 256;

inline int tiles_of(int rows, int rt) { return (rows + rt * kTile - 1) / (rt * kTile); }

// Tiles over all experts from which on expert_rows_held is used.
constexpr long long kHeldTiles = 2048;

template <class W, bool LAYER, int NT, int XC>
void launch_held(hipStream_t s, const RowsArgs& a, int kc) {
    const int nw = (kc + XC - 1) / XC;
    const int groups = tiles_of(LAYER ? a.I : a.w.N, LAYER ? NT / 2 : NT);
    const int slots = a.ids ? (a.n < a.E ? a.n : a.E) : 1;
    const long long items = (long long)slots * groups;
    const long long wgs = (long long)kCus * (kMaxWaves / nw);
    hipLaunchKernelGGL((expert_rows_held<W, LAYER, NT, XC>), dim3(items < wgs ? items : wgs),
                       dim3(nw * kWave), (size_t)2 * nw * NT * 32 * 16, s, a, groups);
}

// Which of the two first kernels runs. Held inputs pay where an expert gets
// few routes (they are multiplied 8 at a time, and more routes read the
// weights again) and every CU has several row groups to go through: 28 fp4
// experts of 7168x2048 with 4-5 routes each take 53 us held against 103 read
// along, 64 int4 experts of 4096x7168 186 against 203. One expert's 5 rows of
// 1001x2504 take 13.1 held and 10.2 read, and at 8 routes an expert and more
// (32 experts, 128 tokens, most of them other ranks') reading along in pairs
// of blocks is at 7.1 TB/s. Inputs beyond what 16 waves hold are read too.
// Two tiles in flight where a wave holds two chunks or more (four spill),
// four where it holds one (60 us against 67 on the fp4 products).
template <class W, bool LAYER>
void launch_rows(hipStream_t s, const RowsArgs& a) {
    const int kc = chunks<W>(a.w.K);
    const int slots = a.ids ? (a.n < a.E ? a.n : a.E) : 1;
    const int rows = LAYER ? a.I : a.w.N;
    if (a.n <= kCols * slots && kc <= W::kMaxHeld * kMaxWaves &&
        (long long)slots * tiles_of(rows, 1) >= kHeldTiles) {
        if (kc <= kMaxWaves)
            launch_held<W, LAYER, 4, 1>(s, a, kc);
        else if (kc <= 2 * kMaxWaves)
            launch_held<W, LAYER, 2, 2>(s, a, kc);
        else if constexpr (W::kMaxHeld == 4)
            launch_held<W, LAYER, 2, 4>(s, a, kc);
        return;
    }
    constexpr int RT = 2, NW = 4;
    // Few work-groups: the passes over 16 routes that an expert has on average
    // run beside each other (86 rows of one 600x3144 matrix: 8 us against
    // 21 one after the other). With many, one work-group goes through them
    // and finds the weights in its caches.
    const int tiles = tiles_of(rows, RT), passes = (a.n / slots + 2 * kCols - 1) / (2 * kCols);
    const int room = 4 * kCus / (tiles * slots);
    const int z = passes < room ? passes : room;
    hipLaunchKernelGGL((expert_rows_read<W, LAYER, RT, NW>), dim3(tiles, slots, z < 1 ? 1 : z),
                       dim3(NW * kWave), 0, s, a);
}

inline size_t down_lds(int nw, int rt, int T, int n) {
    return (size_t)nw * T * rt * 2 * 16 + (size_t)n * (4 + 4 + 2 + 1) + 16;
}

template <class W, int TERMS, int RT, int NW>
void launch_down(hipStream_t s, const DownArgs& d) {
    hipLaunchKernelGGL((expert_down<W, TERMS, RT, NW>), dim3(tiles_of(d.w.N, RT)),
                       dim3(NW * kWave), down_lds(NW, RT, d.T, d.n), s, d);
}

// Four tiles a work-group where that still gives three work-groups to four
// CUs: the inputs, read once per work-group, are then a smaller part of what
// moves (64 int4 experts, 32 tokens: 142 us against 176 with two tiles; a
// rank's 32 bf16 experts, 128 tokens: 144 against 159). For groups of 32 and
// 64 four tiles' scales do not fit the registers. Four waves instead of
// eight above 32 tokens: their sums fill the LDS. Outputs of up to 5120 rows
// leave CUs idle unless each work-group has one tile (9 tokens over 64 fp4
// experts, 2048 rows: 18.6 us against 23.6; 89 tokens, 232 rows, both
// kernels: 23 us against 29).
template <class W, int TERMS>
void launch_down(hipStream_t s, const DownArgs& d) {
    if constexpr (W::kWide) {
        if (tiles_of(d.w.N, 4) >= kCus * 3 / 4)
            return d.T <= 32 ? launch_down<W, TERMS, 4, 8>(s, d) : launch_down<W, TERMS, 4, 4>(s, d);
    }
    if (tiles_of(d.w.N, 1) > kCus * 5 / 2) return launch_down<W, TERMS, 2, 4>(s, d);
    launch_down<W, TERMS, 1, 8>(s, d);
}

template <class W>
void launch_matvec(hipStream_t s, const RowsArgs& a) {
    launch_rows<W, false>(s, a);
}

template <class W>
void launch_layer(hipStream_t s, const RowsArgs& a, const DownArgs& d) {
    launch_rows<W, true>(s, a);
    if (a.terms == 2)
        launch_down<W, 2>(s, d);
    else
        launch_down<W, 3>(s, d);
}

// One per weight kind, each in a source of its own. `group`, `zeros` and
// `f16` have been checked by the caller.
struct Kind {
    int group;
    bool zeros, f16;
};
void matvec_int4(hipStream_t s, const Kind& k, const RowsArgs& a);
void matvec_fp4(hipStream_t s, const Kind& k, const RowsArgs& a);
void layer_bf16(hipStream_t s, const RowsArgs& a, const DownArgs& d);
void layer_int4(hipStream_t s, const Kind& k, const RowsArgs& a, const DownArgs& d);
void layer_fp4(hipStream_t s, const Kind& k, const RowsArgs& a, const DownArgs& d);

}  // namespace experts
}  // namespace mep
