// Kernels of the experts' products for a few routes (gfx950, wave64): the
// routed product y = W[id] x and the two halves of the expert layer. The
// weights are read once per expert that any route reaches; everything else
// is small, so the kernels stream weights and are bound by HBM.
//
// Products run on the matrix cores, one 16x16x32 bf16 MFMA per 16 weight
// rows, 32 inputs and up to 16 routes: its operands are 16 bytes of a weight
// row per lane and 16 bytes of a route's input per lane, so any route count
// up to 16 costs the same weight traffic, and columns of different routes
// never mix (a NaN in one route's input stays in its column). Accumulation
// is fp32.
//
// Lane layout of that MFMA (i = lane % 16, q = lane / 16): A holds row i,
// inputs 8q..8q+7; B holds column i, the same inputs; C holds column i, rows
// 4q..4q+3.
#pragma once

#include "rows.h"

namespace mep {
namespace experts {

using rows::f32x4;
using rows::u32x4;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 16;       // weight rows of one MFMA
constexpr int kChunk = 128;     // inputs of one load step: four MFMAs
constexpr int kMaxRoutes = 2048;
constexpr int kMaxExperts = 1024;
constexpr int kMaxLayerTokens = 128;

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
    int tiles;  // packed: ceil(N / 16)
    int KB;     // ceil(K / 128)
    int KS;     // packed: ceil(K / 512), superblocks of scales
};

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------- weights
//
// A weight kind gives: Ptr (where a lane's part of one 16-row tile starts),
// Reg (one chunk of it in registers), load, and mma (chunk times NTB column
// blocks, each the sum of NX input terms).

struct Bf16Weights {
    struct Ptr {
        const u32x4* p;
    };
    struct Reg {
        u32x4 a[4];
    };
    static __device__ __forceinline__ Ptr at(const Weights& w, int e, int row0, int lane) {
        const int row = min(row0 + (lane & 15), w.N - 1);
        return {w.codes + ((size_t)e * w.N + row) * w.KV + (lane >> 4)};
    }
    static __device__ __forceinline__ void load(Reg& r, const Ptr& p, const Weights& w, int c,
                                                int lane) {
        if (c * 16 + 16 <= w.KV) {
#pragma unroll
            for (int j = 0; j < 4; ++j) r.a[j] = __builtin_nontemporal_load(p.p + c * 16 + j * 4);
        } else {  // the last, cut chunk: inputs past K count as zero on both sides
            const int q = lane >> 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int v = c * 16 + j * 4 + q;
                const u32x4 a = p.p[min(v, w.KV - 1) - q];
                r.a[j] = v < w.KV ? a : u32x4{0, 0, 0, 0};
            }
        }
    }
    template <int NT, int NTB, int NX>
    static __device__ __forceinline__ void mma(const Reg (&r)[NT], const u32x4 (&x)[NTB][NX][4],
                                               f32x4 (&acc)[NT][NTB]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int b = 0; b < NTB; ++b)
#pragma unroll
                for (int n = 0; n < NX; ++n)
#pragma unroll
                    for (int i = 0; i < NT; ++i) acc[i][b] = mfma(r[i].a[j], x[b][n][j], acc[i][b]);
    }
};

// 4-bit codes in the packed layout (see pack_codes): 1 KiB per 16 rows and
// 128 inputs, 16 bytes per lane in MFMA order; scales and zero points
// [tile][superblock of 512 inputs][4 row quads][groups][4 rows], the order
// in which the accumulator's lanes need them.
//
// An int4 code q becomes the bf16 number 128 + q by or-ing it into the
// mantissa of 128 (one shift and one and-or per two codes). The constant is
// taken out of the sum again by a product of the same inputs with a constant
// row, -(128 + 8) for symmetric codes, whose result is the accumulator that
// the code product starts from: sum (128 + q) x - sum 136 x = sum (q - 8) x.
// With zero points the constant row is -128 and z of the row times
// sum x = -1/128 of that result is subtracted per row. All terms are exact
// products summed in fp32; the offset makes them at most 27 times larger
// than the terms of the result, which costs under five of fp32's 24 bits.
// A 4-bit float is converted by the hardware, two codes per instruction.
template <bool FP4, int G, bool ZP, bool F16>
struct PackedWeights {
    static constexpr int GP = kChunk / G;  // groups per chunk
    static constexpr int GM = G / 32;      // MFMAs per group
    struct Ptr {
        const u32x4* p;
        const uint32_t* s;
        const uint32_t* z;
    };
    struct Reg {
        u32x4 a;
        uint32_t s[GP * 2];
        uint32_t z[ZP ? GP : 1];
    };
    static __device__ __forceinline__ Ptr at(const Weights& w, int e, int row0, int lane) {
        const int np = w.tiles * kTile;
        const int row = min(row0 + (lane & 15), np - 1);
        const int quad = min((row0 >> 2) + (lane >> 4), np / 4 - 1);
        const size_t tile = (size_t)e * w.tiles + (row >> 4);
        const size_t qt = (size_t)e * w.tiles + (quad >> 2);
        const size_t group0 = (qt * w.KS * 4 + (quad & 3)) * (512 / G);  // in quads of rows
        return {w.codes + tile * w.KB * 64 + (lane >> 4) * 16 + (row & 15),
                (const uint32_t*)w.scales + group0 * 2, (const uint32_t*)w.zeros + group0};
    }
    static __device__ __forceinline__ void load(Reg& r, const Ptr& p, const Weights&, int c,
                                                int) {
        r.a = __builtin_nontemporal_load(p.p + (size_t)c * 64);
        const int g = (c >> 2) * (4 * (512 / G)) + (c & 3) * GP;
#pragma unroll
        for (int i = 0; i < GP * 2; ++i) r.s[i] = p.s[(size_t)g * 2 + i];
        if constexpr (ZP) {
#pragma unroll
            for (int i = 0; i < GP; ++i) r.z[i] = p.z[(size_t)g + i];
        }
    }
    static __device__ __forceinline__ float scale(uint32_t w, int hi) {
        if constexpr (F16) {
            const uint16_t b = (uint16_t)(hi ? w >> 16 : w);
            return (float)__builtin_bit_cast(_Float16, b);
        }
        return __uint_as_float(hi ? w & 0xffff0000u : w << 16);
    }
    static __device__ __forceinline__ u32x4 decode(uint32_t d) {
        u32x4 o;
        if constexpr (FP4) {
            o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 0));
            o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 1));
            o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 2));
            o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 3));
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) o[p] = ((d >> (4 * p)) & 0x000f000fu) | 0x43004300u;
        }
        return o;
    }
    template <int NT, int NTB, int NX>
    static __device__ __forceinline__ void mma(const Reg (&r)[NT], const u32x4 (&x)[NTB][NX][4],
                                               f32x4 (&acc)[NT][NTB]) {
        constexpr uint32_t kOff = ZP ? 0xc300c300u : 0xc308c308u;  // -128, -136
        const u32x4 off = {kOff, kOff, kOff, kOff};
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            f32x4 x0[NTB];
#pragma unroll
            for (int b = 0; b < NTB; ++b) {
                x0[b] = f32x4{0, 0, 0, 0};
                if constexpr (!FP4) {
#pragma unroll
                    for (int j = 0; j < GM; ++j)
#pragma unroll
                        for (int n = 0; n < NX; ++n) x0[b] = mfma(off, x[b][n][g * GM + j], x0[b]);
                }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                f32x4 c[NTB];
#pragma unroll
                for (int b = 0; b < NTB; ++b) c[b] = x0[b];
#pragma unroll
                for (int j = 0; j < GM; ++j) {
                    const u32x4 a = decode(r[i].a[g * GM + j]);
#pragma unroll
                    for (int b = 0; b < NTB; ++b)
#pragma unroll
                        for (int n = 0; n < NX; ++n) c[b] = mfma(a, x[b][n][g * GM + j], c[b]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float s = scale(r[i].s[g * 2 + k / 2], k & 1);
#pragma unroll
                    for (int b = 0; b < NTB; ++b) {
                        float v = c[b][k];
                        if constexpr (ZP) {
                            const float z = (float)((r[i].z[g] >> (8 * k)) & 0xffu) * (1.0f / 128);
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

// bf16 rows of K inputs, read as they are. A lane of a column past the last
// route reads a real route's row; its column is not stored.
struct PlainInput {
    static constexpr int NX = 1;
    const u32x4* p;
    __device__ __forceinline__ void load(u32x4 (&x)[1][4], int c, int KV, int q) const {
        if (c * 16 + 16 <= KV) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[0][j] = p[c * 16 + j * 4 + q];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int v = c * 16 + j * 4 + q;
                const u32x4 a = p[min(v, KV - 1)];
                x[0][j] = v < KV ? a : u32x4{0, 0, 0, 0};
            }
        }
    }
};

// fp32 values held as a sum of bf16 terms, each the rest of the ones before
// rounded (two terms lose at most 2^-17 of the value, three at most 2^-25),
// in rows padded with zeros to whole chunks; per 8 values 16 bytes of each
// term. Two terms serve a bf16 output (its own rounding is 2^-8), three an
// fp32 one: with two, an fp32 output measured 2.7e-6 from the exact result
// where 2.5e-7 is fp32's share.
template <int TERMS>
struct SplitInput {
    static constexpr int NX = TERMS;
    const u32x4* p;
    __device__ __forceinline__ void load(u32x4 (&x)[TERMS][4], int c, int, int q) const {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < TERMS; ++n) x[n][j] = p[(c * 16 + j * 4 + q) * TERMS + n];
    }
};

// acc[i][b] += tile i of the weights times column block b over chunks
// [lo, hi), with the next chunk's loads issued before a chunk is used.
template <class W, class X, int NT, int NTB>
__device__ __forceinline__ void stream(const Weights& w, const typename W::Ptr (&wp)[NT],
                                       const X (&xp)[NTB], int lo, int hi, int lane,
                                       f32x4 (&acc)[NT][NTB]) {
    typename W::Reg r0[NT], r1[NT];
    u32x4 x0[NTB][X::NX][4], x1[NTB][X::NX][4];
    const int q = lane >> 4;
    auto load = [&](typename W::Reg (&r)[NT], u32x4 (&x)[NTB][X::NX][4], int c) {
#pragma unroll
        for (int i = 0; i < NT; ++i) W::load(r[i], wp[i], w, c, lane);
#pragma unroll
        for (int b = 0; b < NTB; ++b) xp[b].load(x[b], c, w.KV, q);
    };
    if (lo >= hi) return;
    load(r0, x0, lo);
    for (int c = lo;;) {
        if (c + 1 < hi) load(r1, x1, c + 1);
        W::template mma<NT, NTB, X::NX>(r0, x0, acc);
        if (++c >= hi) break;
        if (c + 1 < hi) load(r0, x0, c + 1);
        W::template mma<NT, NTB, X::NX>(r1, x1, acc);
        if (++c >= hi) break;
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
    u32x4* h;            // [n][Ip / 8][terms]
    int I, Ip, terms;
    Table* table;
};

// Finds the blockIdx.y-th expert that any route reaches and its routes, in
// route order. Returns false (for the whole work-group) past the last one.
template <int NW>
struct Finder {
    uint32_t bits[kMaxExperts / 32];
    int count[NW], less[NW];
    int16_t id[kMaxRoutes];
    uint16_t list[kMaxRoutes];

    __device__ __forceinline__ bool find(const RowsArgs& a, int slot, int* e_out, int* cnt_out,
                                         int* off_out, int* total_out) {
        const int tid = threadIdx.x, lane = lane_id();
        const int wave = __builtin_amdgcn_readfirstlane(tid) / kWave;
        if (tid < kMaxExperts / 32) bits[tid] = 0u;
        lds_barrier();
        for (int i = tid; i < a.n; i += NW * kWave) {
            int v = a.ids[i] - a.first;
            if ((unsigned)v >= (unsigned)a.E || (a.mask && a.mask[i] == 0)) v = -1;
            id[i] = (int16_t)v;
            if (v >= 0) atomicOr(&bits[v >> 5], 1u << (v & 31));
        }
        lds_barrier();
        const uint32_t word = lane < kMaxExperts / 32 ? bits[lane] : 0u;
        const int pop = __popc(word);
        const int inc = wave_inclusive_sum(pop);
        const int total = __builtin_amdgcn_readlane(inc, kWave - 1);
        *total_out = total;
        if (slot >= total) return false;
        const uint64_t hit = __ballot(slot >= inc - pop && slot < inc);
        const int at = (int)__builtin_ctzll(hit);
        int rem = slot - (__builtin_amdgcn_readlane(inc, at) - __builtin_amdgcn_readlane(pop, at));
        uint32_t bw = (uint32_t)__builtin_amdgcn_readlane((int)word, at);
        for (; rem > 0; --rem) bw &= bw - 1;
        const int e = at * 32 + __builtin_ctz(bw);

        // each wave takes a range of whole 64-route rounds
        const int rounds = (a.n + kWave - 1) / kWave;
        const int r0 = rounds * wave / NW, r1 = rounds * (wave + 1) / NW;
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
        int base = 0, cnt = 0, off = 0;
        for (int w = 0; w < NW; ++w) {
            if (w < wave) base += count[w];
            cnt += count[w];
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
        *e_out = e;
        *cnt_out = cnt;
        *off_out = off;
        return true;
    }
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// One work-group: RT 16-row tiles (LAYER: of the gate rows, and the same of
// the up rows) of one expert, NW waves splitting the inputs, joined in wave
// order through LDS.
template <class W, bool LAYER, int RT, int NTB, int NW>
__global__ __launch_bounds__(NW* kWave) void expert_rows(const RowsArgs a) {
    constexpr int NT = LAYER ? 2 * RT : RT;
    __shared__ Finder<NW> s_find;
    __shared__ f32x4 s_part[NW][NT][NTB][kWave];
    const int tid = threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid) / kWave;
    const int row0 = blockIdx.x * (RT * kTile);

    int e = 0, cnt = a.n;
    if (a.ids) {
        int off = 0, total = 0;
        const bool any = s_find.find(a, blockIdx.y, &e, &cnt, &off, &total);
        if constexpr (LAYER) {
            if (blockIdx.x == 0) {
                Table* t = a.table;
                if (blockIdx.y == 0 && tid == 0) t->n_slots = total;
                if (any) {
                    if (tid == 0) {
                        t->expert[blockIdx.y] = e;
                        t->offset[blockIdx.y] = off;
                        if ((int)blockIdx.y == total - 1) t->offset[total] = off + cnt;
                    }
                    for (int i = tid; i < cnt; i += NW * kWave) t->route[off + i] = s_find.list[i];
                }
            }
        }
        if (!any) return;
    }

    const int KC = (a.w.K + kChunk - 1) / kChunk;
    const int lo = KC * wave / NW, hi = KC * (wave + 1) / NW;
    const bool live_tile = !LAYER || row0 < a.I;
    typename W::Ptr wp[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int r = LAYER ? (i / RT) * a.I + row0 + (i % RT) * kTile : row0 + i * kTile;
        wp[i] = W::at(a.w, e, r, lane);
    }

    for (int c0 = 0; c0 < cnt; c0 += NTB * 16) {
        f32x4 acc[NT][NTB];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int b = 0; b < NTB; ++b) acc[i][b] = f32x4{0, 0, 0, 0};
        if (live_tile) {
            PlainInput xp[NTB];
#pragma unroll
            for (int b = 0; b < NTB; ++b) {
                const int j = min(c0 + b * 16 + (lane & 15), cnt - 1);
                const int r = a.ids ? s_find.list[j] : j;
                xp[b].p = a.x + (size_t)(r / a.div) * a.w.KV;
            }
            stream<W, PlainInput, NT, NTB>(a.w, wp, xp, lo, hi, lane, acc);
        }
        if (c0) lds_barrier();  // the last block's sums have been read
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int b = 0; b < NTB; ++b) s_part[wave][i][b][lane] = acc[i][b];
        lds_barrier();
        for (int u = wave; u < RT * NTB; u += NW) {
            const int i = u / NTB, b = u % NTB;
            const int j = c0 + b * 16 + (lane & 15);
            if (j >= cnt) continue;
            const int r = a.ids ? s_find.list[j] : j;
            const int row = row0 + i * kTile + (lane >> 4) * 4;
            f32x4 v = s_part[0][i][b][lane];
#pragma unroll
            for (int w = 1; w < NW; ++w) {
                const f32x4 o = s_part[w][i][b][lane];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = v[k] + o[k];
            }
            if constexpr (LAYER) {
                f32x4 up = s_part[0][RT + i][b][lane];
#pragma unroll
                for (int w = 1; w < NW; ++w) {
                    const f32x4 o = s_part[w][RT + i][b][lane];
#pragma unroll
                    for (int k = 0; k < 4; ++k) up[k] = up[k] + o[k];
                }
                float h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) h[k] = row + k < a.I ? silu(v[k]) * up[k] : 0.0f;
                u32x2* dst = (u32x2*)(a.h + ((size_t)r * (a.Ip / 8) + row / 8) * a.terms) +
                             (row % 8) / 4;
                for (int n = 0; n < a.terms; ++n) {
                    const u32x2 o = {bf16x2_bits(h[0], h[1]), bf16x2_bits(h[2], h[3])};
                    dst[2 * n] = o;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float b =
                            __uint_as_float(k & 1 ? o[k / 2] & 0xffff0000u : o[k / 2] << 16);
                        // an infinite or NaN term has no rest
                        h[k] = fabsf(b) < INFINITY ? h[k] - b : 0.0f;
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
    }
}

// ------------------------------------------------ second half of the layer

struct DownArgs {
    const u32x4* h;
    int Ip;
    const Table* table;
    const float* scores;  // [T*K]
    int T, K, n, E;
    Weights w;            // [E, H, I]
    uint16_t* out_bf16;   // [T, H], either may be NULL
    float* out_f32;
};

// One work-group: RT 16-row tiles of the output for all tokens, its waves
// splitting the (expert, chunk) steps of all experts reached. A wave adds
// score * product into its own [token][row] sums in LDS after each expert it
// visits; the waves' sums are joined in wave order at the end. Every sum has
// a fixed order, so equal inputs give equal bits.
template <class W, int TERMS, int RT, int NTB, int NW>
__global__ __launch_bounds__(NW* kWave) void expert_down(const DownArgs a) {
    extern __shared__ f32x4 s_dyn[];
    constexpr int R4 = RT * 4;  // row quads
    const int tid = threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid) / kWave;
    const int slots_max = min(a.n, a.E);
    f32x4* s_sum = s_dyn;                                   // [NW][T][R4]
    float* s_score = (float*)(s_dyn + NW * a.T * R4);       // [n]
    int* s_expert = (int*)(s_score + a.n);                  // [slots_max]
    int* s_off = s_expert + slots_max;                      // [slots_max + 1]
    uint16_t* s_route = (uint16_t*)(s_off + slots_max + 1); // [n]
    const int row0 = blockIdx.x * (RT * kTile);

    for (int i = tid; i < NW * a.T * R4; i += NW * kWave) s_sum[i] = f32x4{0, 0, 0, 0};
    for (int i = tid; i < a.n; i += NW * kWave) {
        s_score[i] = a.scores[i];
        s_route[i] = a.table->route[i];
    }
    for (int i = tid; i < slots_max; i += NW * kWave) s_expert[i] = a.table->expert[i];
    for (int i = tid; i < slots_max + 1; i += NW * kWave) s_off[i] = a.table->offset[i];
    const int n_slots = a.table->n_slots;
    lds_barrier();

    const int KC = (a.w.K + kChunk - 1) / kChunk;
    const int steps = n_slots * KC;
    const int lo = (int)((long long)steps * wave / NW), hi = (int)((long long)steps * (wave + 1) / NW);
    f32x4* sum = s_sum + (size_t)wave * a.T * R4;
    for (int at = lo; at < hi;) {
        const int slot = at / KC;
        const int k0 = at - slot * KC, k1 = min(KC, k0 + hi - at);
        at += k1 - k0;
        const int e = __builtin_amdgcn_readfirstlane(s_expert[slot]);
        const int off = __builtin_amdgcn_readfirstlane(s_off[slot]);
        const int cnt = __builtin_amdgcn_readfirstlane(s_off[slot + 1]) - off;
        typename W::Ptr wp[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) wp[i] = W::at(a.w, e, row0 + i * kTile, lane);
        for (int c0 = 0; c0 < cnt; c0 += NTB * 16) {
            f32x4 acc[RT][NTB];
            SplitInput<TERMS> xp[NTB];
            int tok[NTB];
            float sc[NTB];
#pragma unroll
            for (int b = 0; b < NTB; ++b) {
                const int j = c0 + b * 16 + (lane & 15);
                const int r = s_route[off + min(j, cnt - 1)];
                xp[b].p = a.h + (size_t)r * (a.Ip / 8) * TERMS;
                tok[b] = j < cnt ? r / a.K : -1;
                sc[b] = s_score[r];
#pragma unroll
                for (int i = 0; i < RT; ++i) acc[i][b] = f32x4{0, 0, 0, 0};
            }
            stream<W, SplitInput<TERMS>, RT, NTB>(a.w, wp, xp, k0, k1, lane, acc);
#pragma unroll
            for (int b = 0; b < NTB; ++b) {
                // a token that names an expert twice has adjacent columns:
                // they are added one after the other
                bool todo = tok[b] >= 0;
                while (__ballot(todo)) {
                    const int before = __shfl(todo ? tok[b] : -1, max(lane - 1, 0), kWave);
                    const bool now = todo && ((lane & 15) == 0 || before != tok[b]);
                    if (now) {
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            f32x4* s = sum + tok[b] * R4 + i * 4 + (lane >> 4);
                            f32x4 v = *s;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                v[k] = __builtin_fmaf(sc[b], acc[i][b][k], v[k]);
                            *s = v;
                        }
                        todo = false;
                    }
                }
            }
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

inline size_t down_lds(int nw, int rt, int T, int n, int E) {
    const int slots = n < E ? n : E;
    return (size_t)nw * T * rt * 4 * 16 + (size_t)n * 6 + (size_t)(2 * slots + 1) * 4 + 8;
}

template <class W>
void launch_matvec(hipStream_t s, const RowsArgs& a) {
    constexpr int NW = 8, RT = 1;
    const int slots = a.ids ? (a.n < a.E ? a.n : a.E) : 1;
    const dim3 g((a.w.N + RT * kTile - 1) / (RT * kTile), slots), b(NW * kWave);
    hipLaunchKernelGGL((expert_rows<W, false, RT, 1, NW>), g, b, 0, s, a);
}

template <class W, int TERMS>
void launch_down(hipStream_t s, const DownArgs& d) {
    constexpr int RT = 1;
    const dim3 g((d.w.N + RT * kTile - 1) / (RT * kTile));
    if (d.T <= 64)
        hipLaunchKernelGGL((expert_down<W, TERMS, RT, 1, 8>), g, dim3(8 * kWave),
                           down_lds(8, RT, d.T, d.n, d.E), s, d);
    else
        hipLaunchKernelGGL((expert_down<W, TERMS, RT, 1, 4>), g, dim3(4 * kWave),
                           down_lds(4, RT, d.T, d.n, d.E), s, d);
}

template <class W>
void launch_layer(hipStream_t s, const RowsArgs& a, const DownArgs& d) {
    constexpr int RT = 1;
    const int slots = a.n < a.E ? a.n : a.E;
    const dim3 g(a.Ip / (RT * kTile), slots), b(8 * kWave);
    hipLaunchKernelGGL((expert_rows<W, true, RT, 1, 8>), g, b, 0, s, a);
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
