// 4-bit weights: codes and group scales from bf16 matrices, and their
// layout for the experts' products (experts.h).
//
// Both run once, when weights are loaded; they are plain one-pass kernels,
// bound by HBM: the codes of 64 matrices 4096x7168 take 589 us, 4.8 TB/s of
// reads and writes, which is a device copy's rate.
#include "experts.h"

namespace mep {
namespace {

using namespace experts;

constexpr int kPackThreads = 256;
// Work-groups of a launch at most (a launch holds fewer than 2^32 threads,
// and a model's experts have more groups of weights than that); each goes on
// from its first piece in steps of the whole launch.
constexpr unsigned kPackBlocks = 1u << 20;

// One thread: the 32 codes that one lane of the product kernels loads at
// once for one 8-row tile and 256 inputs: row lane % 8, and for each of the
// block's four 64-input steps j the 8 inputs of vector lane_vec as one word.
// In a word, int4 code m lies at bit 4 (m / 2) + 3 of half m % 2 (the last
// two run over into the next half, rotated), so that a shift or rotation and
// a mask leave two neighbours at bits 3-6 of the halves, the upper mantissa
// bits of a bf16; 4-bit floats lie in order, as the conversion instruction
// takes them. Rows past N and inputs
// past K get code 0.
__global__ __launch_bounds__(kPackThreads) void pack_codes(const uint8_t* __restrict__ codes,
                                                           u32x4* __restrict__ out, int N, int K,
                                                           int tiles, int KB, int fp4,
                                                           size_t total) {
    for (size_t at = (size_t)blockIdx.x * kPackThreads + threadIdx.x; at < total;
         at += (size_t)gridDim.x * kPackThreads) {
        const int lane = (int)(at & 63);
        const size_t blk = at >> 6;
        const int kb = (int)(blk % KB);
        const size_t et = blk / KB;
        const int row = (int)(et % tiles) * kTile + (lane & 7);
        const size_t e = et / tiles;
        u32x4 o = {0, 0, 0, 0};
        if (row < N) {
            const uint8_t* src = codes + (e * N + row) * (size_t)K;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = kb * kPackK + j * kStep + lane_vec(lane) * 8;
                if (k >= K) continue;  // K is a multiple of 8
                const u32x2 b = *(const u32x2*)(src + k);  // eight codes, one a byte
                uint32_t w = 0;
#pragma unroll
                for (int m = 0; m < 8; ++m)
                    w |= ((b[m >> 2] >> (8 * (m & 3))) & 15u)
                         << (fp4 ? 4 * m : 4 * (m >> 1) + 16 * (m & 1));
                o[j] = fp4 ? w : w << 3 | w >> 29;
            }
        }
        out[at] = o;
    }
}

// [E,N,G] -> [E][tile][block][2 row quads][groups of the block][4 rows];
// groups of 32 with even indices come first. Places past N or the last group
// hold zero.
template <typename T>
__global__ __launch_bounds__(kPackThreads) void pack_groups(const T* __restrict__ src,
                                                            T* __restrict__ out, int N, int G,
                                                            int tiles, int KB, int per,
                                                            size_t total) {
    for (size_t at = (size_t)blockIdx.x * kPackThreads + threadIdx.x; at < total;
         at += (size_t)gridDim.x * kPackThreads) {
        size_t r = at;
        const int i = (int)(r & 3);
        r >>= 2;
        int gi = (int)(r % per);
        r /= per;
        const int quad = (int)(r & 1);
        r >>= 1;
        const int kb = (int)(r % KB);
        r /= KB;
        const int row = (int)(r % tiles) * kTile + quad * 4 + i;
        const size_t e = r / tiles;
        if (per == kPackK / 32) gi = (gi & 3) * 2 + (gi >> 2);
        const int g = kb * per + gi;
        out[at] = row < N && g < G ? src[(e * N + row) * (size_t)G + g] : (T)0;
    }
}

// Symmetric quantization of one group per wave: s = amax / 7 (int4) or
// amax / 6 (4-bit float) rounded to the scale's type, at most its largest
// finite value; codes the nearest of fl(w / s), ties to even.
__global__ __launch_bounds__(kPackThreads) void quant_groups(const uint16_t* __restrict__ w,
                                                             uint8_t* __restrict__ codes,
                                                             uint16_t* __restrict__ scales, int K,
                                                             int group, int G, int fp4, int f16,
                                                             size_t total) {
    const int lane = lane_id();
    constexpr int kPer = kPackThreads / kWave;
    for (size_t at = (size_t)blockIdx.x * kPer + threadIdx.x / kWave; at < total;
         at += (size_t)gridDim.x * kPer) {
        const size_t row = at / G;
        const int k0 = (int)(at % G) * group;
        float v[2], amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int o = lane + i * kWave;
            const bool in = o < group && k0 + o < K;
            v[i] = in ? __uint_as_float((uint32_t)w[row * K + k0 + o] << 16) : 0.0f;
            amax = fmaxf(amax, fabsf(v[i]));
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m, kWave));
        const float s32 = amax / (fp4 ? 6.0f : 7.0f);
        float s;
        uint16_t bits;
        if (f16) {
            const _Float16 h = (_Float16)fminf(s32, 65504.0f);  // codes then stop at their ends
            bits = __builtin_bit_cast(uint16_t, h);
            s = (float)h;
        } else {
            bits = (uint16_t)bf16x2_bits(s32, 0.0f);
            s = __uint_as_float((uint32_t)bits << 16);
        }
        if (lane == 0) scales[at] = bits;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int o = lane + i * kWave;
            if (o >= group || k0 + o >= K) continue;
            const float x = s > 0.0f ? v[i] / s : 0.0f;
            uint32_t q;
            if (fp4) {
                const float a = fabsf(x);
                q = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) +
                    (a >= 3.5f) + (a > 5.0f);
                if (q && x < 0.0f) q |= 8u;
            } else {
                q = (uint32_t)((int)fminf(fmaxf(__builtin_rintf(x), -8.0f), 7.0f) + 8);
            }
            codes[row * K + k0 + o] = (uint8_t)q;
        }
    }
}

bool sizes_ok(int E, int N, int K) {
    return E >= 1 && E <= kMaxExperts && N >= 1 && N <= (1 << 20) && K >= 8 && K <= 65536 &&
           K % 8 == 0;
}

bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }

size_t row_tiles(int N) { return ((size_t)N + kTile - 1) / kTile; }

size_t blocks_of(int K) { return ((size_t)K + kPackK - 1) / kPackK; }

dim3 blocks(size_t n, int per) {
    const size_t b = (n + per - 1) / per;
    return dim3(b < kPackBlocks ? (unsigned)b : kPackBlocks);
}

}  // namespace
}  // namespace mep

using namespace mep;
using namespace mep::experts;

extern "C" size_t mep_packed_code_bytes(int E, int N, int K) {
    if (!sizes_ok(E, N, K)) return 0;
    return (size_t)E * row_tiles(N) * blocks_of(K) * 1024;
}

extern "C" size_t mep_packed_scale_count(int E, int N, int K, int group) {
    if (!sizes_ok(E, N, K) || !group_ok(group)) return 0;
    return (size_t)E * row_tiles(N) * blocks_of(K) * 8 * (kPackK / group);
}

extern "C" int mep_pack_weights(int E, int N, int K, int kind, int group, const uint8_t* codes,
                                const void* scales, const uint8_t* zeros, void* packed_codes,
                                void* packed_scales, uint8_t* packed_zeros, void* stream) {
    if (!sizes_ok(E, N, K)) return MEP_ERR_SHAPE;
    if ((kind != MEP_WEIGHT_INT4 && kind != MEP_WEIGHT_FP4) || !group_ok(group) ||
        (zeros != nullptr) != (packed_zeros != nullptr) || (zeros && kind != MEP_WEIGHT_INT4))
        return MEP_ERR_PARAM;
    if (!codes || !scales || !packed_codes || !packed_scales) return MEP_ERR_NULLPTR;
    if (!rows::aligned16(packed_codes) || !rows::aligned16(packed_scales) ||
        (packed_zeros && !rows::aligned16(packed_zeros)) || ((uintptr_t)scales & 1u) ||
        ((uintptr_t)codes & 7u))
        return MEP_ERR_SHAPE;
    hipStream_t s = (hipStream_t)stream;
    const int tiles = (int)row_tiles(N), KB = (int)blocks_of(K);
    const int G = (K + group - 1) / group, per = kPackK / group;
    const size_t nc = (size_t)E * tiles * KB * 64;
    const size_t ns = mep_packed_scale_count(E, N, K, group);
    hipLaunchKernelGGL(pack_codes, blocks(nc, kPackThreads), dim3(kPackThreads), 0, s, codes,
                       (u32x4*)packed_codes, N, K, tiles, KB, kind == MEP_WEIGHT_FP4 ? 1 : 0, nc);
    hipLaunchKernelGGL(pack_groups<uint16_t>, blocks(ns, kPackThreads), dim3(kPackThreads), 0, s,
                       (const uint16_t*)scales, (uint16_t*)packed_scales, N, G, tiles, KB, per, ns);
    if (zeros)
        hipLaunchKernelGGL(pack_groups<uint8_t>, blocks(ns, kPackThreads), dim3(kPackThreads), 0,
                           s, zeros, packed_zeros, N, G, tiles, KB, per, ns);
    MEP_LAUNCH_CHECK();
    return MEP_OK;
}

extern "C" int mep_quant_weights(int E, int N, int K, int kind, int group, int scale_dtype,
                                 const uint16_t* w, uint8_t* codes, void* scales, void* stream) {
    if (!sizes_ok(E, N, K)) return MEP_ERR_SHAPE;
    if ((kind != MEP_WEIGHT_INT4 && kind != MEP_WEIGHT_FP4) || !group_ok(group) ||
        (scale_dtype != MEP_SCALE_BF16 && scale_dtype != MEP_SCALE_F16))
        return MEP_ERR_PARAM;
    if (!w || !codes || !scales) return MEP_ERR_NULLPTR;
    if (((uintptr_t)w & 1u) || ((uintptr_t)scales & 1u)) return MEP_ERR_SHAPE;
    const int G = (K + group - 1) / group;
    const size_t total = (size_t)E * N * G;
    hipLaunchKernelGGL(quant_groups, blocks(total, kPackThreads / kWave), dim3(kPackThreads), 0,
                       (hipStream_t)stream, w, codes, (uint16_t*)scales, K, group, G,
                       kind == MEP_WEIGHT_FP4 ? 1 : 0, scale_dtype == MEP_SCALE_F16 ? 1 : 0,
                       total);
    MEP_LAUNCH_CHECK();
    return MEP_OK;
}
