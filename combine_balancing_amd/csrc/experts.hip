// Entry points of the experts' products for a few routes (kernels in
// experts.h; one source per weight kind, so that they compile in parallel).
#include "experts.h"

using namespace mep;
using namespace mep::experts;

namespace {

constexpr int kMaxDim = 65536;  // H, I, N, K of the layer's and product's matrices

// Status of a weight set, and its view for the kernels.
int view_of(const mep_weights* m, Weights* w) {
    if (!m) return MEP_ERR_NULLPTR;
    if (m->E < 1 || m->E > kMaxExperts || m->N < 1 || m->N > (1 << 20) || m->K < 8 ||
        m->K > kMaxDim || m->K % 8 != 0)
        return MEP_ERR_SHAPE;
    if (m->kind == MEP_WEIGHT_BF16) {
        if (m->scales || m->zeros) return MEP_ERR_PARAM;
    } else if (m->kind == MEP_WEIGHT_INT4 || m->kind == MEP_WEIGHT_FP4) {
        if (m->group != 32 && m->group != 64 && m->group != 128) return MEP_ERR_PARAM;
        if (m->scale_dtype != MEP_SCALE_BF16 && m->scale_dtype != MEP_SCALE_F16)
            return MEP_ERR_PARAM;
        if (m->zeros && m->kind != MEP_WEIGHT_INT4) return MEP_ERR_PARAM;
        if (!m->scales) return MEP_ERR_NULLPTR;
    } else {
        return MEP_ERR_PARAM;
    }
    if (!m->data) return MEP_ERR_NULLPTR;
    if (!rows::aligned16(m->data) || (m->scales && !rows::aligned16(m->scales)) ||
        (m->zeros && !rows::aligned16(m->zeros)))
        return MEP_ERR_SHAPE;
    w->codes = (const u32x4*)m->data;
    w->scales = (const uint16_t*)m->scales;
    w->zeros = m->zeros;
    w->N = m->N;
    w->K = m->K;
    w->KV = m->K / 8;
    w->tiles = (m->N + kTile - 1) / kTile;
    w->KB = (m->K + kPackK - 1) / kPackK;
    return MEP_OK;
}

Kind kind_of(const mep_weights* m) {
    return {m->group, m->zeros != nullptr, m->scale_dtype == MEP_SCALE_F16};
}

size_t table_bytes() { return (sizeof(Table) + 255) / 256 * 256; }

}  // namespace

extern "C" int mep_expert_matvec(int T, int R, int first, const uint16_t* x, int x_per_route,
                                 const int32_t* ids, const uint8_t* mask, const mep_weights* wts,
                                 uint16_t* out_bf16, float* out_f32, void* stream) {
    Weights w;
    const int rc = view_of(wts, &w);
    if (rc != MEP_OK) return rc;
    const long long n = (long long)T * (ids ? R : 1);
    if (T < 0 || (ids && R < 1) || n > kMaxRoutes) return MEP_ERR_SHAPE;
    if (wts->kind == MEP_WEIGHT_BF16 || (!ids && (wts->E != 1 || mask || x_per_route || first)))
        return MEP_ERR_PARAM;
    if ((out_bf16 != nullptr) == (out_f32 != nullptr) && T > 0)
        return out_bf16 ? MEP_ERR_PARAM : MEP_ERR_NULLPTR;
    if (T == 0) return MEP_OK;
    if (!x) return MEP_ERR_NULLPTR;
    if (!rows::aligned16(x) || ((uintptr_t)out_bf16 & 1u) || ((uintptr_t)out_f32 & 3u))
        return MEP_ERR_SHAPE;
    RowsArgs a = {};
    a.x = (const u32x4*)x;
    a.div = ids && !x_per_route ? R : 1;
    a.ids = (const int*)ids;
    a.mask = mask;
    a.n = (int)n;
    a.first = first;
    a.E = wts->E;
    a.w = w;
    a.out = out_f32 ? (void*)out_f32 : (void*)out_bf16;
    a.out_f32 = out_f32 != nullptr;
    if (wts->kind == MEP_WEIGHT_INT4)
        matvec_int4((hipStream_t)stream, kind_of(wts), a);
    else
        matvec_fp4((hipStream_t)stream, kind_of(wts), a);
    MEP_LAUNCH_CHECK();
    return MEP_OK;
}

extern "C" size_t mep_moe_layer_workspace_size(int T, int K, int I) {
    if (T < 0 || T > kMaxLayerTokens || K < 1 || (long long)T * K > kMaxRoutes || I < 8 ||
        I > kMaxDim || I % 8 != 0)
        return 0;
    return table_bytes() + (size_t)T * K * padded(I) * 2 * 3;  // up to 3 bf16 terms
}

extern "C" int mep_moe_layer(int T, int K, int H, int I, int first, const uint16_t* x,
                             const int32_t* ids, const float* scores, const uint8_t* mask,
                             const mep_weights* w13, const mep_weights* w2, void* workspace,
                             size_t workspace_bytes, uint16_t* out_bf16, float* out_f32,
                             void* stream) {
    const size_t need = mep_moe_layer_workspace_size(T, K, I);
    if (need == 0 || H < 8 || H > kMaxDim || H % 8 != 0) return MEP_ERR_SHAPE;
    Weights up, down;
    int rc = view_of(w13, &up);
    if (rc == MEP_OK) rc = view_of(w2, &down);
    if (rc != MEP_OK) return rc;
    if (w13->N != 2 * I || w13->K != H || w2->N != H || w2->K != I) return MEP_ERR_SHAPE;
    if (w13->E != w2->E || w13->kind != w2->kind || w13->group != w2->group ||
        w13->scale_dtype != w2->scale_dtype || !w13->zeros != !w2->zeros)
        return MEP_ERR_PARAM;
    if (T == 0) return MEP_OK;
    if (!x || !ids || !scores || !workspace || (!out_bf16 && !out_f32)) return MEP_ERR_NULLPTR;
    if (workspace_bytes < need || ((uintptr_t)workspace & 255u)) return MEP_ERR_PARAM;
    if (!rows::aligned16(x) || (out_bf16 && !rows::aligned16(out_bf16)) ||
        (out_f32 && !rows::aligned16(out_f32)))
        return MEP_ERR_SHAPE;
    RowsArgs a = {};
    a.x = (const u32x4*)x;
    a.div = K;
    a.ids = (const int*)ids;
    a.mask = mask;
    a.n = T * K;
    a.first = first;
    a.E = w13->E;
    a.w = up;
    a.h = (u32x4*)((char*)workspace + table_bytes());
    a.I = I;
    a.terms = out_f32 ? 3 : 2;
    a.table = (Table*)workspace;
    DownArgs d = {};
    d.h = a.h;
    d.table = a.table;
    d.ids = a.ids;
    d.mask = mask;
    d.first = first;
    d.scores = scores;
    d.T = T;
    d.K = K;
    d.n = T * K;
    d.E = w2->E;
    d.w = down;
    d.out_bf16 = out_bf16;
    d.out_f32 = out_f32;
    hipStream_t s = (hipStream_t)stream;
    if (w13->kind == MEP_WEIGHT_BF16)
        layer_bf16(s, a, d);
    else if (w13->kind == MEP_WEIGHT_INT4)
        layer_int4(s, kind_of(w13), a, d);
    else
        layer_fp4(s, kind_of(w13), a, d);
    MEP_LAUNCH_CHECK();
    return MEP_OK;
}
