// The experts' products and the expert layer for 4-bit float weights.
#include "experts.h"

namespace mep {
namespace experts {
namespace {

template <class F>
void with_kind(const Kind& k, F f) {
#define MEP_GROUP(G)                                     \
    if (k.f16) f(PackedWeights<true, G, false, true>{}); \
    else f(PackedWeights<true, G, false, false>{});
    if (k.group == 32) {
        MEP_GROUP(32)
    } else if (k.group == 64) {
        MEP_GROUP(64)
    } else {
        MEP_GROUP(128)
    }
#undef MEP_GROUP
}

}  // namespace

void matvec_fp4(hipStream_t s, const Kind& k, const RowsArgs& a) {
    with_kind(k, [&](auto w) { launch_matvec<decltype(w)>(s, a); });
}

void layer_fp4(hipStream_t s, const Kind& k, const RowsArgs& a, const DownArgs& d) {
    with_kind(k, [&](auto w) { launch_layer<decltype(w)>(s, a, d); });
}

}  // namespace experts
}  // namespace mep
