// The experts' products and the expert layer for int4 weights.
#include "experts.h"

namespace mep {
namespace experts {
namespace {

template <class F>
void with_kind(const Kind& k, F f) {
#define MEP_KIND(G, Z, H) f(PackedWeights<false, G, Z, H>{})
#define MEP_GROUP(G)                                          \
    if (k.zeros) {                                            \
        if (k.f16) MEP_KIND(G, true, true); else MEP_KIND(G, true, false);   \
    } else {                                                  \
        if (k.f16) MEP_KIND(G, false, true); else MEP_KIND(G, false, false); \
    }
    if (k.group == 32) {
        MEP_GROUP(32)
    } else if (k.group == 64) {
        MEP_GROUP(64)
    } else {
        MEP_GROUP(128)
    }
#undef MEP_GROUP
#undef MEP_KIND
}

}  // namespace

void matvec_int4(hipStream_t s, const Kind& k, const RowsArgs& a) {
    with_kind(k, [&](auto w) { launch_matvec<decltype(w)>(s, a); });
}

void layer_int4(hipStream_t s, const Kind& k, const RowsArgs& a, const DownArgs& d) {
    with_kind(k, [&](auto w) { launch_layer<decltype(w)>(s, a, d); });
}

}  // namespace experts
}  // namespace mep
