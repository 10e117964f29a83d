// The expert layer's kernels for bf16 weights.
#include "experts.h"

namespace mep {
namespace experts {

void layer_bf16(hipStream_t s, const RowsArgs& a, const DownArgs& d) {
    if (a.w.K % 128 == 0 && d.w.K % 128 == 0)
        launch_layer<Bf16Weights<true>>(s, a, d);
    else
        launch_layer<Bf16Weights<false>>(s, a, d);
}

}  // namespace experts
}  // namespace mep
