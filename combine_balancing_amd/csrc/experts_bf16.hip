// The expert layer's kernels for bf16 weights.
#include "experts.h"

namespace mep {
namespace experts {

void layer_bf16(hipStream_t s, const RowsArgs& a, const DownArgs& d) {
    launch_layer<Bf16Weights>(s, a, d);
}

}  // namespace experts
}  // namespace mep
