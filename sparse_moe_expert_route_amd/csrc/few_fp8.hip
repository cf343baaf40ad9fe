// The layer kernel for few tokens (few_layer.h) with FP8 block-scaled experts.
#include "few_layer.h"

namespace moe {

hipError_t launch_few_layer_fp8(const FewArgs& a, int packed, hipStream_t stream) {
    return packed ? launch_layer<1, true>(a, stream) : launch_layer<1, false>(a, stream);
}

}  // namespace moe
