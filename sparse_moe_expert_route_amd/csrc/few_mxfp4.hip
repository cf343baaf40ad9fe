// The layer kernel for few tokens (few_layer.h) with MXFP4 experts.
#include "few_layer.h"

namespace moe {

hipError_t launch_few_layer_mxfp4(const FewArgs& a, int packed, hipStream_t stream) {
    return packed ? launch_layer<0, true>(a, stream) : launch_layer<2, false>(a, stream);
}

}  // namespace moe
