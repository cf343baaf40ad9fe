// Host-side declarations of the kernels around the layer (block_norm.hip) and
// of the layer for few tokens (few.hip): argument blocks and launchers, shared
// with the host code of the ABI (abi_block.cpp).  Plain C++ over the HIP
// runtime API.  Not part of the public ABI (include/moe_block.h is).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "moe_launch.h"

namespace moe {

// The tail of the block (moe_block_tail of moe_block.h) as the kernels take it.
struct TailArgs {
    const void* r;
    void* r_out;
    const void* w_post;   // null: ones
    const void* gate;     // null: ones
    const void* w_next;   // null: ones
    void* n_next;         // null: not written
    float scale, eps;
    int res_bf16, param_bf16, post_norm, gate_per_token;
};

// n[t] = bf16(RMSNorm(r[t]; w)) for T rows of H channels.
hipError_t launch_block_norm(const void* r, int res_bf16, const void* w, int param_bf16, float eps, uint16_t* n,
                             int64_t T, int H, hipStream_t stream);
// The tail on a given y [T][H].
hipError_t launch_block_residual(const void* y, int y_bf16, const TailArgs& t, int64_t T, int H, hipStream_t stream);
// The tail on y[t] = sum_j w[t][j] y_perm[row_of_slot[t k + j]].
hipError_t launch_combine_residual(const float* y_perm, const int32_t* row_of_slot, const float* w, const TailArgs& t,
                                   int64_t T, int H, int k, hipStream_t stream);

}  // namespace moe
