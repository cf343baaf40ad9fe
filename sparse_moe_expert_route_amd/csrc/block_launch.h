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

// ---------------------------------------------------------------------------
// The layer for few tokens (few.hip).
// ---------------------------------------------------------------------------
constexpr int kFewMaxT = 16;              // tokens: one 16-row MFMA tile per expert
constexpr int kFewMaxWidth = 65536;       // H and I: item counts and offsets inside an expert stay 32-bit
constexpr int kFewRowBytes = 122880;      // T (H + 16) at most: the FP8 rows of x in LDS
constexpr int kFewParts = 4;              // partial sums of a router logit
constexpr int kFewTailMaxH = 16384;       // H of the block: a row of the tail in a workgroup's registers
constexpr int kFewCounterStride = 32;     // words between counters: each has its own 128-byte line
constexpr uint32_t kErrStalled = 8u;      // error word 0: a wait inside the kernel was given up

// Counters of one call: the ticket, then per touched expert (at most 8 kFewMaxT)
// the quantised 128-channel blocks of h (with at most 8 experts, 8 times over: the
// workgroups' polls are spread), then the finished down items of each
// 32 output features, then the summed features, then the finished parts of each
// block of h; behind them kFewPad words that stay zero (what the kernel
// loads past the end of K).
constexpr int kFewPad = 512;
constexpr int kFewGrid = 256;             // workgroups of the layer kernel: one per CU
constexpr int kFewMaxSplit = 8;           // parts of K in the gate/up items
constexpr int kFewSplitBlocks = kFewGrid / 2;   // blocks of h at most, where K is split
// floats of the parts' sums: 8 items of two 16 x 16 tiles to each of kFewGrid runs
constexpr size_t kFewPartFloats = (size_t)kFewGrid * 8 * 512;
inline int few_counters(int H) { return kFewCounterStride * (2 + 8 * kFewMaxT + H / 32 + kFewSplitBlocks) + kFewPad; }

struct FewArgs {
    const uint16_t* x;          // [T][H] bf16 (null: the norm of r)
    const void* r;              // [T][H] residual stream, tail.res_bf16, normalised with w_pre and tail.eps
    const void* w_pre;          // [H] tail.param_bf16, or null (ones)
    const uint16_t* w_router;   // [E][H] bf16
    const float* bias;          // [E] or null
    const uint8_t* w13;
    const uint8_t* w13_scale;
    const uint8_t* w2;
    const uint8_t* w2_scale;
    void* y;                    // [T][H] float32 or bf16 (fuse_tail: float32 workspace)
    int out_bf16;
    int fuse_tail;              // the block's tail on y in the same launch
    TailArgs tail;
    int T, H, I, E, k, sigmoid;
    // workspace
    uint32_t* err;              // two error words
    uint32_t* counters;         // few_counters(H)
    int n_counters;
    float* logits;              // [kFewParts][T][E]
    uint8_t* xq;                // [T][H] e4m3
    void* xs;                   // [T][H / 128] e8m0 or float32
    uint8_t* hq;                // [T k][I] e4m3
    void* hs;                   // [T k][I / 128]
    float* y_slot;              // [T k][H]
    float* part;                // kFewPartFloats
};
hipError_t launch_few_layer(const FewArgs& a, int packed, int fp8_block, hipStream_t stream);
// its second kernel, by the experts' format
hipError_t launch_few_layer_mxfp4(const FewArgs& a, int packed, hipStream_t stream);
hipError_t launch_few_layer_fp8(const FewArgs& a, int packed, hipStream_t stream);

}  // namespace moe
