// Argument checks and workspace arithmetic shared by the host code of the C ABI
// (abi.cpp, abi_block.cpp).  Plain C++: it also builds with a host compiler.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "moe.h"
#include "moe_launch.h"

namespace moe {

constexpr size_t kAlign = 256;

inline size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline moe_status check_problem(const moe_problem* p) {
    if (!p) return MOE_ERR_INVALID_ARGUMENT;
    if (p->num_tokens < 0) return MOE_ERR_INVALID_ARGUMENT;
    if (p->hidden <= 0 || p->hidden % kFp8Block) return MOE_ERR_INVALID_ARGUMENT;
    if (p->intermediate <= 0 || p->intermediate % kFp8Block) return MOE_ERR_INVALID_ARGUMENT;
    if (p->num_experts < 1 || p->num_experts > 512) return MOE_ERR_INVALID_ARGUMENT;
    if (p->top_k < 1 || p->top_k > 8 || p->top_k > p->num_experts) return MOE_ERR_INVALID_ARGUMENT;
    if (p->score_func != MOE_SCORE_SOFTMAX_TOPK && p->score_func != MOE_SCORE_SIGMOID_BIAS) return MOE_ERR_UNSUPPORTED;
    if (p->expert_format != MOE_EXPERTS_MXFP4 && p->expert_format != MOE_EXPERTS_FP8_BLOCK) return MOE_ERR_UNSUPPORTED;
    if (p->num_tokens * (int64_t)p->top_k >= ((int64_t)1 << 31)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

template <typename T>
T* at(void* ws, size_t off) { return (T*)((char*)ws + off); }

inline moe_status check_weights(const moe_expert_weights* w) {
    if (!w || !w->w13 || !w->w13_scale || !w->w2 || !w->w2_scale) return MOE_ERR_INVALID_ARGUMENT;
    if (!aligned16(w->w13) || !aligned16(w->w13_scale) || !aligned16(w->w2) || !aligned16(w->w2_scale))
        return MOE_ERR_INVALID_ARGUMENT;
    if (w->layout != MOE_WEIGHTS_CANONICAL && w->layout != MOE_WEIGHTS_PACKED) return MOE_ERR_INVALID_ARGUMENT;
    return MOE_OK;
}

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// What the expert GEMMs leave in the workspace for a combine.
struct ExpertRows {
    const float* y_perm;
    const int32_t* row_of_slot;
    const float* w;
};

// The launches of moe_forward but its combine, on checked arguments, num_tokens > 0
// and a workspace of moe_workspace_size bytes (abi.cpp).
moe_status forward_rows(const moe_problem* p, const void* x_bf16, const void* w_router_bf16, const float* sel_bias,
                        const moe_expert_weights* weights, void* ws, ExpertRows* out, hipStream_t stream);

inline bool all_aligned() { return true; }
template <typename P, typename... R>
inline bool all_aligned(P p, R... rest) { return p && aligned16(p) && all_aligned(rest...); }

}  // namespace moe

#define MOE_CHECK(expr)                          \
    do {                                         \
        const moe_status st_ = (expr);           \
        if (st_ != MOE_OK) return st_;           \
    } while (0)
#define MOE_LAUNCH(expr)                         \
    do {                                         \
        if ((expr) != hipSuccess) return MOE_ERR_HIP; \
    } while (0)
