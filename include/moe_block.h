/*
 * moe_block.h - C ABI of the decoder block around the routed Mixture-of-Experts
 * layer of moe.h, and of the layer's form for few tokens (gfx950).
 *
 * With r [T][H] the residual stream and moe() the layer of moe.h:
 *
 *   n  = RMSNorm(r; w_pre)                   moe_block_norm
 *   y  = moe(n)                              moe_forward, or moe_forward_few (T <= 16)
 *   z  = RMSNorm(y; w_post), or y            \
 *   r' = r + scale * gate * z                 | moe_block_residual, moe_combine_residual
 *   n' = RMSNorm(r'; w_next)   (optional)    /
 *   all of it                                moe_block_forward
 *
 *   RMSNorm(v; w)[c] = v[c] * w[c] / sqrt(sum_c v[c]^2 / H + eps),   w = 1 where it is NULL
 *
 * Arithmetic: norms, gate and residual sums in float32 (a 32-bit sum of squares
 * over the row); n and n' are rounded once to bf16, r' once to its own type.
 * n' is the norm of r' as stored, so it equals what a moe_block_norm of r_out
 * would write.
 *
 * The conventions of moe.h hold for every entry point here: device pointers,
 * 16-byte aligned, row-major and dense; work enqueued on `stream` (a stream of
 * the current device) and not waited for; nothing allocated; outputs fully
 * overwritten; argument errors found before anything is enqueued;
 * num_tokens == 0 returns MOE_OK and launches nothing; inputs finite, and every
 * sum of squares inside the float32 range.  hidden is at most
 * MOE_BLOCK_MAX_HIDDEN where a norm is taken (MOE_ERR_UNSUPPORTED above).  Calls
 * captured into a graph may be replayed; calls that can overlap need a workspace
 * each.
 */
#ifndef MOE_BLOCK_MI355X_H
#define MOE_BLOCK_MI355X_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest num_tokens of moe_forward_few: one 16-row MFMA tile per expert. */
#define MOE_FEW_MAX_TOKENS 16
/* Largest hidden and intermediate of moe_forward_few, and the largest
 * num_tokens * (hidden + 16): the FP8 rows of x are kept in LDS (16 tokens up to
 * hidden 7664, 14 at 8192, 7 at 16384). */
#define MOE_FEW_MAX_WIDTH 65536
#define MOE_FEW_MAX_ROW_BYTES 122880
/* Largest hidden of the entry points of this header that take a norm. */
#define MOE_BLOCK_MAX_HIDDEN 16384

/* Bit of device error word 0 (moe_error_words_offset) after moe_forward_few or
 * moe_block_forward: a wait inside the kernel was given up after seconds, and
 * the call's results are unspecified.  No argument or data leads to it.     */
#define MOE_DEVERR_STALLED 8

/* What follows the layer.  Types are moe_out_dtype values (MOE_OUT_F32,
 * MOE_OUT_BF16).
 *   r          [T][H] residual stream, res_dtype
 *   r_out      [T][H] out, res_dtype; r itself (in place) or memory that does
 *              not overlap any input
 *   w_post     [H] param_dtype, or NULL (= 1); read only if post_norm is 1
 *   gate       NULL (= 1), [H] (gate_per_token 0) or [T][H] (gate_per_token 1),
 *              param_dtype
 *   w_next     [H] param_dtype, or NULL (= 1); read only with n_next
 *   n_next     [T][H] bf16 out, or NULL: not computed
 *   scale      residual scale, finite
 *   eps        finite and > 0; of every norm of the call
 *   post_norm  1: z = RMSNorm(y; w_post), 0: z = y                         */
typedef struct {
    const void* r;
    void* r_out;
    const void* w_post;
    const void* gate;
    const void* w_next;
    void* n_next;
    float scale;
    float eps;
    int32_t res_dtype;
    int32_t param_dtype;
    int32_t post_norm;
    int32_t gate_per_token;
} moe_block_tail;

/* Workspace bytes for every entry point of this header that takes one (and
 * for moe_forward on the same problem).  Returns 0 for an invalid problem. */
size_t moe_block_workspace_size(const moe_problem* problem);

/* n = bf16(RMSNorm(r; w)).
 *   r [T][H] res_dtype, w [H] param_dtype or NULL, n [T][H] bf16 out (not
 *   overlapping r)                                                          */
moe_status moe_block_norm(const moe_problem* problem, const void* r, int32_t res_dtype, const void* w,
                          int32_t param_dtype, float eps, void* n_bf16, hipStream_t stream);

/* The tail on a layer output y [T][H] (y_dtype): r_out and, if asked for, n_next. */
moe_status moe_block_residual(const moe_problem* problem, const void* y, int32_t y_dtype,
                              const moe_block_tail* tail, hipStream_t stream);

/* The tail on y[t] = sum_j topk_w[t][j] * y_perm[row_of_slot[t*k + j]], the
 * weighted sum of moe_combine (same order, float32, not rounded; slots whose
 * row is outside [0, T*k) add nothing), which is not stored.               */
moe_status moe_combine_residual(const moe_problem* problem, const float* y_perm, const int32_t* row_of_slot,
                                const float* topk_w, const moe_block_tail* tail, hipStream_t stream);

/* The whole layer for few tokens: num_tokens <= MOE_FEW_MAX_TOKENS, hidden and
 * intermediate <= MOE_FEW_MAX_WIDTH and num_tokens * (hidden + 16) <=
 * MOE_FEW_MAX_ROW_BYTES (MOE_ERR_UNSUPPORTED above): the computation of
 * moe_forward with every rounding of its definition (FP8 activations, FP8 h), in
 * two launches.  Float32 sums are taken in another order than moe_forward's, one
 * that depends on the sizes alone.  With FP8 block-scaled experts the
 * activation and h scales are the float32 product amax * (1 / 448), at most an
 * ulp from moe_forward's quotient (bf16 activations often lie on the border of
 * two codes, so about one code in a thousand differs); codes are the e4m3
 * rounding of v / scale as there.  workspace: at least
 * moe_block_workspace_size(problem) bytes, 256-byte aligned.               */
moe_status moe_forward_few(const moe_problem* problem, const void* x_bf16, const void* w_router_bf16,
                           const float* sel_bias, const moe_expert_weights* weights, void* y, int32_t out_dtype,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/* The block: n = RMSNorm(tail->r; w_pre), the layer on n, the tail.  w_pre is
 * [H] tail->param_dtype or NULL (= 1).  Any num_tokens; within
 * the limits of moe_forward_few the layer runs as there, beyond them as in
 * moe_forward (the bits of norm, moe_forward and residual in turn).         */
moe_status moe_block_forward(const moe_problem* problem, const void* w_pre, const void* w_router_bf16,
                             const float* sel_bias, const moe_expert_weights* weights, const moe_block_tail* tail,
                             void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_MI355X_H */
