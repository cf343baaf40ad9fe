// Host side of the C ABI declared in include/moe_block.h: argument validation,
// workspace carving and the launch sequence of each entry point.
//
// Nothing here allocates, synchronises or throws; every check happens before
// the first launch, so a rejected call enqueues nothing.
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "abi_checks.h"
#include "block_launch.h"
#include "moe_block.h"

namespace {

using namespace moe;

bool dtype_ok(int32_t d) { return d == MOE_OUT_F32 || d == MOE_OUT_BF16; }
size_t dtype_size(int32_t d) { return d == MOE_OUT_BF16 ? 2 : 4; }
bool eps_ok(float eps) { return std::isfinite(eps) && eps > 0.0f; }
// a pointer that may be NULL
bool opt_aligned(const void* p) { return aligned16(p); }

// A problem of this header: valid, and its rows fit the norm kernels.
moe_status check_block_problem(const moe_problem* p) {
    MOE_CHECK(check_problem(p));
    if (p->hidden > MOE_BLOCK_MAX_HIDDEN) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Within the limits of moe_forward_few.
bool few_supported(const moe_problem& p) {
    return p.num_tokens <= kFewMaxT && p.hidden <= kFewMaxWidth && p.intermediate <= kFewMaxWidth &&
           p.num_tokens * (p.hidden + 16) <= kFewRowBytes;
}

struct Span { const void* p; size_t n; };

// The tail's own fields, and that neither of its outputs overlaps an input
// (r_out may be r itself) or the other.  `in` are the call's further inputs.
template <size_t N>
moe_status check_tail(const moe_problem& p, const moe_block_tail* t, const Span (&in)[N]) {
    if (!t || !dtype_ok(t->res_dtype) || !dtype_ok(t->param_dtype)) return MOE_ERR_INVALID_ARGUMENT;
    if (!all_aligned(t->r, t->r_out)) return MOE_ERR_INVALID_ARGUMENT;
    if (!opt_aligned(t->w_post) || !opt_aligned(t->gate) || !opt_aligned(t->w_next) || !opt_aligned(t->n_next))
        return MOE_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(t->scale) || !eps_ok(t->eps)) return MOE_ERR_INVALID_ARGUMENT;
    if ((t->post_norm != 0 && t->post_norm != 1) || (t->gate_per_token != 0 && t->gate_per_token != 1))
        return MOE_ERR_INVALID_ARGUMENT;
    const size_t T = (size_t)p.num_tokens, H = (size_t)p.hidden;
    const size_t nr = T * H * dtype_size(t->res_dtype), nn = T * H * 2, np = H * dtype_size(t->param_dtype);
    const Span own[3] = {{t->w_post, np}, {t->gate, t->gate_per_token ? T * np : np}, {t->w_next, np}};
    auto hits = [&](const void* out, size_t n) {
        for (const Span& s : own)
            if (s.p && overlaps(out, n, s.p, s.n)) return true;
        for (const Span& s : in)
            if (s.p && overlaps(out, n, s.p, s.n)) return true;
        return false;
    };
    if (t->r_out != t->r && overlaps(t->r_out, nr, t->r, nr)) return MOE_ERR_INVALID_ARGUMENT;
    if (hits(t->r_out, nr)) return MOE_ERR_INVALID_ARGUMENT;
    if (t->n_next && (hits(t->n_next, nn) || overlaps(t->n_next, nn, t->r, nr) || overlaps(t->n_next, nn, t->r_out, nr)))
        return MOE_ERR_INVALID_ARGUMENT;
    return MOE_OK;
}

TailArgs tail_args(const moe_block_tail& t) {
    TailArgs a;
    a.r = t.r; a.r_out = t.r_out; a.w_post = t.w_post; a.gate = t.gate; a.w_next = t.w_next; a.n_next = t.n_next;
    a.scale = t.scale; a.eps = t.eps;
    a.res_bf16 = t.res_dtype == MOE_OUT_BF16; a.param_bf16 = t.param_dtype == MOE_OUT_BF16;
    a.post_norm = t.post_norm; a.gate_per_token = t.gate_per_token;
    return a;
}

// The layer's own workspace first (so that its error words stay where
// moe_error_words_offset says), then the block's intermediates.
struct BlockLayout {
    size_t layer, n, total;
    // few_supported() only
    size_t y, counters, logits, xq, xs, hq, hs, y_slot, part;
};

static_assert(kFewTailMaxH == MOE_BLOCK_MAX_HIDDEN && kFewMaxT == MOE_FEW_MAX_TOKENS && kFewMaxWidth == MOE_FEW_MAX_WIDTH &&
                  kFewRowBytes == MOE_FEW_MAX_ROW_BYTES && kErrStalled == MOE_DEVERR_STALLED,
              "constants of the kernels and of moe_block.h");

BlockLayout block_layout(const moe_problem& p) {
    const size_t T = (size_t)p.num_tokens, H = (size_t)p.hidden;
    BlockLayout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off += round_up(bytes ? bytes : 1); return o; };
    L.layer = take(moe_workspace_size(&p));
    L.n = take(T * H * 2);
    if (few_supported(p)) {
        L.y = take(T * H * 4);
        const size_t I = (size_t)p.intermediate, N = T * (size_t)p.top_k;
        L.counters = take((size_t)few_counters(p.hidden) * 4);
        L.logits = take(kFewParts * T * (size_t)p.num_experts * 4);
        L.xq = take(T * H);
        L.xs = take(T * (H / kFp8Block) * 4);
        L.hq = take(N * I);
        L.hs = take(N * (I / kFp8Block) * 4);
        L.y_slot = take(N * H * 4);
        L.part = take(kFewPartFloats * 4);
    }
    L.total = off;
    return L;
}

moe_status check_block_ws(const moe_problem& p, const void* ws, size_t ws_bytes) {
    if (!ws || ((uintptr_t)ws % kAlign) != 0) return MOE_ERR_INVALID_ARGUMENT;
    if (ws_bytes < block_layout(p).total) return MOE_ERR_WORKSPACE_TOO_SMALL;
    return MOE_OK;
}

// The layer for few tokens on x, or, with x null, the block on tail's residual
// stream (y: workspace then).  The tail joins the layer's launch where a row fits
// a wave's registers.
moe_status run_few(const moe_problem& p, const void* x, const void* w_pre, const moe_block_tail* tail,
                   const void* w_router, const float* bias, const moe_expert_weights& w, void* y, bool out_bf16,
                   void* ws, hipStream_t stream) {
    const BlockLayout L = block_layout(p);
    FewArgs a{};
    a.x = (const uint16_t*)x;
    if (!x) {
        a.tail = tail_args(*tail);
        a.r = tail->r;
        a.w_pre = w_pre;
        a.fuse_tail = 1;
    }
    a.w_router = (const uint16_t*)w_router; a.bias = bias;
    a.w13 = w.w13; a.w13_scale = w.w13_scale; a.w2 = w.w2; a.w2_scale = w.w2_scale;
    a.y = y; a.out_bf16 = out_bf16;
    a.T = (int)p.num_tokens; a.H = p.hidden; a.I = p.intermediate; a.E = p.num_experts; a.k = p.top_k;
    a.sigmoid = p.score_func == MOE_SCORE_SIGMOID_BIAS;
    a.err = at<uint32_t>(ws, moe_error_words_offset());
    a.counters = at<uint32_t>(ws, L.counters);
    a.n_counters = few_counters(p.hidden);
    a.logits = at<float>(ws, L.logits);
    a.xq = at<uint8_t>(ws, L.xq); a.xs = at<void>(ws, L.xs);
    a.hq = at<uint8_t>(ws, L.hq); a.hs = at<void>(ws, L.hs);
    a.y_slot = at<float>(ws, L.y_slot);
    a.part = at<float>(ws, L.part);
    MOE_LAUNCH(launch_few_layer(a, w.layout == MOE_WEIGHTS_PACKED, p.expert_format == MOE_EXPERTS_FP8_BLOCK, stream));
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_block_workspace_size(const moe_problem* p) {
    if (check_problem(p) != MOE_OK) return 0;
    return block_layout(*p).total;
}

moe_status moe_block_norm(const moe_problem* p, const void* r, int32_t res_dtype, const void* w, int32_t param_dtype,
                          float eps, void* n_bf16, hipStream_t stream) {
    MOE_CHECK(check_block_problem(p));
    if (!dtype_ok(res_dtype) || !dtype_ok(param_dtype) || !eps_ok(eps)) return MOE_ERR_INVALID_ARGUMENT;
    if (!all_aligned(r, n_bf16) || !opt_aligned(w)) return MOE_ERR_INVALID_ARGUMENT;
    const size_t n = (size_t)p->num_tokens * (size_t)p->hidden;
    if (overlaps(n_bf16, n * 2, r, n * dtype_size(res_dtype))) return MOE_ERR_INVALID_ARGUMENT;
    if (w && overlaps(n_bf16, n * 2, w, (size_t)p->hidden * dtype_size(param_dtype))) return MOE_ERR_INVALID_ARGUMENT;
    if (p->num_tokens == 0) return MOE_OK;
    MOE_LAUNCH(launch_block_norm(r, res_dtype == MOE_OUT_BF16, w, param_dtype == MOE_OUT_BF16, eps, (uint16_t*)n_bf16,
                                 p->num_tokens, p->hidden, stream));
    return MOE_OK;
}

moe_status moe_block_residual(const moe_problem* p, const void* y, int32_t y_dtype, const moe_block_tail* tail,
                              hipStream_t stream) {
    MOE_CHECK(check_block_problem(p));
    if (!dtype_ok(y_dtype) || !all_aligned(y)) return MOE_ERR_INVALID_ARGUMENT;
    const Span in[1] = {{y, (size_t)p->num_tokens * (size_t)p->hidden * dtype_size(y_dtype)}};
    MOE_CHECK(check_tail(*p, tail, in));
    if (p->num_tokens == 0) return MOE_OK;
    MOE_LAUNCH(launch_block_residual(y, y_dtype == MOE_OUT_BF16, tail_args(*tail), p->num_tokens, p->hidden, stream));
    return MOE_OK;
}

moe_status moe_combine_residual(const moe_problem* p, const float* y_perm, const int32_t* row_of_slot,
                                const float* topk_w, const moe_block_tail* tail, hipStream_t stream) {
    MOE_CHECK(check_block_problem(p));
    if (!all_aligned(y_perm, row_of_slot, topk_w)) return MOE_ERR_INVALID_ARGUMENT;
    const size_t N = (size_t)p->num_tokens * (size_t)p->top_k;
    const Span in[3] = {{y_perm, N * (size_t)p->hidden * 4}, {row_of_slot, N * 4}, {topk_w, N * 4}};
    MOE_CHECK(check_tail(*p, tail, in));
    if (p->num_tokens == 0) return MOE_OK;
    MOE_LAUNCH(launch_combine_residual(y_perm, row_of_slot, topk_w, tail_args(*tail), p->num_tokens, p->hidden,
                                       p->top_k, stream));
    return MOE_OK;
}

moe_status moe_forward_few(const moe_problem* p, const void* x_bf16, const void* w_router_bf16, const float* sel_bias,
                           const moe_expert_weights* weights, void* y, int32_t out_dtype, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
    MOE_CHECK(check_problem(p));
    if (!few_supported(*p)) return MOE_ERR_UNSUPPORTED;
    MOE_CHECK(check_weights(weights));
    if (!dtype_ok(out_dtype) || !all_aligned(x_bf16, w_router_bf16, y)) return MOE_ERR_INVALID_ARGUMENT;
    if (!opt_aligned(sel_bias)) return MOE_ERR_INVALID_ARGUMENT;
    MOE_CHECK(check_block_ws(*p, ws, ws_bytes));
    if (p->num_tokens == 0) return MOE_OK;
    return run_few(*p, x_bf16, nullptr, nullptr, w_router_bf16, sel_bias, *weights, y, out_dtype == MOE_OUT_BF16, ws,
                   stream);
}

moe_status moe_block_forward(const moe_problem* p, const void* w_pre, const void* w_router_bf16, const float* sel_bias,
                             const moe_expert_weights* weights, const moe_block_tail* tail, void* ws, size_t ws_bytes,
                             hipStream_t stream) {
    MOE_CHECK(check_block_problem(p));
    MOE_CHECK(check_weights(weights));
    if (!all_aligned(w_router_bf16) || !opt_aligned(w_pre) || !opt_aligned(sel_bias)) return MOE_ERR_INVALID_ARGUMENT;
    if (!tail || !dtype_ok(tail->param_dtype)) return MOE_ERR_INVALID_ARGUMENT;
    const size_t H = (size_t)p->hidden, E = (size_t)p->num_experts;
    MOE_CHECK(check_block_ws(*p, ws, ws_bytes));
    const Span in[4] = {{w_pre, H * dtype_size(tail->param_dtype)}, {w_router_bf16, E * H * 2}, {sel_bias, E * 4},
                        {ws, block_layout(*p).total}};
    MOE_CHECK(check_tail(*p, tail, in));
    if (p->num_tokens == 0) return MOE_OK;
    const BlockLayout L = block_layout(*p);
    uint16_t* n = at<uint16_t>(ws, L.n);
    if (few_supported(*p))
        return run_few(*p, nullptr, w_pre, tail, w_router_bf16, sel_bias, *weights, at<float>(ws, L.y), false, ws,
                       stream);
    MOE_LAUNCH(launch_block_norm(tail->r, tail->res_dtype == MOE_OUT_BF16, w_pre, tail->param_dtype == MOE_OUT_BF16,
                                 tail->eps, n, p->num_tokens, p->hidden, stream));
    ExpertRows rows;
    MOE_CHECK(forward_rows(p, n, w_router_bf16, sel_bias, weights, ws, &rows, stream));
    MOE_LAUNCH(launch_combine_residual(rows.y_perm, rows.row_of_slot, rows.w, tail_args(*tail), p->num_tokens, p->hidden,
                                       p->top_k, stream));
    return MOE_OK;
}

}  // extern "C"
