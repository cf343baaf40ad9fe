// Host-only stand-ins of the kernel launchers behind include/moe_block.h, beside
// those of abi_host_stubs.cpp: the sanitizer build of abi_block.cpp links them
// (tests/test_block_sanitize.py).  Test infrastructure: each checks the arguments
// the host code hands over, counts the call and touches no memory.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "block_launch.h"

namespace {

struct Calls {
    int norm, residual, combine, few, few_tail;
} g_calls;

void need(bool ok, const char* fn, const char* what) {
    if (!ok) {
        std::fprintf(stderr, "stub %s: %s\n", fn, what);
        std::abort();
    }
}

void check_tail(const char* fn, const moe::TailArgs& t) {
    need(t.r && t.r_out, fn, "tail pointers");
    need(t.eps > 0.0f, fn, "eps");
}

bool inside(const void* p, size_t n, const void* lo, const void* hi) {
    return (const char*)p >= (const char*)lo && (const char*)p + n <= (const char*)hi;
}

}  // namespace

extern "C" int moe_block_stub_calls(const char* name) {
    if (!std::strcmp(name, "norm")) return g_calls.norm;
    if (!std::strcmp(name, "residual")) return g_calls.residual;
    if (!std::strcmp(name, "combine")) return g_calls.combine;
    if (!std::strcmp(name, "few")) return g_calls.few;
    if (!std::strcmp(name, "few_tail")) return g_calls.few_tail;
    return -1;
}

namespace moe {

hipError_t launch_block_norm(const void* r, int, const void*, int, float eps, uint16_t* n, int64_t T, int H, hipStream_t) {
    need(r && n && T >= 1 && H >= 128 && H <= 16384 && eps > 0.0f, "launch_block_norm", "arguments");
    ++g_calls.norm;
    return hipSuccess;
}

hipError_t launch_block_residual(const void* y, int, const TailArgs& t, int64_t T, int H, hipStream_t) {
    need(y && T >= 1 && H >= 128 && H <= 16384, "launch_block_residual", "arguments");
    check_tail("launch_block_residual", t);
    ++g_calls.residual;
    return hipSuccess;
}

hipError_t launch_combine_residual(const float* yp, const int32_t* ros, const float* w, const TailArgs& t, int64_t T, int H,
                                   int k, hipStream_t) {
    need(yp && ros && w && T >= 1 && H >= 128 && H <= 16384 && k >= 1 && k <= 8, "launch_combine_residual", "arguments");
    check_tail("launch_combine_residual", t);
    ++g_calls.combine;
    return hipSuccess;
}

hipError_t launch_few_layer(const FewArgs& a, int, int fp8_block, hipStream_t) {
    const char* fn = "launch_few_layer";
    need((a.x != nullptr) != (a.r != nullptr), fn, "one source of rows");
    need(a.w_router && a.w13 && a.w13_scale && a.w2 && a.w2_scale && a.y, fn, "null pointer");
    need(a.T >= 1 && a.T <= kFewMaxT && a.T * (a.H + 16) <= kFewRowBytes && a.E <= 512 && a.k <= 8, fn, "sizes");
    need(a.n_counters == few_counters(a.H), fn, "counters");
    // every intermediate in the workspace, in order and without overlap
    const size_t T = a.T, H = a.H, I = a.I, N = T * a.k, sb = 4;
    (void)fp8_block;
    need(inside(a.counters, (size_t)a.n_counters * 4, a.counters, a.logits), fn, "counters past their place");
    need(inside(a.logits, kFewParts * T * a.E * 4, a.logits, a.xq), fn, "logits past their place");
    need(inside(a.xq, T * H, a.xq, a.xs), fn, "xq past its place");
    need(inside(a.xs, T * (H / 128) * sb, a.xs, a.hq), fn, "xs past its place");
    need(inside(a.hq, N * I, a.hq, a.hs), fn, "hq past its place");
    need(inside(a.hs, N * (I / 128) * sb, a.hs, a.y_slot), fn, "hs past its place");
    need(inside(a.y_slot, N * H * 4, a.y_slot, a.part), fn, "y_slot past its place");
    need((uintptr_t)a.part % 256 == 0, fn, "alignment");
    if (a.fuse_tail) {
        need(a.H <= kFewTailMaxH, fn, "tail");
        check_tail(fn, a.tail);
        ++g_calls.few_tail;
    }
    ++g_calls.few;
    return hipSuccess;
}

}  // namespace moe
