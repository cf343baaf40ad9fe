// The layer for few tokens: the route kernel (router logits, the FP8 copy of x,
// cleared counters) and the launch of it and the layer kernel (few_layer.h).
#include "block_launch.h"
#include "block_rows.h"
#include "fp8_rows.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kRouteWaves = 8;   // waves per workgroup

// ---------------------------------------------------------------------------
// Route kernel.  Workgroups of 8 waves:
//   [0, gx kFewParts)   router logits of 16 experts x 16 tokens over a quarter of
//                       K on the bf16 MFMA, the 8 waves splitting it again (H =
//                       4096: 4 steps each, all loads of a wave in flight at
//                       once), summed through LDS in wave order.  The quarters
//                       are summed, in order, by the layer kernel.  (Whole
//                       rows in 16 or 24 workgroups waited on the few CUs'
//                       own load paths: 17 us for 16 tokens of the Pro layer.)
//   the next T          the FP8 copy of one token row;
//   the last            the counters and error words of the layer kernel, cleared.
// SRC: what the rows are made of: 0 the layer's input x (bf16); 1, 2 the
// residual stream (bf16, float32), normalised here: every workgroup that needs
// rows takes their sums of squares itself (they are a few 8 to 24 KB rows in the
// L2), which spares the block its own norm launch.
// ---------------------------------------------------------------------------
enum RowSource { kRowsX = 0, kRowsBf16 = 1, kRowsF32 = 2 };

// 8 channels at c of row t of the layer's input
template <int SRC>
__device__ __forceinline__ v8bf input8(const FewArgs& a, int t, int c, float rstd) {
    const size_t o = (size_t)t * a.H + c;
    if constexpr (SRC == kRowsX) {
        return *(const v8bf*)(a.x + o);
    } else {
        float v[8];
        load8<false>(a.r, SRC == kRowsBf16, o, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= rstd;
        if (a.w_pre) {
            float w[8];
            load8<false>(a.w_pre, a.tail.param_bf16, c, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= w[i];
        }
        return __builtin_bit_cast(v8bf, pack8(v));
    }
}

// sum of squares of row t over a wave
template <int SRC>
__device__ __forceinline__ float row_squares(const FewArgs& a, int t, int first, int step) {
    float s = 0.0f;
#pragma unroll 4
    for (int c = first * 8; c < a.H; c += step * 8) {
        float v[8];
        load8<false>(a.r, SRC == kRowsBf16, (size_t)t * a.H + c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
    }
    return wave_sum(s);
}

template <bool F32S, int SRC>
__global__ void __launch_bounds__(64 * kRouteWaves) few_route_kernel(FewArgs a) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int gx = (a.E + 15) / 16 * kFewParts;
    const int b = blockIdx.x;
    if (b >= gx + a.T) {
        for (int i = tid; i < a.n_counters; i += 64 * kRouteWaves) a.counters[i] = 0u;
        if (tid < 2) a.err[tid] = 0u;
        return;
    }
    __shared__ float squares[kFewMaxT];
    __shared__ v4f red[kRouteWaves][64];
    if (b >= gx) {
        const int t = b - gx;
        float rstd = 1.0f;
        if constexpr (SRC != kRowsX) {
            const float s = row_squares<SRC>(a, t, tid, 64 * kRouteWaves);
            if (lane == 0) squares[wave] = s;
            __syncthreads();
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < kRouteWaves; ++q) v += squares[q];
            rstd = inv_rms(v, a.H, a.tail.eps);
        }
        quantise_channels<F32S, 64 * kRouteWaves, true>([&](int c) { return __builtin_bit_cast(uint4, input8<SRC>(a, t, c, rstd)); },
                                                       a.xq, a.xs, t, a.H);
        return;
    }
    const int g = lane >> 4, r = lane & 15, e0 = b / kFewParts * 16;
    const int t = min(r, a.T - 1);
    const uint16_t* wp = a.w_router + (size_t)min(e0 + r, a.E - 1) * a.H + 8 * g;
    const int ns = a.H / 32, q = b % kFewParts * kRouteWaves + wave;
    const int s0 = q * ns / (kFewParts * kRouteWaves), s1 = (q + 1) * ns / (kFewParts * kRouteWaves);
    float rstd = 1.0f;
    if constexpr (SRC != kRowsX) {
        for (int u = wave; u < a.T; u += kRouteWaves) {
            const float s = row_squares<SRC>(a, u, lane, 64);
            if (lane == 0) squares[u] = s;
        }
        __syncthreads();
        rstd = inv_rms(squares[t], a.H, a.tail.eps);
    }
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    constexpr int U = 6;
    for (int s = s0; s < s1; s += U) {   // past the end: the last step again, left out
        v8bf wa[U], xb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            wa[u] = *(const v8bf*)(wp + 32 * min(s + u, s1 - 1));
            xb[u] = input8<SRC>(a, t, 32 * min(s + u, s1 - 1) + 8 * g, rstd);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s + u < s1) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa[u], xb[u], acc, 0, 0, 0);
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (tid < 256) {
        // component i of lane l: expert e0 + 4 (l / 16) + i, token l mod 16
        const int l = tid >> 2, i = tid & 3;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kRouteWaves; ++w) v += red[w][l][i];
        const int e = e0 + 4 * (l >> 4) + i, tt = l & 15;
        if (e < a.E && tt < a.T) a.logits[((size_t)(b % kFewParts) * a.T + tt) * a.E + e] = v;
    }
}

template <bool F32S>
hipError_t launch_route(const FewArgs& a, hipStream_t stream) {
    const dim3 grid((a.E + 15) / 16 * kFewParts + a.T + 1), block(64 * kRouteWaves);
    if (!a.r) hipLaunchKernelGGL((few_route_kernel<F32S, kRowsX>), grid, block, 0, stream, a);
    else if (a.tail.res_bf16) hipLaunchKernelGGL((few_route_kernel<F32S, kRowsBf16>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((few_route_kernel<F32S, kRowsF32>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few_layer(const FewArgs& a, int packed, int fp8_block, hipStream_t stream) {
    if (a.T < 1 || a.T > kFewMaxT || a.T * (a.H + 16) > kFewRowBytes || a.n_counters < few_counters(a.H))
        return hipErrorInvalidValue;
    if (a.fuse_tail && a.H > kFewTailMaxH) return hipErrorInvalidValue;   // the tail's registers
    const hipError_t st = fp8_block ? launch_route<true>(a, stream) : launch_route<false>(a, stream);
    if (st != hipSuccess) return st;
    return fp8_block ? launch_few_layer_fp8(a, packed, stream) : launch_few_layer_mxfp4(a, packed, stream);
}

}  // namespace moe
