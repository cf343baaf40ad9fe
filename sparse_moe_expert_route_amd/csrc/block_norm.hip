// The norms before and after the layer, with the gate and the residual sum.
//
//   norm      n  = bf16(RMSNorm(r; w))
//   residual  z  = RMSNorm(y; w_post) or y,  r' = r + scale * gate * z,
//             n' = bf16(RMSNorm(r'; w_next)) if asked for
//   combine   the residual on y = sum_j w_j y_perm[row_j], never stored
//
// RMSNorm(v; w) = v w / sqrt(sum v^2 / H + eps).  All of it in float32: the
// sum of squares is a float32 sum of at most 64 squares per lane, then a tree
// over the lanes and waves.  r' is rounded once to its type, and n' is taken
// from the rounded r' (what a later norm of the stored stream would give).
//
// One workgroup per row; the row stays in registers between its reads, its
// reduction(s) and its stores, so every byte moves once: the kernels are bound
// by HBM (long batches) or by the launch (decode batches).
#include "block_launch.h"
#include "block_rows.h"
#include "moe_internal.h"

namespace moe {

namespace {

enum Source { kFromR = 0, kFromY = 1, kFromRows = 2 };

struct NormArgs {
    const void* y;               // kFromR: r itself; kFromY: the layer output; kFromRows: y_perm
    int y_bf16;
    const int32_t* row_of_slot;  // kFromRows
    const float* w;              // kFromRows: combine weights
    int k;
    int rows;                    // kFromRows: rows of y_perm (T k)
    const void* w_pre;           // kFromR
    uint16_t* n;                 // kFromR
    TailArgs t;
    int H;
};

template <int NT>
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < NT / 64; ++q) s += red[q];
    return s;
}

template <int SRC, int NT, int V>
__global__ void __launch_bounds__(NT) block_norm_kernel(NormArgs a) {
    __shared__ float red[2][NT / 64];
    const size_t row = (size_t)blockIdx.x * a.H;
    float v[V][8];
    // ---- the row: r, y, or the weighted sum of its slots' rows ----
    if constexpr (SRC == kFromRows) {
        const size_t s0 = (size_t)blockIdx.x * a.k;
        int rows[8];
        float ws[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            rows[j] = j < a.k ? a.row_of_slot[s0 + j] : -1;
            ws[j] = j < a.k ? a.w[s0 + j] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int c = (u * NT + threadIdx.x) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
            if (c < a.H) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    // a slot without a row adds nothing and is not read
                    if ((unsigned)rows[j] < (unsigned)a.rows) {
                        float p[8];
                        load8<true>(a.y, 0, (size_t)rows[j] * a.H + c, p);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[u][i] = fmaf(ws[j], p[i], v[u][i]);
                    }
                }
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int c = (u * NT + threadIdx.x) * 8;
            if (c < a.H) {
                load8<true>(a.y, a.y_bf16, row + c, v[u]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
            }
        }
    }
    const bool norm = SRC == kFromR || a.t.post_norm;
    float rstd = 1.0f;
    if (norm) {
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(v[u][i], v[u][i], s);
        rstd = inv_rms(block_sum<NT>(s, red[0]), a.H, a.t.eps);
    }
    const void* wn = SRC == kFromR ? a.w_pre : a.t.w_post;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int c = (u * NT + threadIdx.x) * 8;
        if (c >= a.H) continue;
        if (norm) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] *= rstd;
            if (wn) {
                float w[8];
                load8<false>(wn, a.t.param_bf16, c, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= w[i];
            }
        }
        if constexpr (SRC == kFromR) {
            __builtin_nontemporal_store(pack8(v[u]), (v4u*)(a.n + row + c));
        } else {
            if (a.t.gate) {
                float g[8];
                load8<false>(a.t.gate, a.t.param_bf16, (a.t.gate_per_token ? row : 0) + c, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= g[i];
            }
            float r[8];
            load8<true>(a.t.r, a.t.res_bf16, row + c, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = fmaf(a.t.scale, v[u][i], r[i]);
            if (a.t.res_bf16) {
                const v4u o = pack8(v[u]);
                __builtin_nontemporal_store(o, (v4u*)((uint16_t*)a.t.r_out + row + c));
                unpack8(o, v[u]);   // n' is the norm of r' as stored
            } else {
                v4f* o = (v4f*)((float*)a.t.r_out + row + c);
                __builtin_nontemporal_store(v4f{v[u][0], v[u][1], v[u][2], v[u][3]}, o);
                __builtin_nontemporal_store(v4f{v[u][4], v[u][5], v[u][6], v[u][7]}, o + 1);
            }
        }
    }
    if constexpr (SRC != kFromR) {
        if (!a.t.n_next) return;
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(v[u][i], v[u][i], s);   // channels past H hold zeros
        rstd = inv_rms(block_sum<NT>(s, red[1]), a.H, a.t.eps);
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int c = (u * NT + threadIdx.x) * 8;
            if (c >= a.H) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] *= rstd;
            if (a.t.w_next) {
                float w[8];
                load8<false>(a.t.w_next, a.t.param_bf16, c, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= w[i];
            }
            __builtin_nontemporal_store(pack8(v[u]), (v4u*)((uint16_t*)a.t.n_next + row + c));
        }
    }
}

template <int SRC>
hipError_t launch_rows(const NormArgs& a, int64_t T, hipStream_t stream) {
    const dim3 grid((unsigned)T);
    const int n = (a.H + 2047) / 2048;   // vectors of 8 per thread at 256 threads
    if (n <= 1) hipLaunchKernelGGL((block_norm_kernel<SRC, 256, 1>), grid, dim3(256), 0, stream, a);
    else if (n <= 2) hipLaunchKernelGGL((block_norm_kernel<SRC, 256, 2>), grid, dim3(256), 0, stream, a);
    else if (n <= 4) hipLaunchKernelGGL((block_norm_kernel<SRC, 256, 4>), grid, dim3(256), 0, stream, a);
    else if (n <= 8) hipLaunchKernelGGL((block_norm_kernel<SRC, 256, 8>), grid, dim3(256), 0, stream, a);
    else return hipErrorInvalidValue;
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const void* r, int res_bf16, const void* w, int param_bf16, float eps, uint16_t* n,
                             int64_t T, int H, hipStream_t stream) {
    NormArgs a{};
    a.y = r; a.y_bf16 = res_bf16; a.w_pre = w; a.n = n; a.H = H;
    a.t.param_bf16 = param_bf16; a.t.eps = eps;
    return launch_rows<kFromR>(a, T, stream);
}

hipError_t launch_block_residual(const void* y, int y_bf16, const TailArgs& t, int64_t T, int H, hipStream_t stream) {
    NormArgs a{};
    a.y = y; a.y_bf16 = y_bf16; a.t = t; a.H = H;
    return launch_rows<kFromY>(a, T, stream);
}

hipError_t launch_combine_residual(const float* y_perm, const int32_t* row_of_slot, const float* w, const TailArgs& t,
                                   int64_t T, int H, int k, hipStream_t stream) {
    NormArgs a{};
    a.y = y_perm; a.row_of_slot = row_of_slot; a.w = w; a.k = k; a.rows = (int)(T * k); a.t = t; a.H = H;
    return launch_rows<kFromRows>(a, T, stream);
}

}  // namespace moe
