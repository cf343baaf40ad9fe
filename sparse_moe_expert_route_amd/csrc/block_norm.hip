// The norms before and after the layer, with the gate and the residual sum.
//
//   norm      n  = bf16(RMSNorm(r; w))
//   residual  z  = RMSNorm(y; w_post) or y,  r' = r + scale * gate * z,
//             n' = bf16(RMSNorm(r'; w_next)) if asked for
//   combine   the residual on y = sum_j w_j y_perm[row_j], never stored
//
// RMSNorm(v; w) = v w / sqrt(sum v^2 / H + eps).  All of it in float32: the
// sum of squares is a float32 sum of at most 16 squares per lane, then a tree
// over the lanes and a sum over the waves.  r' is rounded once to its type, and n' is taken
// from the rounded r' (what a later norm of the stored stream would give).
//
// One workgroup per row; the row and all it is combined with stay in registers
// between their reads, the reduction(s) and the stores, so every byte moves once:
// the kernels are bound by HBM (long batches) or by the launch (decode batches).
// Stores go past the caches, and so do the loads where the expert rows, read
// once, are most of the traffic; rows of r and y are read through them (norm of
// 16384 x 6144 float32: 101 us, 113 past the caches; combine of 8192 x 8 rows of
// 4096: 232 us, 239 with r through the caches).
//
// Measured: norm of 16384 x 6144 float32 101 us (6.0 TB/s), residual of 8191 x
// 4096 float32 with the next norm 73 us (5.5 TB/s), combine of 8192 x 8 rows of
// 4096 into a bf16 stream 232 us (5.5 TB/s); a copy of 4 GiB runs at 4.7 TB/s.
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
    int64_t T;
    int H;
};

// a launch has fewer than 2^32 threads along x
constexpr int64_t kMaxGrid = 1 << 20;

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
    const void* wn = SRC == kFromR ? a.w_pre : a.t.w_post;
    const bool norm = SRC == kFromR || a.t.post_norm;
    int c[V];
    bool in[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        c[u] = (u * NT + threadIdx.x) * 8;
        in[u] = c[u] < a.H;
    }
    // rows past kMaxGrid run on along y (a loop over rows instead: norm 100 -> 118 us,
    // combine 232 -> 289 us)
    const int64_t t = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (t >= a.T) return;
    const size_t row = (size_t)t * a.H;
    // ---- the row: r, y, or the weighted sum of its slots' rows ----
    float v[V][8];
    if constexpr (SRC == kFromRows) {
        const size_t s0 = (size_t)t * a.k;
        int rows[8];
        float ws[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            rows[j] = __builtin_amdgcn_readfirstlane(j < a.k ? a.row_of_slot[s0 + j] : -1);
            ws[j] = j < a.k ? a.w[s0 + j] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            // every load before the first sum; a slot without a row adds nothing and is not read
            v4f p[8][2];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j][0] = p[j][1] = v4f{0.f, 0.f, 0.f, 0.f};
                if ((unsigned)rows[j] < (unsigned)a.rows && in[u]) {
                    const v4f* q = (const v4f*)((const float*)a.y + (size_t)rows[j] * a.H + c[u]);
                    p[j][0] = __builtin_nontemporal_load(q);
                    p[j][1] = __builtin_nontemporal_load(q + 1);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = fmaf(ws[j], p[j][i >> 2][i & 3], v[u][i]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < V; ++u) {
            if (in[u]) {
                load8<false>(a.y, a.y_bf16, row + c[u], v[u]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
            }
        }
    }
    // ---- everything else the row needs, on its way while the row is reduced ----
    float w[V][8], g[V][8], r[V][8], w2[V][8];
#pragma unroll
    for (int u = 0; u < V; ++u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) { w[u][i] = g[u][i] = w2[u][i] = 1.0f; r[u][i] = 0.0f; }
        if (in[u]) {
            if constexpr (SRC != kFromR) load8<SRC == kFromRows>(a.t.r, a.t.res_bf16, row + c[u], r[u]);
            if (norm && wn) load8<false>(wn, a.t.param_bf16, c[u], w[u]);
            if constexpr (SRC != kFromR) {
                if (a.t.gate) load8<false>(a.t.gate, a.t.param_bf16, (a.t.gate_per_token ? row : 0) + c[u], g[u]);
                if (a.t.n_next && a.t.w_next) load8<false>(a.t.w_next, a.t.param_bf16, c[u], w2[u]);
            }
        }
    }
    auto rstd = [&](float* part) {
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(v[u][i], v[u][i], s);   // channels past H hold zeros
        return inv_rms(block_sum<NT>(s, part), a.H, a.t.eps);
    };
    const float post = norm ? rstd(red[0]) : 1.0f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        if (!in[u]) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] *= post * w[u][i];
        if constexpr (SRC == kFromR) {
            __builtin_nontemporal_store(pack8(v[u]), (v4u*)(a.n + row + c[u]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = fmaf(a.t.scale, v[u][i] * g[u][i], r[u][i]);
            if (a.t.res_bf16) {
                const v4u o = pack8(v[u]);
                __builtin_nontemporal_store(o, (v4u*)((uint16_t*)a.t.r_out + row + c[u]));
                unpack8(o, v[u]);   // n' is the norm of r' as stored
            } else {
                v4f* o = (v4f*)((float*)a.t.r_out + row + c[u]);
                __builtin_nontemporal_store(v4f{v[u][0], v[u][1], v[u][2], v[u][3]}, o);
                __builtin_nontemporal_store(v4f{v[u][4], v[u][5], v[u][6], v[u][7]}, o + 1);
            }
        }
    }
    if constexpr (SRC != kFromR) {
        if (!a.t.n_next) return;
        const float next = rstd(red[1]);
#pragma unroll
        for (int u = 0; u < V; ++u) {
            if (!in[u]) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] *= next * w2[u][i];
            __builtin_nontemporal_store(pack8(v[u]), (v4u*)((uint16_t*)a.t.n_next + row + c[u]));
        }
    }
}

template <int SRC>
hipError_t launch_rows(NormArgs a, int64_t T, hipStream_t stream) {
    a.T = T;
    const dim3 grid((unsigned)(T < kMaxGrid ? T : kMaxGrid), (unsigned)((T + kMaxGrid - 1) / kMaxGrid));
    // as many threads as the row has pieces of 8 channels: the residual of 8191 x
    // 4096 takes 75 us with 512 threads and 78 with 256 (two pieces each)
    if (a.H <= 2048) hipLaunchKernelGGL((block_norm_kernel<SRC, 256, 1>), grid, dim3(256), 0, stream, a);
    else if (a.H <= 4096) hipLaunchKernelGGL((block_norm_kernel<SRC, 512, 1>), grid, dim3(512), 0, stream, a);
    else if (a.H <= 8192) hipLaunchKernelGGL((block_norm_kernel<SRC, 1024, 1>), grid, dim3(1024), 0, stream, a);
    else hipLaunchKernelGGL((block_norm_kernel<SRC, 1024, 2>), grid, dim3(1024), 0, stream, a);
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
