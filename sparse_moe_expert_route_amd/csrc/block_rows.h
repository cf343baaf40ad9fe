// Rows of the residual stream, of the layer's output and of the norm
// parameters: loads and stores of 8 channels, bf16 or float32, and the root mean
// square.  Shared by the norm kernels and the block for few tokens.
#pragma once

#include "moe_internal.h"

namespace moe {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// 8 consecutive channels at element offset i of a bf16 or float32 array
__device__ __forceinline__ void unpack8(const v4u raw, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = bf16_bits_to_float(raw[q] & 0xFFFFu);
        v[2 * q + 1] = bf16_bits_to_float(raw[q] >> 16);
    }
}
template <bool NT>
__device__ __forceinline__ void load8(const void* p, int bf16, size_t i, float (&v)[8]) {
    if (bf16) {
        const v4u* q = (const v4u*)((const uint16_t*)p + i);
        unpack8(NT ? __builtin_nontemporal_load(q) : *q, v);
    } else {
        const v4f* q = (const v4f*)((const float*)p + i);
        const v4f a = NT ? __builtin_nontemporal_load(q) : q[0];
        const v4f b = NT ? __builtin_nontemporal_load(q + 1) : q[1];
#pragma unroll
        for (int u = 0; u < 4; ++u) { v[u] = a[u]; v[4 + u] = b[u]; }
    }
}
__device__ __forceinline__ v4u pack8(const float (&v)[8]) {
    v4u o;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        o[q] = (uint32_t)float_to_bf16_rne(v[2 * q]) | ((uint32_t)float_to_bf16_rne(v[2 * q + 1]) << 16);
    return o;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// 1 / sqrt(sum / H + eps): a correctly rounded quotient of a correctly rounded
// root (the hardware's reciprocal root is an ulp less exact; once per row, the
// division costs nothing that shows)
__device__ __forceinline__ float inv_rms(float sum, int H, float eps) { return 1.0f / sqrtf(sum / (float)H + eps); }

}  // namespace moe
