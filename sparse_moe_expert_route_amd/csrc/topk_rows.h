// Top-k selection and combine weights of N tokens by one wave, shared by the
// router's top-k kernel and the layer for few tokens.
//
// key = fp32(L + b), mapped to an unsigned integer that orders like the float
// (after -0 -> +0).  k rounds: each lane's largest key (equal ones: the lowest of
// its experts), the wave's largest of those by DPP, and the lane that holds it; a
// second maximum, over ~id, only where several lanes do, so that equal keys go to
// the lowest expert id.  The winner retires its key.
// Weights: softmax over the k selected *unbiased* logits, max-subtracted.
// Several tokens share the rounds, whose dependent steps then overlap.
#pragma once

#include "moe_internal.h"

namespace moe {

__device__ __forceinline__ uint32_t ordered_key(float f) {
    if (f == 0.0f) f = 0.0f;   // -0 == +0
    uint32_t u = __float_as_uint(f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Largest value over the wave, returned wave-uniform: DPP shifts by 1, 2, 4
// and 8 lanes leave each 16-lane row's maximum in its lane 15, two row
// broadcasts (row 0 into row 1 and row 2 into row 3, then lane 31 into rows 2
// and 3) carry the maxima to lane 63, and a readlane returns it.  DPP moves
// stay in the VALU; a shuffle goes through LDS and costs far more latency.
__device__ __forceinline__ uint32_t dpp_max_step(uint32_t v, uint32_t t) { return t > v ? t : v; }
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = dpp_max_step(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x111, 0xf, 0xf, false));   // row_shr:1
    v = dpp_max_step(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x112, 0xf, 0xf, false));   // row_shr:2
    v = dpp_max_step(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x114, 0xf, 0xf, false));   // row_shr:4
    v = dpp_max_step(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x118, 0xf, 0xf, false));   // row_shr:8
    v = dpp_max_step(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x142, 0xa, 0xf, false));   // row_bcast:15
    v = dpp_max_step(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x143, 0xc, 0xf, false));   // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// The same pattern for a float maximum and a float sum (lanes without a DPP
// source add 0).
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_f(float old, float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, ROW_MASK, 0xf, false));
}
__device__ __forceinline__ float wave_max_f32(float v) {
    v = fmaxf(v, dpp_f<0x111, 0xf>(v, v));
    v = fmaxf(v, dpp_f<0x112, 0xf>(v, v));
    v = fmaxf(v, dpp_f<0x114, 0xf>(v, v));
    v = fmaxf(v, dpp_f<0x118, 0xf>(v, v));
    v = fmaxf(v, dpp_f<0x142, 0xa>(v, v));
    v = fmaxf(v, dpp_f<0x143, 0xc>(v, v));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_sum_f32(float v) {
    v += dpp_f<0x111, 0xf>(0.0f, v);
    v += dpp_f<0x112, 0xf>(0.0f, v);
    v += dpp_f<0x114, 0xf>(0.0f, v);
    v += dpp_f<0x118, 0xf>(0.0f, v);
    v += dpp_f<0x142, 0xa>(0.0f, v);
    v += dpp_f<0x143, 0xc>(0.0f, v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// SIG: sigmoid scoring (teardown "How Big Is Each Expert?": sigmoid expert
// scores and a per-expert load-balancing bias): key = fp32(sigmoid(L) + b),
// weights = sigmoid of the selected logits over their sum.  Otherwise softmax
// scoring as above.
// L[n]: token n's E logits, E <= 64 EJ, each the sum of PARTS values `stride`
// apart.  Lane j < k returns the j-th selected expert and its weight.
// mid() runs once the logits have arrived (a memory access issued there is not
// waited for by the loads' own waits).
template <int EJ, int N, int PARTS, bool SIG, typename Mid>
__device__ __forceinline__ void topk_rows(const float* const (&L)[N], size_t stride, const float* __restrict__ bias, int E,
                                          int k, int (&id)[N], float (&w)[N], Mid mid) {
    const int lane = threadIdx.x & 63;
    float lv[N][EJ];
    uint32_t key[N][EJ];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < EJ; ++j) {
            const float* p = L[n] + min(lane + 64 * j, E - 1);
            lv[n][j] = p[0];
#pragma unroll
            for (int q = 1; q < PARTS; ++q) lv[n][j] += p[q * stride];
        }
    float bv[EJ];
    if (bias) {
#pragma unroll
        for (int j = 0; j < EJ; ++j) bv[j] = bias[min(lane + 64 * j, E - 1)];
    }
#pragma unroll
    for (int j = 0; j < EJ; ++j) {
        const int e = lane + 64 * j;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float l = lv[n][j];
            // the score replaces the logit: sigmoid evaluated in float64 and
            // rounded once to float32, so that two implementations of it agree
            // on the float32 score (and with it on the selection) unless the
            // float64 value lies within an ulp or two of a float32 midpoint
            if constexpr (SIG) l = (float)(1.0 / (1.0 + exp(-(double)l)));
            lv[n][j] = l;
            // 0 is a retired key or no expert
            key[n][j] = e < E ? max(ordered_key(bias ? l + bv[j] : l), 1u) : 0u;
        }
    }

    mid();

    float sel[N];   // lane j (< k) keeps the j-th selected logit
#pragma unroll
    for (int n = 0; n < N; ++n) { sel[n] = 0.0f; id[n] = 0; }
    for (int r = 0; r < k; ++r) {
        uint32_t best[N], top[N];
        int at[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            best[n] = key[n][0];
            at[n] = 0;
#pragma unroll
            for (int j = 1; j < EJ; ++j) {
                const bool more = key[n][j] > best[n];
                best[n] = more ? key[n][j] : best[n];
                at[n] = more ? j : at[n];
            }
        }
#pragma unroll
        for (int n = 0; n < N; ++n) top[n] = wave_max_u32(best[n]);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const unsigned long long holds = __ballot(best[n] == top[n]);
            int owner = __builtin_ctzll(holds);
            if (holds & (holds - 1))
                owner = (int)(~wave_max_u32(best[n] == top[n] ? ~(uint32_t)(64 * at[n] + lane) : 0u) & 63u);
            const int j0 = __builtin_amdgcn_readlane(at[n], owner);
            float l = lv[n][0];
#pragma unroll
            for (int j = 1; j < EJ; ++j) l = j == j0 ? lv[n][j] : l;
            l = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(l), owner));
            const int e = 64 * j0 + owner;
#pragma unroll
            for (int j = 0; j < EJ; ++j) key[n][j] = e == lane + 64 * j ? 0u : key[n][j];
            if (lane == r) { sel[n] = l; id[n] = e; }
        }
    }

    // softmax over the k selected logits held by lanes 0..k-1, or the
    // selected sigmoid scores over their sum
#pragma unroll
    for (int n = 0; n < N; ++n) {
        float z;
        if constexpr (SIG) {
            z = lane < k ? sel[n] : 0.0f;
        } else {
            const float m = wave_max_f32(lane < k ? sel[n] : -__builtin_inff());
            z = lane < k ? expf(sel[n] - m) : 0.0f;
        }
        w[n] = z / wave_sum_f32(z);
    }
}

}  // namespace moe
