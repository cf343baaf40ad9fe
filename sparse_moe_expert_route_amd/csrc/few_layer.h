// The whole layer for at most 16 tokens, in two kernels.
//
//   few_route_kernel   router logits, the FP8 copy of x, cleared counters
//   few_layer_kernel   top-k, gate/up + SwiGLU + FP8 of h, down, weighted sum
//
// With T <= 16 tokens an expert has at most 16 rows: one MFMA tile of tokens
// per expert, and every weight byte of every touched expert is read once.  The
// layer is then bound by HBM (8 experts of 13.4 MB for one token, over a
// hundred for 16) and, for the fewest tokens, by the waits between its steps.
// Separate launches for the gate/up GEMM, the down GEMM and the sum each drain
// the memory pipeline; here one launch holds all of it, so the reads of W2
// start while the last of W13 is still being multiplied.
//
// Work split: a wave is on its own.  It draws items in order: first the gate/up
// items (16 features of one expert: 16 gate and 16 up rows), then the down items
// (32 output features of one expert).  A workgroup takes 8 items at a time from
// one counter in memory and hands them to its waves through LDS (one counter
// for every wave of the chip would be drawn tens of thousands of times, and
// atomics on one address leave memory one after the other).  What an item needs
// from others is counted:
//   - the 8 gate/up items of a workgroup's run are one 128-channel block of h,
//     kept in LDS; the wave that completes it quantises it and counts it for its
//     expert.  With few blocks, K is cut into S parts, a run each, whose sums go
//     through memory; the workgroup that completes the last part adds them up.
//     (A run's 8 waves then wait for each other; they are the workgroup's 8 waves,
//     each with one item of the run.)
//   - a down item loads its first weights, then waits until its expert's blocks
//     are all counted;
//   - the wave whose down item is the last on its 32 features (one from every
//     touched expert) sums them over the k slots of every token, in slot order.
//     With at most 8 routing slots (one token of a top-8 layer) a run of 8 down
//     items is the same 32 features of every touched expert: its sum needs LDS
//     only, and the rows of h come to LDS in one trip instead of stage by stage;
//   - in the block's form (moe_block_forward) the runs after the last down item
//     are the rows of the residual stream: the workgroup that draws one waits until
//     all of y is summed and does gate, residual sum and norms of that row.
// Which wave does that depends on timing, what it computes does not: results
// have the same bits on every run.
//
// Every wait ends: a running workgroup draws the items in order and its waves
// take them in order, one at a time; gate/up items wait for nothing and have the
// lower numbers.  The lowest unfinished item therefore lies with a running
// workgroup, in a wave that waits for nothing unfinished or next in line for its
// first free wave (whose items, being lower, are finished), whatever part of the
// grid is resident, and also when several of these kernels share the device.  (A
// wait is bounded all the same: past kFewMaxPolls polls, seconds, it gives up and
// sets an error bit.)
//
// Memory order: the XCDs' L2 caches are not coherent with each other, so what
// crosses workgroups (the codes and scales of h, the rows of y) is stored and
// loaded with agent-scope accesses, which do not stay in an L2.  A wave's stores
// are complete (vmcnt 0) before it counts; a reader sees the count before it
// issues its loads.
//
// Measured, both kernels (packed MXFP4 layer of 256 experts, H = 4096, I = 2048;
// reads of one contiguous chunk per workgroup reach 7.0 TB/s): 8 tokens 115 us (770
// MB, 6.7 TB/s); 16 tokens of 384 experts with H = 6144 351 us (2.21 GB, 6.3
// TB/s); one token 36.4 us (109 MB), of which route 4.5, the top-k and the plan 5,
// the reads of W13 13, the last block of h with its sums and counts 7 (the reads of
// W2 run beside it), the down items and the sum 4.  As separate launches: 138, 399
// and 49 us.
#pragma once

#include "block_launch.h"
#include "block_rows.h"
#include "moe_internal.h"
#include "topk_rows.h"

namespace moe {

namespace {

constexpr int kFewWaves = 8;                  // waves per workgroup of the layer kernel
constexpr int kFewPlaces = 4;                 // runs a workgroup can have in work
constexpr int kFewSlots = kFewMaxT * 8;       // routing slots, and so touched experts, at most
constexpr uint32_t kFewMaxPolls = 1u << 23;

// ---- agent-scope accesses and counters ------------------------------------
__device__ __forceinline__ void put8(void* p, uint32_t lo, uint32_t hi) {
    __hip_atomic_store((unsigned long long*)p, (unsigned long long)lo | ((unsigned long long)hi << 32), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put16(void* p, const v4f v) {
    put8(p, __float_as_uint(v[0]), __float_as_uint(v[1]));
    put8((uint8_t*)p + 8, __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint2 get8(const void* p) {
    const unsigned long long v = __hip_atomic_load((const unsigned long long*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return make_uint2((uint32_t)v, (uint32_t)(v >> 32));
}
__device__ __forceinline__ uint4 get16(const void* p) {
    const uint2 a = get8(p), b = get8((const uint8_t*)p + 8);
    return make_uint4(a.x, a.y, b.x, b.y);
}
// all of the wave's earlier memory accesses are complete
__device__ __forceinline__ void wave_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
// adds 1 to a counter; the value before, the same in every lane
__device__ __forceinline__ uint32_t count(uint32_t* c) {
    uint32_t v = 0;
    if ((threadIdx.x & 63) == 0) v = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    v = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
    asm volatile("" ::: "memory");
    return v;
}
// Sums that some lanes use only: the MFMAs before need every lane (the compiler
// may take them for the lanes' own work and move them under the mask of their use,
// where the operands of the other lanes are not computed).
__device__ __forceinline__ void keep_whole(v4f (&acc)[2]) { asm volatile("" : "+v"(acc[0]), "+v"(acc[1])); }

// ---------------------------------------------------------------------------
// One pipeline stage of an item: two 16-row weight tiles and the token rows.
//
// Gate/up is multiplied on the bf16 MFMA (16x16x32), the codes converted in
// registers, which is exact: e2m1 and e4m3 have at most 4 significant bits, and
// the e8m0 scales go into the conversion.  The block-scaled MFMA would take the
// codes as stored, at a fifth of the vector instructions, but its internal sum
// keeps about 13 bits below its largest product, which moves h enough to flip
// some of its FP8 codes (error of y against 64 bits, 16 tokens of the Flash
// layer with MXFP4 experts: 4e-4, with the bf16 MFMA 2e-5).  The conversions stay
// under the memory time (16 tokens of the Pro layer: 350 us either way; one token
// of the Flash layer: 39.6 us against 38.9).  Down, whose result is not rounded to FP8 again, runs on
// the block-scaled MFMA (on the bf16 MFMA the error would be 2e-7, at 369 us and
// 43.6 us).
//
// A dot product may take K in any order as long as both operands do: on the bf16
// MFMA a lane's 32 columns go to 4 instructions, 8 at a time.
//
// MXFP4 packed: 512 of K.  The lane group g = lane / 16 takes the stage's g-th
// 128 columns, the 32 of step j = 0..3 among them: the four scales of a weight row
// over those 128 columns are then one dword of the lane (byte j for step j), and
// the activation scale is one byte per lane and stage.  A last stage shorter than
// 512 reads its last block again and leaves it out.
//
// MXFP4 in the canonical layout: the same 512 of K, but step j takes the j-th 128
// columns, of which the lane group g holds columns 32 g ..: one load then covers
// 64 bytes in a row of each of the 16 weight rows (in the order above it would be
// 64 single 16-byte pieces), and the second load finds its lines on their way.
// The scales are loaded as above, group j holding those of the j-th 128 columns,
// and go to the other groups by a lane permutation.
//
// FP8 block-scaled: 256 of K, two 128-column blocks, whose partial sums gain
// their two float32 scales each.
//
// On the block-scaled MFMA an e2m1 operand's lane holds 32 consecutive columns of
// the instruction's 128, an e4m3 operand's columns 16 g .. and 64 + 16 g ..; the
// rows' pieces are picked so that both agree on the order above.
// ---------------------------------------------------------------------------
// Formats: 0 MXFP4 packed, 1 FP8 block-scaled, 2 MXFP4 canonical.
template <int FMT>
struct FewStageW;
template <int FMT>
struct FewScales;   // of the rows

template <>
struct FewStageW<0> {
    static constexpr int kCols = 512;
    v4u w[2][4];
    uint32_t ws[2];
};
template <>
struct FewScales<0> { uint32_t xs; };
template <>
struct FewStageW<2> : FewStageW<0> {};
template <>
struct FewScales<2> : FewScales<0> {};
template <>
struct FewStageW<1> {
    static constexpr int kCols = 256;
    v4u w[2][2][2];
    float ws[2][2];
};
template <>
struct FewScales<1> { float xs[2]; };
// rows held in registers: 16-byte pieces of MFMA (FP8: block) i
template <int FMT>
struct FewStageX : FewScales<FMT> { uint4 x[FMT == 1 ? 2 : 4][2]; };

// Wave-uniform bases and the lane's 32-bit offsets from them.
struct FewPtrs {
    const uint8_t* w[2];     // the weight tiles
    const uint8_t* ws[2];    // their scales
    const uint8_t* x;        // the token rows
    const uint8_t* xs;       // their scales
    uint32_t wo, wso;        // the lane's place in a tile and in its scales
    uint32_t xo, xso;        // its token row and that row's scales
    int KB;                  // 128-column blocks of K
    int all;                 // stages of K
    int lo, nst, first;      // the item's stages [lo, lo + nst), from lo + first on, wrapping around
    const uint8_t* pad;      // zeros

    // The item's i-th stage; `all` for every i past its end.  Loads past the end go
    // to the pad (one cached line or a few) and add nothing: with them every load
    // is unconditional, and each wait on the in-order load counter covers the
    // stage about to be used and no later one.
    __device__ __forceinline__ int stage(int i) const {
        const int q = i + first;
        return i >= nst ? all : lo + (q >= nst ? q - nst : q);
    }
    template <bool PAD>
    __device__ __forceinline__ const uint8_t* base(const uint8_t* p, int st) const { return !PAD || st < all ? p : pad; }
    template <bool PAD>
    __device__ __forceinline__ uint32_t off(uint32_t o, int st) const { return !PAD || st < all ? o : 0u; }
};

template <int FMT, bool PK>
__device__ __forceinline__ void few_lane_offsets(FewPtrs& P, int K) {
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    constexpr int per = FewStageW<FMT>::kCols / kFp8Block;
    P.KB = K / kFp8Block;
    P.all = P.nst = (P.KB + per - 1) / per;
    P.lo = 0;
    if constexpr (FMT == 0) {
        P.wo = 16 * r;
        P.wso = 4 * r;
    } else if constexpr (FMT == 2) {
        P.wo = r * (K / 2) + 16 * g;
        P.wso = r * (K / 32);
    } else {
        P.wo = PK ? 16 * lane : r * K + 16 * g;
        P.wso = 0;
    }
}
template <int FMT>
__device__ __forceinline__ void few_tile(FewPtrs& P, int i, const uint8_t* w, const uint8_t* ws, size_t row0, int K) {
    P.w[i] = w + row0 * (FMT == 1 ? K : K / 2);
    P.ws[i] = FMT == 1 ? ws + (row0 / 128) * (K / 128) * 4 : ws + row0 * (K / 32);
}

template <bool PK>
__device__ __forceinline__ v4u load_w(const uint8_t* p) {
    // packed: whole lines of weights that are read once go past the caches
    if constexpr (PK) return __builtin_nontemporal_load((const v4u*)p);
    else return *(const v4u*)p;
}

template <int FMT, bool PK, bool PAD>
__device__ __forceinline__ void load_weights(const FewPtrs& P, int st, FewStageW<FMT>& s) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    if constexpr (FMT == 0) {
        const int c = min(4 * st + g, P.KB - 1);
        const uint32_t o = P.off<PAD>(P.wo + 1024 * c, st), os = P.off<PAD>(P.wso + 64 * c, st);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t* w = P.base<PAD>(P.w[i], st);
#pragma unroll
            for (int j = 0; j < 4; ++j) s.w[i][j] = load_w<true>(w + o + 256 * j);
            s.ws[i] = *(const uint32_t*)(P.base<PAD>(P.ws[i], st) + os);
        }
    } else if constexpr (FMT == 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t* w = P.base<PAD>(P.w[i], st);
#pragma unroll
            for (int j = 0; j < 4; ++j) s.w[i][j] = load_w<false>(w + P.off<PAD>(P.wo + 64 * min(4 * st + j, P.KB - 1), st));
        }
        const uint32_t os = P.off<PAD>(P.wso + 4 * min(4 * st + g, P.KB - 1), st);
#pragma unroll
        for (int i = 0; i < 2; ++i) s.ws[i] = *(const uint32_t*)(P.base<PAD>(P.ws[i], st) + os);
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int c = min(2 * st + b, P.KB - 1);
            const uint32_t o = P.off<PAD>(P.wo + (PK ? 2048 : 128) * c, st);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t* w = P.base<PAD>(P.w[i], st);
                s.w[i][b][0] = load_w<PK>(w + o);
                s.w[i][b][1] = load_w<PK>(w + o + (PK ? 1024 : 64));
                s.ws[i][b] = *(const float*)(P.base<PAD>(P.ws[i], st) + (P.wso + P.off<PAD>(4 * c, st)));
            }
        }
    }
}

// SHARED: written by other workgroups of this launch
template <bool SHARED, typename T>
__device__ __forceinline__ T load_xs(const uint8_t* p) {
    if constexpr (SHARED) return __hip_atomic_load((const T*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    else return *(const T*)p;
}

// First column, in a token row, of the lane's h-th 16 columns for step (FP8:
// block) i.  BF: for the bf16 MFMA, where a lane's rows are its weights' columns.
template <int FMT, bool BF>
__device__ __forceinline__ uint32_t row_col(const FewPtrs& P, int st, int i, int h) {
    const int g = (threadIdx.x & 63) >> 4;
    if constexpr (FMT == 1) return 128 * min(2 * st + i, P.KB - 1) + 16 * g + 64 * h;
    else if constexpr (BF) return FMT == 0 ? 128 * min(4 * st + g, P.KB - 1) + 32 * i + 16 * h
                                           : 128 * min(4 * st + i, P.KB - 1) + 32 * g + 16 * h;
    else return FMT == 0 ? 128 * min(4 * st + 2 * h + (g >> 1), P.KB - 1) + 16 * (g & 1) + 32 * i
                         : 128 * min(4 * st + i, P.KB - 1) + 16 * g + 64 * h;
}
template <int FMT, bool SHARED>
__device__ __forceinline__ void load_row_scales(const FewPtrs& P, int st, FewScales<FMT>& s) {
    const uint8_t* xs = P.base<!SHARED>(P.xs, st);
    if constexpr (FMT == 1) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
            s.xs[b] = load_xs<SHARED, float>(xs + P.off<!SHARED>(P.xso + 4 * min(2 * st + b, P.KB - 1), st));
    } else {
        s.xs = load_xs<SHARED, uint8_t>(xs + P.off<!SHARED>(P.xso + min(4 * st + (int)((threadIdx.x & 63) >> 4), P.KB - 1), st));
    }
}
// rows that other workgroups of this launch wrote, with their scales: in memory
struct FewRowsMemory {
    template <int FMT>
    __device__ __forceinline__ void load(const FewPtrs& P, int st, FewStageX<FMT>& s) const {
#pragma unroll
        for (int i = 0; i < (FMT == 1 ? 2 : 4); ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) s.x[i][h] = get16(P.x + (P.xo + row_col<FMT, false>(P, st, i, h)));
        load_row_scales<FMT, true>(P, st, s);
    }
};
// ... or copied to LDS (the lane's row, its scales)
struct FewRowsLds {
    const uint8_t *row, *scales;
    template <int FMT>
    __device__ __forceinline__ void load(const FewPtrs& P, int st, FewStageX<FMT>& s) const {
#pragma unroll
        for (int i = 0; i < (FMT == 1 ? 2 : 4); ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) s.x[i][h] = *(const uint4*)(row + row_col<FMT, false>(P, st, i, h));
        if constexpr (FMT == 1) {
#pragma unroll
            for (int b = 0; b < 2; ++b) s.xs[b] = *(const float*)(scales + 4 * min(2 * st + b, P.KB - 1));
        } else {
            s.xs = scales[min(4 * st + (int)((threadIdx.x & 63) >> 4), P.KB - 1)];
        }
    }
};

// 8 codes -> 8 bf16 times a power of two (exact)
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
__device__ __forceinline__ v8bf join(v2bf a, v2bf b, v2bf c, v2bf d) { return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]}; }
__device__ __forceinline__ v8bf fp8_to_bf16(uint32_t lo, uint32_t hi, float scale) {
    return join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, scale, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, scale, true),
                __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, scale, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, scale, true));
}
__device__ __forceinline__ v8bf fp4_to_bf16(uint32_t v, float scale) {
    return join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1),
                __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3));
}

// Scales of step j of an MXFP4 stage as e8m0 bytes in the low bits; past K both
// are 0 (2^-127, so that products of both are below any float).
template <int FMT>
__device__ __forceinline__ void step_scales(const FewPtrs& P, int st, int j, const FewStageW<FMT>& s, uint32_t rows, uint32_t (&ws)[2],
                                            uint32_t& xs) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const uint32_t keep = 4 * st + (FMT == 0 ? g : j) < P.KB ? 0xFFu : 0u;
    if constexpr (FMT == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) ws[i] = s.ws[i] >> (8 * j) & keep;
        xs = rows & keep;
    } else {
        const int from = 4 * (16 * j + (lane & 15));   // group j's lane of this row
#pragma unroll
        for (int i = 0; i < 2; ++i) ws[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)s.ws[i]) >> (8 * g) & keep;
        xs = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)rows) & keep;
    }
}
__device__ __forceinline__ float e8m0(uint32_t byte) { return __uint_as_float(byte << 23); }

// bf16 MFMA.  rows(i, scale, x): the lane's 32 columns of the rows for step
// (block) i, times the scale where the rows do not hold it yet; rs: the rows'
// scales.
template <int FMT, typename Rows, typename RS>
__device__ __forceinline__ void compute_bf16(const FewPtrs& P, int st, FewStageW<FMT>& s, Rows rows, const RS& rs, v4f (&acc)[2]) {
    v8bf x[4];
    if constexpr (FMT != 1) {
        if (4 * st + 4 > P.KB) {   // codes past K to 0
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t keep = 4 * st + (FMT == 0 ? (int)((threadIdx.x & 63) >> 4) : j) < P.KB ? ~0u : 0u;
#pragma unroll
                for (int i = 0; i < 2; ++i) s.w[i][j] &= keep;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t ws[2], xs;
            step_scales<FMT>(P, st, j, s, rs.xs, ws, xs);
            rows(j, e8m0(xs), x);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp4_to_bf16(s.w[i][j][m], e8m0(ws[i])), x[m], acc[i], 0, 0, 0);
        }
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const bool live = 2 * st + b < P.KB;   // past K: finite codes again, at scale 0
            rows(b, 1.0f, x);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v4f part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const v4u w = s.w[i][b][m / 2];
                    part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(w[2 * (m % 2)], w[2 * (m % 2) + 1], 1.0f), x[m], part, 0, 0, 0);
                }
                const float c = live ? s.ws[i][b] * rs.xs[b] : 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][q] = fmaf(part[q], c, acc[i][q]);
            }
        }
    }
}

// Block-scaled MFMA, the rows in registers.
template <int FMT>
__device__ __forceinline__ void compute_scaled(const FewPtrs& P, int st, const FewStageW<FMT>& s, const FewStageX<FMT>& x, v4f (&acc)[2]) {
    if constexpr (FMT != 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t ws[2], xs;
            step_scales<FMT>(P, st, j, s, x.xs, ws, xs);
            const uint4 lo = x.x[j][0], hi = x.x[j][1];
            const v8i xb = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const v4u w = s.w[i][j];
                const v8i wa = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
                acc[i] = mfma_w4a8<0, 0>(wa, xb, acc[i], (int)ws[i], (int)xs);
            }
        }
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const bool live = 2 * st + b < P.KB;
            const uint4 lo = x.x[b][0], hi = x.x[b][1];
            const v8i xb = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const v4u wl = s.w[i][b][0], wh = s.w[i][b][1];
                const v8i wa = {(int)wl[0], (int)wl[1], (int)wl[2], (int)wl[3], (int)wh[0], (int)wh[1], (int)wh[2], (int)wh[3]};
                // both operands e4m3, scales 2^0
                const v4f part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xb, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, 127);
                const float c = live ? s.ws[i][b] * x.xs[b] : 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][q] = fmaf(part[q], c, acc[i][q]);
            }
        }
    }
}

// Gate/up: acc[i] = tile i . rows over the whole of K, R stages of weights in
// flight; the rows come from their copy in LDS: FP8 codes, or (XB) the bf16 they
// stand for.
template <int FMT, bool PK, bool XB>
__device__ __forceinline__ void few_item(const FewPtrs& P, const uint8_t* row, v4f (&acc)[2]) {
    constexpr int R = 4;
    const int nst = P.nst;
    FewStageW<FMT> w[R];
    FewScales<FMT> xs[R];
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    auto load = [&](int st, int i) {
        load_weights<FMT, PK, true>(P, P.stage(st), w[i]);
        if constexpr (XB && FMT != 1) xs[i].xs = 0;   // in the rows
        else load_row_scales<FMT, false>(P, P.stage(st), xs[i]);
    };
#pragma unroll
    for (int i = 0; i < R; ++i) load(i, i);
    for (int at = 0; at < nst; at += R) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int st = P.stage(at + i);
            auto rows = [&](int j, float scale, v8bf (&x)[4]) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t c = row_col<FMT, true>(P, st, j, h);
                    if constexpr (XB) {
                        x[2 * h] = *(const v8bf*)(row + 2 * c);
                        x[2 * h + 1] = *(const v8bf*)(row + 2 * c + 16);
                    } else {
                        const uint4 v = *(const uint4*)(row + c);
                        x[2 * h] = fp8_to_bf16(v.x, v.y, scale);
                        x[2 * h + 1] = fp8_to_bf16(v.z, v.w, scale);
                    }
                }
            };
            __builtin_amdgcn_sched_barrier(0);
            if (at + i < nst) compute_bf16<FMT>(P, st, w[i], rows, xs[i], acc);
            __builtin_amdgcn_sched_barrier(0);
            load(at + i + R, i);
        }
    }
}

// Down: the first kDownW stages of weights are loaded ahead (before the item in
// front is stored), the rows, which other workgroups wrote, kDownX stages ahead.
// A stage's rows are asked for before the weights of a later one, so that the
// in-order load counter lets the wait for the rows leave those weights out.
// (Loads past the end are branched around here: an item of I <= 2048 has all its
// weights in the first kDownW stages.)
constexpr int kDownW = 4, kDownX = 2;

template <int FMT, bool PK>
__device__ __forceinline__ void down_prefetch(const FewPtrs& P, FewStageW<FMT> (&w)[kDownW]) {
#pragma unroll
    for (int i = 0; i < kDownW; ++i)
        if (i < P.nst) load_weights<FMT, PK, false>(P, P.stage(i), w[i]);
}

template <int FMT, bool PK, typename Rows>
__device__ __forceinline__ void down_item(const FewPtrs& P, const Rows& rows, FewStageW<FMT> (&w)[kDownW], v4f (&acc)[2]) {
    const int nst = P.nst;
    FewStageX<FMT> x[kDownX];
    static_assert(kDownW % kDownX == 0, "the rows' places repeat with the weights'");
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int at, int i) { compute_scaled<FMT>(P, P.stage(at), w[i % kDownW], x[i % kDownX], acc); };
#pragma unroll
    for (int i = 0; i < kDownX; ++i)
        if (i < nst) rows.template load<FMT>(P, P.stage(i), x[i]);
    int st = 0;
    for (; st + 2 * kDownW <= nst; st += kDownW) {
#pragma unroll
        for (int i = 0; i < kDownW; ++i) {
            compute(st + i, i);
            __builtin_amdgcn_sched_barrier(0);
            rows.template load<FMT>(P, P.stage(st + i + kDownX), x[i % kDownX]);
            load_weights<FMT, PK, false>(P, P.stage(st + i + kDownW), w[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // kDownW stages of weights loaded, up to kDownW - 1 more to come
#pragma unroll
    for (int i = 0; i < 2 * kDownW - 1; ++i) {
        if (st + i < nst) compute(st + i, i);
        if (st + i + kDownX < nst) rows.template load<FMT>(P, P.stage(st + i + kDownX), x[i % kDownX]);
        if (i < kDownW - 1 && st + i + kDownW < nst) load_weights<FMT, PK, false>(P, P.stage(st + i + kDownW), w[i]);
    }
}

// What every workgroup derives from the logits.
struct FewPlan {
    uint32_t mask[512];                 // bit t: token t selected expert e
    int16_t index[512];                 // its place among the touched experts
    int16_t expert[kFewSlots];          // touched experts, ascending
    uint8_t slot[kFewSlots][kFewMaxT];  // routing slot of each of their rows (rows by ascending token)
    int16_t ids[kFewSlots];
    float w[kFewSlots];                 // combine weights by slot
    int wave_count[kFewWaves];
    // runs of 8 items drawn by the workgroup, the c-th in place c mod kFewPlaces
    uint32_t drawn;                          // items handed to waves
    uint32_t read[kFewPlaces];               // waves that have their item of the place's runs
    uint32_t finished[kFewPlaces];           // gate/up items whose h is in the place
    uint32_t summed_parts[kFewPlaces];       // gate/up items whose part is in memory
    uint32_t verdict[kFewPlaces];            // 2 x runs counted for their block, + 1 if the last was its last part
    uint32_t freed[kFewPlaces];              // the place's runs that are over
    uint32_t ready[kFewSlots];               // experts whose h is known to be there
    float red[2][kFewWaves];                 // sums of squares of the tail
    uint32_t summed;                         // all of y is known to be there
    uint32_t polling;                        // a wave is asking memory
    unsigned long long run[kFewPlaces];      // (c + 1) << 32 | number of run c
    float h[kFewPlaces][kFewMaxT][kFp8Block + 4];   // h of a gate/up run: rows of 128 channels
};

template <typename T>
__device__ __forceinline__ T lds_load(T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP); }
__device__ __forceinline__ void lds_store(uint32_t* p, uint32_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ uint32_t lds_add(uint32_t* p) {
    return __hip_atomic_fetch_add(p, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ uint32_t next_run(uint32_t* ticket) {
    return __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Waits until poll(), which asks memory, says so; `known`, in LDS, says that a wave
// has seen it.  One wave of the workgroup at a time asks (polls of one address
// leave memory one after the other, and the counts that they wait for queue behind
// them); the others look at LDS.
template <typename Poll>
__device__ __forceinline__ void wait_until(const FewArgs& a, FewPlan& s, uint32_t* known, Poll poll) {
    for (uint32_t i = 0; !lds_load(known); ++i) {
        uint32_t busy = 1;
        if ((threadIdx.x & 63) == 0) busy = __hip_atomic_exchange(&s.polling, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        if (!uniform((int)busy)) {
            const bool there = poll(), over = i >= kFewMaxPolls;
            if (there || over) lds_store(known, 1u);
            if (!there && over) __hip_atomic_store(a.err, kErrStalled, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            lds_store(&s.polling, 0u);
            if (there) break;
        }
        __builtin_amdgcn_s_sleep(8);
    }
    asm volatile("" ::: "memory");
}
// ... until *c >= n
__device__ __forceinline__ void wait_for(const FewArgs& a, FewPlan& s, const uint32_t* c, uint32_t n, uint32_t* known) {
    wait_until(a, s, known, [&] {
        return (uint32_t)uniform((int)__hip_atomic_load(c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) >= n;
    });
}

// The wave's next item, 8 run + its place in the run; `place`: the run's place in LDS.
__device__ __forceinline__ int draw(uint32_t* ticket, FewPlan& s, int& place) {
    uint32_t q = 0;
    if ((threadIdx.x & 63) == 0) q = lds_add(&s.drawn);
    q = (uint32_t)uniform((int)q);
    const uint32_t c = q / kFewWaves, pos = q % kFewWaves;
    place = (int)(c % kFewPlaces);
    uint32_t run = 0;
    if ((threadIdx.x & 63) == 0) {
        if (pos == 0 && c > 0) {
            // the place's last run is over: its waves have read it and its h is used
            while (lds_load(&s.freed[place]) != c / kFewPlaces) __builtin_amdgcn_s_sleep(1);
            __hip_atomic_store(&s.run[place], ((unsigned long long)(c + 1) << 32) | next_run(ticket), __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_WORKGROUP);
        }
        unsigned long long v;
        while ((uint32_t)((v = lds_load(&s.run[place])) >> 32) != c + 1) __builtin_amdgcn_s_sleep(1);
        run = (uint32_t)v;
    }
    return uniform((int)(run * kFewWaves + pos));
}

template <int FMT, int EJ, bool SIG, bool XB>
__device__ __forceinline__ int few_plan(const FewArgs& a, FewPlan& s, uint8_t* x_rows, uint32_t pitch) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    static_assert(64 * kFewWaves == 512, "one thread per expert");
    static_assert(kFewMaxT <= 2 * kFewWaves, "two tokens per wave");
    s.mask[tid] = 0;
    if (tid < kFewPlaces) { s.read[tid] = 0; s.finished[tid] = 0; s.summed_parts[tid] = 0; s.verdict[tid] = 0; s.freed[tid] = 0; s.run[tid] = 0; }
    if (tid < kFewSlots) s.ready[tid] = 0;
    if (tid == 0) { s.drawn = 0; s.summed = 0; s.polling = 0; }
    __syncthreads();
    // the first run, drawn beside the top-k
    uint32_t first = 0;
    auto mid = [&] {
        if (tid == 64 * kFewWaves - 1) first = next_run(a.counters);
    };
    auto token = [&](int t, int id, float w) {
        if (lane < a.k) {
            s.ids[t * a.k + lane] = (int16_t)id;
            s.w[t * a.k + lane] = w;
            atomicOr(&s.mask[id], 1u << t);
        }
    };
    if (wave + kFewWaves < a.T) {
        const float* const L[2] = {a.logits + (size_t)wave * a.E, a.logits + (size_t)(wave + kFewWaves) * a.E};
        int id[2];
        float w[2];
        topk_rows<EJ, 2, kFewParts, SIG>(L, (size_t)a.T * a.E, a.bias, a.E, a.k, id, w, mid);
        token(wave, id[0], w[0]);
        token(wave + kFewWaves, id[1], w[1]);
    } else if (wave < a.T) {
        const float* const L[1] = {a.logits + (size_t)wave * a.E};
        int id[1];
        float w[1];
        topk_rows<EJ, 1, kFewParts, SIG>(L, (size_t)a.T * a.E, a.bias, a.E, a.k, id, w, mid);
        token(wave, id[0], w[0]);
    } else {
        mid();
    }
    // the rows of x, behind the top-k of the waves that have tokens
    const int pieces = a.H / 16;
#pragma unroll 4
    for (int i = tid; i < a.T * pieces; i += 64 * kFewWaves) {
        const int t = i / pieces, c = i - t * pieces;
        const uint4 v = *(const uint4*)(a.xq + (size_t)t * a.H + 16 * c);
        if constexpr (XB) {
            // MXFP4: with the scale of their 128 channels
            const float scale = FMT == 1 ? 1.0f : e8m0(((const uint8_t*)a.xs)[(size_t)t * (a.H / kFp8Block) + c / (kFp8Block / 16)]);
            v8bf* d = (v8bf*)(x_rows + t * pitch + 32 * c);
            d[0] = fp8_to_bf16(v.x, v.y, scale);
            d[1] = fp8_to_bf16(v.z, v.w, scale);
        } else {
            *(uint4*)(x_rows + t * pitch + 16 * c) = v;
        }
    }
    if (tid == 64 * kFewWaves - 1) s.run[0] = (1ull << 32) | first;
    __syncthreads();
    const uint32_t m = s.mask[tid];
    const unsigned long long any = __ballot(m != 0);
    if (lane == 0) s.wave_count[wave] = __popcll(any);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int q = 0; q < kFewWaves; ++q) {
        if (q < wave) before += s.wave_count[q];
        total += s.wave_count[q];
    }
    if (m) {
        const int u = before + __popcll(any & ((1ull << lane) - 1));
        s.index[tid] = (int16_t)u;
        s.expert[u] = (int16_t)tid;
    }
    __syncthreads();
    if (tid < a.T * a.k) {
        const int t = tid / a.k, e = s.ids[tid];
        s.slot[s.index[e]][__popc(s.mask[e] & ((1u << t) - 1))] = (uint8_t)tid;
    }
    __syncthreads();
    return total;
}

// FP8 of one 128-channel block of h (in LDS) for the n rows of touched expert
// u: 16 lanes per row, 8 channels each, the rule of quantise_row.
template <bool F32S>
__device__ __forceinline__ void quantise_h_block(const FewArgs& a, const FewPlan& s, int place, int u, int n, int blk) {
    const int lane = threadIdx.x & 63;
    for (int r0 = 0; r0 < n; r0 += 4) {
        const int row = min(r0 + (lane >> 4), n - 1);   // past n: the last row again, not stored
        const v4f* p = (const v4f*)&s.h[place][row][8 * (lane & 15)];
        const v4f p0 = p[0], p1 = p[1];
        const float v[8] = {p0[0], p0[1], p0[2], p0[3], p1[0], p1[1], p1[2], p1[3]};
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d, 16));
        float q[8];
        uint32_t scale;
        if constexpr (F32S) {
            const float sc = fp8_f32_scale_product(amax), dv = amax > 0.0f ? sc : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = fp8_f32_quotient(v[i], dv);
            scale = __float_as_uint(sc);
        } else {
            const int e = fp8_block_exponent(amax);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = __builtin_amdgcn_ldexpf(v[i], -e);
            scale = (uint32_t)(e + 127);
        }
        if (r0 + (lane >> 4) < n) {
            const size_t slot = s.slot[u][row];
            put8(a.hq + slot * a.I + blk * kFp8Block + 8 * (lane & 15), pack_fp8x4(q[0], q[1], q[2], q[3]),
                 pack_fp8x4(q[4], q[5], q[6], q[7]));
            if ((lane & 15) == 0) {
                const size_t o = slot * (a.I / kFp8Block) + blk;
                if constexpr (F32S)
                    __hip_atomic_store((uint32_t*)a.hs + o, scale, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                else
                    __hip_atomic_store((uint8_t*)a.hs + o, (uint8_t)scale, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
    }
}

// y[t][c .. c+32) = sum_j w[t][j] y_(t,j), in slot order: 8 lanes per token.
// get(slot, i): channels c + i .. of the slot's row.
template <typename Get>
__device__ __forceinline__ void combine_block(const FewArgs& a, const FewPlan& s, int fb, Get get) {
    const int lane = threadIdx.x & 63;
    const int c = 32 * fb + 4 * (lane & 7);
    for (int t = lane >> 3; t < a.T; t += 8) {
        uint4 p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < a.k) p[j] = get(t * a.k + j, 4 * (lane & 7));
        v4f acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j < a.k) {
                const float w = s.w[t * a.k + j];
                acc[0] = fmaf(w, __uint_as_float(p[j].x), acc[0]);
                acc[1] = fmaf(w, __uint_as_float(p[j].y), acc[1]);
                acc[2] = fmaf(w, __uint_as_float(p[j].z), acc[2]);
                acc[3] = fmaf(w, __uint_as_float(p[j].w), acc[3]);
            }
        }
        if (a.fuse_tail) {
            put16((float*)a.y + (size_t)t * a.H + c, acc);
        } else if (a.out_bf16) {
            uint2 o;
            o.x = (uint32_t)float_to_bf16_rne(acc[0]) | ((uint32_t)float_to_bf16_rne(acc[1]) << 16);
            o.y = (uint32_t)float_to_bf16_rne(acc[2]) | ((uint32_t)float_to_bf16_rne(acc[3]) << 16);
            *(uint2*)((uint16_t*)a.y + (size_t)t * a.H + c) = o;
        } else {
            *(v4f*)((float*)a.y + (size_t)t * a.H + c) = acc;
        }
    }
}

// sum over the workgroup, in wave order
__device__ __forceinline__ float group_sum(float v, float* red) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < kFewWaves; ++q) s += red[q];
    return s;
}

// The block's tail on row t of y, by the workgroup: gate, residual sum and norms
// as in block_norm.hip.  What does not depend on y is loaded before the wait.
template <typename Wait>
__device__ __forceinline__ void tail_row(const FewArgs& a, int t, float (*red)[kFewWaves], Wait wait) {
    constexpr int NT = 64 * kFewWaves, V = kFewTailMaxH / (8 * NT);   // pieces of 8 channels per thread
    const TailArgs& T = a.tail;
    const size_t row = (size_t)t * a.H;
    float v[V][8], r[V][8], wp[V][8], gt[V][8], wn[V][8];
    int c[V];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        c[u] = (u * NT + threadIdx.x) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) { v[u][i] = 0.0f; wp[u][i] = gt[u][i] = wn[u][i] = 1.0f; }
        if (c[u] < a.H) {
            load8<false>(T.r, T.res_bf16, row + c[u], r[u]);
            if (T.post_norm && T.w_post) load8<false>(T.w_post, T.param_bf16, c[u], wp[u]);
            if (T.gate) load8<false>(T.gate, T.param_bf16, (T.gate_per_token ? row : 0) + c[u], gt[u]);
            if (T.n_next && T.w_next) load8<false>(T.w_next, T.param_bf16, c[u], wn[u]);
        }
    }
    wait();
#pragma unroll
    for (int u = 0; u < V; ++u) {
        if (c[u] < a.H) {
            const uint4 p0 = get16((const float*)a.y + row + c[u]), p1 = get16((const float*)a.y + row + c[u] + 4);
            const uint32_t b[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = __uint_as_float(b[i]);
        }
    }
    auto rstd = [&](float* part) {
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(v[u][i], v[u][i], s);   // channels past H hold zeros
        return inv_rms(group_sum(s, part), a.H, T.eps);
    };
    const float post = T.post_norm ? rstd(red[0]) : 1.0f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        if (c[u] < a.H) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = fmaf(T.scale, v[u][i] * (post * wp[u][i]) * gt[u][i], r[u][i]);
            if (T.res_bf16) {
                const v4u o = pack8(v[u]);
                *(v4u*)((uint16_t*)T.r_out + row + c[u]) = o;
                unpack8(o, v[u]);   // n' is the norm of r' as stored
            } else {
                v4f* o = (v4f*)((float*)T.r_out + row + c[u]);
                o[0] = v4f{v[u][0], v[u][1], v[u][2], v[u][3]};
                o[1] = v4f{v[u][4], v[u][5], v[u][6], v[u][7]};
            }
        }
    }
    if (!T.n_next) return;
    const float next = rstd(red[1]);
#pragma unroll
    for (int u = 0; u < V; ++u) {
        if (c[u] < a.H) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] *= next * wn[u][i];
            *(v4u*)((uint16_t*)T.n_next + row + c[u]) = pack8(v[u]);
        }
    }
}

// Parts into which K of the gate/up items is cut: with fewer blocks of h than
// half the workgroups, the rest would only wait (four-way split Pro layer: 32
// blocks for one token, 31 us in parts and 38 us whole; one token of the Flash
// layer, 128 blocks, 38.8 and 39.6 us, before its down runs were joined).  At least two stages to a part.  By the sizes
// alone, not by the touched experts, so that the order of a token's sums does not
// depend on the other tokens' routing.
__device__ __forceinline__ int split_of(const FewArgs& a, int stage_cols) {
    const int blocks = min(a.T * a.k, a.E) * (a.I / kFp8Block), stages = (a.H + stage_cols - 1) / stage_cols;
    int S = 1;
    while (2 * S * blocks <= kFewGrid && 4 * S <= stages && S < kFewMaxSplit) S *= 2;
    return S;
}

// XB: x as bf16 in LDS.  JOIN (8 routing slots at most): a down run is one block of
// 32 features of all touched experts, on rows of h copied to LDS, and is summed there.
template <int FMT, bool PK, int EJ, bool SIG, bool XB, bool JOIN>
__global__ void __launch_bounds__(64 * kFewWaves, 2) few_layer_kernel(FewArgs a) {
    __shared__ FewPlan s;
    // rows of x, 16 bytes of padding each: the 16 rows of an MFMA operand then lie
    // on different banks
    __shared__ __attribute__((aligned(16))) uint8_t x_rows[kFewRowBytes];
    const uint32_t pitch = (XB ? 2 : 1) * a.H + 16;
    const int U = few_plan<FMT, EJ, SIG, XB>(a, s, x_rows, pitch);
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int KBI = a.I / kFp8Block;
    uint32_t* ticket = a.counters;
    uint32_t* ready = a.counters + kFewCounterStride;                     // [U] quantised blocks
    uint32_t* fb_count = ready + kFewSlots * kFewCounterStride;           // [H / 32] down items
    const int f2 = a.H / 32;
    uint32_t* done = fb_count + f2 * kFewCounterStride;                   // summed features of y, in 32s
    uint32_t* parts = done + kFewCounterStride;                           // finished parts of a block of h
    const uint8_t* pad = (const uint8_t*)(parts + kFewSplitBlocks * kFewCounterStride);   // kFewPad words of zeros
    // gate/up items: 8 to a run, which is a 128-channel block of h or one of its S parts
    const int S = split_of(a, FewStageW<FMT>::kCols);
    const int n1 = U * KBI * S * kFewWaves;
    const uint32_t h_pitch = a.I + 16, hs_row = KBI * (FMT == 1 ? 4 : 1);
    const int n2 = (JOIN ? kFewWaves : U) * f2;                         // down items
    const int n3 = (n2 + kFewWaves - 1) / kFewWaves * kFewWaves;          // first item behind their runs
    const uint32_t xs_row = (a.H / kFp8Block) * (FMT == 1 ? 4 : 1);

    int place;
    int item = draw(ticket, s, place);
    while (item < n1) {
        const int run = item / kFewWaves, bg = run / S, ks = run - bg * S;
        const int u = bg / KBI, blk = bg - u * KBI, f = item % kFewWaves;   // 16 features of the block
        const int e = uniform(s.expert[u]), n = __popc(uniform(s.mask[e]));
        const uint32_t slot = s.slot[u][min(r, n - 1)];
        const int row0 = blk * kFp8Block + 16 * f;
        FewPtrs P;
        P.pad = pad;
        few_lane_offsets<FMT, PK>(P, a.H);
        few_tile<FMT>(P, 0, a.w13, a.w13_scale, (size_t)e * 2 * a.I + row0, a.H);
        few_tile<FMT>(P, 1, a.w13, a.w13_scale, (size_t)e * 2 * a.I + a.I + row0, a.H);
        const uint32_t t = slot / (uint32_t)a.k;
        P.xs = (const uint8_t*)a.xs;
        P.xso = t * xs_row;
        P.lo = ks * P.all / S;
        P.nst = (ks + 1) * P.all / S - P.lo;
        // the run's 8 items start at 8 different places of K (see expert_gemm.hip):
        // their rows lie 8 K or 16 K bytes apart and read in step would fall on
        // the same memory channels
        P.first = f * P.nst / kFewWaves;
        v4f acc[2];
        few_item<FMT, PK, XB>(P, x_rows + t * pitch, acc);
        keep_whole(acc);
        bool whole = true;
        if (S > 1) {
            // The part's sums go to memory.  The wave that finishes the run counts it
            // for its block; where it was the block's last part, every wave adds up the
            // parts of its own 16 features, in their order.
            auto part = [&](int q) { return a.part + (((size_t)(bg * S + q) * kFewWaves + f) * 64 + lane) * 8; };
            if (r < n) {
                put16(part(ks), acc[0]);
                put16(part(ks) + 4, acc[1]);
            }
            wave_done();
            uint32_t before = 0;
            if (lane == 0) before = lds_add(&s.summed_parts[place]);
            before = (uint32_t)uniform((int)before);
            const uint32_t runs = before / kFewWaves + 1;   // of this place, this one included
            if (before % kFewWaves == kFewWaves - 1) {
                whole = count(parts + bg * kFewCounterStride) == (uint32_t)(S - 1);
                if (lane == 0) lds_store(&s.verdict[place], 2 * runs + (whole ? 1u : 0u));
            } else {
                uint32_t v = 0;
                while (((v = (uint32_t)uniform((int)lds_load(&s.verdict[place]))) >> 1) != runs) __builtin_amdgcn_s_sleep(1);
                asm volatile("" ::: "memory");
                whole = v & 1u;
            }
            if (whole && r < n) {
                v4f sum[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                uint4 p[kFewMaxSplit][2];
#pragma unroll
                for (int q = 0; q < kFewMaxSplit; ++q) {
                    if (q < S) {
                        p[q][0] = get16(part(q));
                        p[q][1] = get16(part(q) + 4);
                    }
                }
#pragma unroll
                for (int q = 0; q < kFewMaxSplit; ++q) {
                    if (q < S) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            sum[i] += v4f{__uint_as_float(p[q][i].x), __uint_as_float(p[q][i].y), __uint_as_float(p[q][i].z),
                                          __uint_as_float(p[q][i].w)};
                    }
                }
                acc[0] = sum[0];
                acc[1] = sum[1];
            }
        }
        if (whole && r < n) {
            // silu(gate) * up of features 16 f + 4 g .. of the block
            v4f h;
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = silu_f32(acc[0][i]) * acc[1][i];
            *(v4f*)&s.h[place][r][16 * f + 4 * g] = h;
        }
        // LDS serves a wave's accesses in order: the h of 8 counted items is there
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        uint32_t before = 0;
        if (lane == 0) before = lds_add(&s.finished[place]);
        if (uniform((int)before) % kFewWaves == kFewWaves - 1) {
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
            if (whole) {
                quantise_h_block<FMT == 1>(a, s, place, u, n, blk);
                wave_done();
                if constexpr (!JOIN) count(ready + u * kFewCounterStride);
                else if (lane < kFewWaves)
                    __hip_atomic_fetch_add(ready + (u * kFewWaves + lane) * kFewCounterStride, 1u, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
            }
            if (lane == 0) lds_add(&s.freed[place]);
        }
        item = draw(ticket, s, place);
    }
    // Down items.  An item's first weights are loaded before the item in front of
    // it is stored, and that one is counted once the wave has waited for its next
    // rows anyway.
    struct Item { int u, f, n; uint32_t slot; FewPtrs P; };
    FewStageW<FMT> w[kDownW];
    auto begin = [&](int i, Item& it) {
        // the run is over for its place once its 8 waves have read it
        if (!JOIN && lane == 0 && lds_add(&s.read[place]) % kFewWaves == kFewWaves - 1) lds_add(&s.freed[place]);
        it.u = JOIN ? min(i % kFewWaves, U - 1) : i / f2;
        it.f = JOIN ? i / kFewWaves : i - it.u * f2;
        const int e = uniform(s.expert[it.u]);
        it.n = __popc(uniform(s.mask[e]));
        it.slot = s.slot[it.u][min(r, it.n - 1)];
        it.P.pad = pad;
        few_lane_offsets<FMT, PK>(it.P, a.I);
        few_tile<FMT>(it.P, 0, a.w2, a.w2_scale, (size_t)e * a.H + 32 * it.f, a.I);
        few_tile<FMT>(it.P, 1, a.w2, a.w2_scale, (size_t)e * a.H + 32 * it.f + 16, a.I);
        if (JOIN && i % kFewWaves >= U) it.n = it.P.nst = 0;   // fewer experts than waves: nothing to do
        it.P.first = (JOIN ? e : it.f) % kFewWaves * it.P.nst / kFewWaves;
        it.P.x = a.hq;
        it.P.xs = (const uint8_t*)a.hs;
        it.P.xo = it.slot * a.I;
        it.P.xso = it.slot * hs_row;
        down_prefetch<FMT, PK>(it.P, w);
    };
    auto sum = [&](int f, auto get) {
        combine_block(a, s, f, get);
        if (a.fuse_tail) {
            wave_done();
            count(done);
        }
    };
    auto finish = [&](int f) {
        wave_done();
        if (count(fb_count + f * kFewCounterStride) == (uint32_t)(U - 1))
            sum(f, [&](int slot, int i) { return get16(a.y_slot + (size_t)slot * a.H + 32 * f + i); });
    };
    // JOIN: every expert's blocks are all counted.  Each count went to 8 counters,
    // so that the workgroups' polls are spread over them.
    auto all_ready = [&] {
        uint32_t v = (uint32_t)KBI;
        if (lane < U)
            v = __hip_atomic_load(ready + (lane * kFewWaves + blockIdx.x % kFewWaves) * kFewCounterStride, __ATOMIC_RELAXED,
                                  __HIP_MEMORY_SCOPE_AGENT);
        return (bool)__all(v >= (uint32_t)KBI);
    };
    // a wave's next item, the rest of the last down run left out: every wave then
    // ends with one item >= n3, and a workgroup's 8 waves (8 items to a run, all
    // earlier runs used up) with the 8 items of one run
    auto draw_down = [&]() {
        int i;
        do i = draw(ticket, s, place) - n1;
        while (i >= n2 && i < n3);
        return i;
    };
    item -= n1;
    if (item >= n2 && item < n3) item = draw_down();
    int stored = -1;   // features whose rows are stored, not yet counted
    Item it;
    if (item < n2) begin(item, it);
    while (item < n2) {
        if constexpr (JOIN) wait_until(a, s, &s.ready[0], all_ready);
        else wait_for(a, s, ready + it.u * kFewCounterStride, (uint32_t)KBI, &s.ready[it.u]);
        if (stored >= 0) finish(stored);
        v4f acc[2];
        if constexpr (JOIN) {
            // The expert's rows of h come to LDS, in one trip, over the rows of x:
            // with all of h there no wave multiplies x any more.  (Waves of two runs
            // may copy the same rows: the same bytes.)
            uint8_t* const scales = x_rows + a.T * a.k * h_pitch;
            const int pieces = a.I / 16;
#pragma unroll 4
            for (int i = lane; i < it.n * pieces; i += 64) {
                const int j = i / pieces, c = 16 * (i - j * pieces);
                const uint32_t slot = s.slot[it.u][j];
                *(uint4*)(x_rows + slot * h_pitch + c) = get16(a.hq + (size_t)slot * a.I + c);
            }
            for (int i = lane; i < it.n * KBI; i += 64) {
                const int j = i / KBI, b = i - j * KBI;
                const uint32_t slot = s.slot[it.u][j];
                if constexpr (FMT == 1) {
                    *(float*)(scales + slot * hs_row + 4 * b) = load_xs<true, float>((const uint8_t*)a.hs + slot * hs_row + 4 * b);
                } else {
                    scales[slot * hs_row + b] = load_xs<true, uint8_t>((const uint8_t*)a.hs + slot * hs_row + b);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
            down_item<FMT, PK>(it.P, FewRowsLds{x_rows + it.slot * h_pitch, scales + it.slot * hs_row}, w, acc);
        } else {
            down_item<FMT, PK>(it.P, FewRowsMemory{}, w, acc);
        }
        keep_whole(acc);
        if constexpr (JOIN) {
            // rows by slot, 32 channels each, where the gate/up runs keep h
            if (r < it.n) {
                float* o = &s.h[place][it.slot][4 * g];
                *(v4f*)o = acc[0];
                *(v4f*)(o + 16) = acc[1];
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
            uint32_t before = 0;
            if (lane == 0) before = lds_add(&s.finished[place]);
            if (uniform((int)before) % kFewWaves == kFewWaves - 1) {
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
                sum(it.f, [&](int slot, int i) { return *(const uint4*)&s.h[place][slot][i]; });
                if (lane == 0) lds_add(&s.freed[place]);
            }
        } else {
            if (r < it.n) {
                float* o = a.y_slot + (size_t)it.slot * a.H + 32 * it.f + 4 * g;
                put16(o, acc[0]);
                put16(o + 16, acc[1]);
            }
            stored = it.f;
        }
        item = draw_down();
        if (item < n2) begin(item, it);
    }
    if (stored >= 0) finish(stored);
    // The block's tail: the runs behind the down items are the rows, and the last
    // run of a workgroup, one item per wave, is the same for all its waves.
    const int t = (item - n3) / kFewWaves;
    if (a.fuse_tail && t < a.T)
        tail_row(a, t, s.red, [&] { wait_for(a, s, done, (uint32_t)f2, &s.summed); });
}

template <int FMT, bool PK, int EJ, bool SIG>
hipError_t launch_layer(const FewArgs& a, hipStream_t stream) {
    const dim3 grid(kFewGrid), block(64 * kFewWaves);
    // x as bf16 in LDS where it fits (16 tokens up to H = 3832, 14 at 4096, 9 at
    // 6144): a third fewer conversions (one token of the Flash layer 39.6 us, 40.7
    // without; 3 of the canonical four-way split Pro layer 64.7 and 67.5)
    const bool xb = a.T * (2 * a.H + 16) <= kFewRowBytes;
    // Runs of all touched experts, where their rows of h fit in LDS: one token of
    // the Flash layer 36.4 us and 38.6 without, FP8 experts 50.0 and 54.2, the
    // canonical layout 43.2 and 46.0.  With more experts than waves a run would have
    // to wait for experts that others are still at.
    const int slots = a.T * a.k;
    if (xb && slots <= kFewWaves && slots * (a.I + 16 + a.I / kFp8Block * 4) <= kFewRowBytes)
        hipLaunchKernelGGL((few_layer_kernel<FMT, PK, EJ, SIG, true, true>), grid, block, 0, stream, a);
    else if (xb)
        hipLaunchKernelGGL((few_layer_kernel<FMT, PK, EJ, SIG, true, false>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((few_layer_kernel<FMT, PK, EJ, SIG, false, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}
template <int FMT, bool PK>
hipError_t launch_layer(const FewArgs& a, hipStream_t stream) {
    // keys per lane of the top-k: up to 256 experts, and the rest
    if (a.E <= 256) return a.sigmoid ? launch_layer<FMT, PK, 4, true>(a, stream) : launch_layer<FMT, PK, 4, false>(a, stream);
    return a.sigmoid ? launch_layer<FMT, PK, 8, true>(a, stream) : launch_layer<FMT, PK, 8, false>(a, stream);
}

}  // namespace

}  // namespace moe
