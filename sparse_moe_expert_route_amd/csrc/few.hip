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
//     expert;
//   - a down item loads its first weights, then waits until its expert's blocks
//     are all counted;
//   - the wave whose down item is the last on its 32 features (one from every
//     touched expert) sums them over the k slots of every token, in slot order.
// Which wave does that depends on timing, what it computes does not: results
// have the same bits on every run.
//
// Every wait ends: a running workgroup draws the items in order and its waves
// take them in order, one at a time; gate/up items wait for nothing and have the
// lower numbers.  The lowest unfinished item therefore lies with a running
// workgroup, in a wave that waits for nothing unfinished or next in line for its
// first free wave (whose items, being lower, are finished), whatever part of the
// grid is resident, and also when several of these kernels share the device.  (A wait is bounded all the
// same: past kFewMaxPolls polls, seconds, it gives up and sets an error bit.)
//
// Memory order: the XCDs' L2 caches are not coherent with each other, so what
// crosses workgroups (the codes and scales of h, the rows of y) is stored and
// loaded with agent-scope accesses, which do not stay in an L2.  A wave's stores
// are complete (vmcnt 0) before it counts; a reader sees the count before it
// issues its loads.
#include <type_traits>

#include "block_launch.h"
#include "moe_internal.h"
#include "fp8_rows.h"
#include "topk_rows.h"

namespace moe {

namespace {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kFewWaves = 8;                  // waves per workgroup of the layer kernel
constexpr int kFewPlaces = 4;                 // runs a workgroup can have in work
constexpr int kFewGrid = 256;                 // its workgroups: one per CU
constexpr int kFewSlots = kFewMaxT * 8;       // routing slots, and so touched experts, at most
constexpr uint32_t kFewMaxPolls = 1u << 23;
constexpr int kRouteWaves = 16;               // waves per workgroup of the route kernel

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
// waits until *c >= n
__device__ __forceinline__ void wait_for(const uint32_t* c, uint32_t n, uint32_t* err) {
    for (uint32_t i = 0;; ++i) {
        const uint32_t v = (uint32_t)__builtin_amdgcn_readfirstlane(
            (int)__hip_atomic_load(c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        if (v >= n) break;
        if (i >= kFewMaxPolls) {
            if ((threadIdx.x & 63) == 0) __hip_atomic_store(err, kErrStalled, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            break;
        }
        __builtin_amdgcn_s_sleep(2);
    }
    asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// Route kernel.  Workgroups of 16 waves:
//   [0, gx)        router logits of 16 experts x 16 tokens on the bf16 MFMA, the
//                  16 waves splitting K (H = 4096: 8 steps each, all loads of a
//                  wave in flight at once), summed through LDS in wave order;
//   [gx, gx + T)   the FP8 copy of one token row;
//   gx + T         the counters and error words of the layer kernel, cleared.
// ---------------------------------------------------------------------------
template <bool F32S>
__global__ void __launch_bounds__(64 * kRouteWaves) few_route_kernel(FewArgs a) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int gx = (a.E + 15) / 16;
    const int b = blockIdx.x;
    if (b >= gx + a.T) {
        for (int i = tid; i < a.n_counters; i += 64 * kRouteWaves) a.counters[i] = 0u;
        if (tid < 2) a.err[tid] = 0u;
        return;
    }
    if (b >= gx) {
        quantise_row<F32S, 64 * kRouteWaves, true>(a.x + (size_t)(b - gx) * a.H, a.xq, a.xs, b - gx, a.H);
        return;
    }
    __shared__ v4f red[kRouteWaves][64];
    const int g = lane >> 4, r = lane & 15, e0 = 16 * b;
    const uint16_t* wp = a.w_router + (size_t)min(e0 + r, a.E - 1) * a.H + 8 * g;
    const uint16_t* xp = a.x + (size_t)min(r, a.T - 1) * a.H + 8 * g;
    const int ns = a.H / 32;
    const int s0 = wave * ns / kRouteWaves, s1 = (wave + 1) * ns / kRouteWaves;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    constexpr int U = 8;
    int s = s0;
    for (; s + U <= s1; s += U) {
        v8bf wa[U], xb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            wa[u] = *(const v8bf*)(wp + 32 * (s + u));
            xb[u] = *(const v8bf*)(xp + 32 * (s + u));
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa[u], xb[u], acc, 0, 0, 0);
    }
    if (s < s1) {   // the last, shorter chunk: past its end the last step is loaded again and left out
        v8bf wa[U], xb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            wa[u] = *(const v8bf*)(wp + 32 * min(s + u, s1 - 1));
            xb[u] = *(const v8bf*)(xp + 32 * min(s + u, s1 - 1));
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
        for (int q = 0; q < kRouteWaves; ++q) v += red[q][l][i];
        const int e = e0 + 4 * (l >> 4) + i, t = l & 15;
        if (e < a.E && t < a.T) a.logits[(size_t)t * a.E + e] = v;
    }
}

// ---------------------------------------------------------------------------
// One pipeline stage of an item: two 16-row weight tiles and the token rows.
//
// MXFP4: 512 of K.  The lane group g = lane / 16 takes the stage's g-th 128
// columns, and MFMA j the j-th 32 of each: the four e8m0 scales of a weight row
// over those 128 columns are then one dword of the lane, whose byte j the MFMA
// picks, and the activation scale is one byte per lane and stage.  (A dot
// product may take K in any order as long as both operands do.)  Operand bytes:
// A (e2m1) 16 bytes = columns 32 j .. of the lane's 128; B (e4m3) lane group g'
// holds instruction columns 16 g'.. and 64 + 16 g'.., that is 16 (g' & 1) of
// sub-block j of the 128-column blocks g' / 2 and 2 + g' / 2.
// A last stage shorter than 512 reads its last block again with scales that
// leave nothing of it.
//
// FP8 block-scaled: 256 of K, two 128-column blocks.  The block-scaled MFMA's
// internal sum keeps about 13 bits below its largest product, which at the 448
// full scale of e4m3 x e4m3 moves h by up to 1e-3 and flips a few percent of
// its FP8 codes; here the codes go to bf16 (exact) and the bf16 MFMA, at twice
// the vector work, which stays under the memory time.  Each block's partial sum
// gains its two float32 scales.
// ---------------------------------------------------------------------------
template <int FMT>
struct FewStage;

template <>
struct FewStage<0> {
    static constexpr int kCols = 512;
    v4u w[2][4];
    uint32_t ws[2];
    uint4 x[4][2];
    uint32_t xs;
};
template <>
struct FewStage<1> {
    static constexpr int kCols = 256;
    v4u w[2][2][2];
    float ws[2][2];
    uint4 x[2][2];
    float xs[2];
};

// Wave-uniform bases and the lane's 32-bit offsets from them.
struct FewPtrs {
    const uint8_t* w[2];     // the weight tiles
    const uint8_t* ws[2];    // their scales
    const uint8_t* x;        // the token rows
    const uint8_t* xs;       // their scales
    uint32_t wo, wso;        // the lane's place in a tile and in its scales
    uint32_t xo, xso;        // its token row and that row's scales
    int KB;                  // 128-column blocks of K
};

template <int FMT, bool PK>
__device__ __forceinline__ void few_lane_offsets(FewPtrs& P, int K) {
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    P.KB = K / kFp8Block;
    if constexpr (FMT == 0) {
        P.wo = PK ? 16 * r : r * (K / 2);
        P.wso = PK ? 4 * r : r * (K / 32);
    } else {
        P.wo = PK ? 16 * lane : r * K + 16 * g;
        P.wso = 0;
    }
}
template <int FMT>
__device__ __forceinline__ void few_tile(FewPtrs& P, int i, const uint8_t* w, const uint8_t* ws, size_t row0, int K) {
    P.w[i] = w + row0 * (FMT ? K : K / 2);
    P.ws[i] = FMT ? ws + (row0 / 128) * (K / 128) * 4 : ws + row0 * (K / 32);
}

template <bool PK>
__device__ __forceinline__ v4u load_w(const uint8_t* p) {
    // packed: whole lines of weights that are read once go past the caches
    if constexpr (PK) return __builtin_nontemporal_load((const v4u*)p);
    else return *(const v4u*)p;
}

template <int FMT, bool PK>
__device__ __forceinline__ void load_weights(const FewPtrs& P, int st, FewStage<FMT>& s) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    if constexpr (FMT == 0) {
        const int c = min(4 * st + g, P.KB - 1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s.w[i][j] = load_w<PK>(P.w[i] + (P.wo + (PK ? 1024 : 64) * c) + (PK ? 256 : 16) * j);
            s.ws[i] = *(const uint32_t*)(P.ws[i] + (P.wso + (PK ? 64 : 4) * c));
        }
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int c = min(2 * st + b, P.KB - 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s.w[i][b][0] = load_w<PK>(P.w[i] + (P.wo + (PK ? 2048 : 128) * c));
                s.w[i][b][1] = load_w<PK>(P.w[i] + (P.wo + (PK ? 2048 : 128) * c) + (PK ? 1024 : 64));
                s.ws[i][b] = ((const float*)P.ws[i])[c];
            }
        }
    }
}

// SHARED: the rows were written by other workgroups of this launch
template <bool SHARED>
__device__ __forceinline__ uint4 load_x(const uint8_t* p) {
    if constexpr (SHARED) return get16(p);
    else return *(const uint4*)p;
}

template <int FMT, bool SHARED>
__device__ __forceinline__ void load_rows(const FewPtrs& P, int st, FewStage<FMT>& s) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
    if constexpr (FMT == 0) {
        const int c0 = min(4 * st + (g >> 1), P.KB - 1), c1 = min(4 * st + 2 + (g >> 1), P.KB - 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s.x[j][0] = load_x<SHARED>(P.x + (P.xo + 128 * c0 + 16 * (g & 1)) + 32 * j);
            s.x[j][1] = load_x<SHARED>(P.x + (P.xo + 128 * c1 + 16 * (g & 1)) + 32 * j);
        }
        const uint8_t* xs = P.xs + (P.xso + min(4 * st + g, P.KB - 1));
        s.xs = SHARED ? __hip_atomic_load(xs, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : *xs;
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int c = min(2 * st + b, P.KB - 1);
            s.x[b][0] = load_x<SHARED>(P.x + (P.xo + 128 * c + 16 * g));
            s.x[b][1] = load_x<SHARED>(P.x + (P.xo + 128 * c + 16 * g) + 64);
            const float* xs = (const float*)(P.xs + (P.xso + 4 * c));
            s.xs[b] = SHARED ? __hip_atomic_load(xs, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : *xs;
        }
    }
}

// 8 e4m3 codes -> 8 bf16 (exact)
__device__ __forceinline__ v8bf fp8_to_bf16(uint32_t lo, uint32_t hi) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, false);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, true);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, false);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, true);
    return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <int FMT>
__device__ __forceinline__ void few_compute(const FewPtrs& P, int st, const FewStage<FMT>& s, v4f (&acc)[2]) {
    if constexpr (FMT == 0) {
        const int g = (threadIdx.x & 63) >> 4;
        // past K: both scales 2^-127, so the products are below any float
        const uint32_t keep = 4 * st + g < P.KB ? ~0u : 0u;
        const int ws[2] = {(int)(s.ws[0] & keep), (int)(s.ws[1] & keep)}, xs = (int)(s.xs & keep);
        auto step = [&](auto jc) {
            constexpr int j = decltype(jc)::value;
            const uint4 lo = s.x[j][0], hi = s.x[j][1];
            const v8i xb = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const v4u w = s.w[i][j];
                const v8i wa = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
                acc[i] = mfma_w4a8<j, 0>(wa, xb, acc[i], ws[i], xs);
            }
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float live = 2 * st + b < P.KB ? 1.0f : 0.0f;   // past K: the last block again, with scale 0
            const uint4 lo = s.x[b][0], hi = s.x[b][1];
            const v8bf x0 = fp8_to_bf16(lo.x, lo.y), x1 = fp8_to_bf16(lo.z, lo.w);
            const v8bf x2 = fp8_to_bf16(hi.x, hi.y), x3 = fp8_to_bf16(hi.z, hi.w);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const v4u wl = s.w[i][b][0], wh = s.w[i][b][1];
                v4f part = {0.f, 0.f, 0.f, 0.f};
                part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(wl[0], wl[1]), x0, part, 0, 0, 0);
                part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(wl[2], wl[3]), x1, part, 0, 0, 0);
                part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(wh[0], wh[1]), x2, part, 0, 0, 0);
                part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_to_bf16(wh[2], wh[3]), x3, part, 0, 0, 0);
                const float c = live * s.ws[i][b] * s.xs[b];
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][q] = fmaf(part[q], c, acc[i][q]);
            }
        }
    }
}

// acc[i] = tile i . rows over the whole of K, R stages in flight.  ready() runs
// between the first weight loads and the first loads of the rows.
template <int FMT, bool PK, bool SHARED, typename Ready>
__device__ __forceinline__ void few_item(const FewPtrs& P, v4f (&acc)[2], Ready ready) {
    constexpr int R = 3;
    const int nst = (P.KB + FewStage<FMT>::kCols / 128 - 1) / (FewStage<FMT>::kCols / 128);
    FewStage<FMT> s[R];
#pragma unroll
    for (int i = 0; i < 2; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < nst) load_weights<FMT, PK>(P, i, s[i]);
    ready();
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (i < nst) load_rows<FMT, SHARED>(P, i, s[i]);
    int st = 0;
    for (; st + 2 * R <= nst; st += R) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            few_compute<FMT>(P, st + i, s[i], acc);
            __builtin_amdgcn_sched_barrier(0);
            load_weights<FMT, PK>(P, st + i + R, s[i]);
            load_rows<FMT, SHARED>(P, st + i + R, s[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // R stages loaded, up to R - 1 more to come
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (st + i < nst) few_compute<FMT>(P, st + i, s[i], acc);
        if (st + i + R < nst) {
            load_weights<FMT, PK>(P, st + i + R, s[i]);
            load_rows<FMT, SHARED>(P, st + i + R, s[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (st + i + R < nst) few_compute<FMT>(P, st + i + R, s[i], acc);
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
    uint32_t freed[kFewPlaces];              // the place's runs that are over
    unsigned long long run[kFewPlaces];      // (c + 1) << 32 | number of run c
    float h[kFewPlaces][kFewMaxT][kFp8Block + 4];   // h of a gate/up run: rows of 128 channels
};

template <typename T>
__device__ __forceinline__ T lds_load(T* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP); }
__device__ __forceinline__ uint32_t lds_add(uint32_t* p) {
    return __hip_atomic_fetch_add(p, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}
__device__ __forceinline__ uint32_t next_run(uint32_t* ticket) {
    return __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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

template <int EJ>
__device__ __forceinline__ int few_plan(const FewArgs& a, FewPlan& s) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    static_assert(64 * kFewWaves == 512, "one thread per expert");
    static_assert(kFewMaxT <= 2 * kFewWaves, "two tokens per wave");
    s.mask[tid] = 0;
    if (tid < kFewPlaces) { s.read[tid] = 0; s.finished[tid] = 0; s.freed[tid] = 0; s.run[tid] = 0; }
    if (tid == 0) s.drawn = 0;
    __syncthreads();
    // the first run, while the others wait for the logits
    if (tid == 64 * kFewWaves - 1) s.run[0] = (1ull << 32) | next_run(a.counters);
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
        topk_rows<EJ, 2>(L, a.bias, a.E, a.k, a.sigmoid, id, w);
        token(wave, id[0], w[0]);
        token(wave + kFewWaves, id[1], w[1]);
    } else if (wave < a.T) {
        const float* const L[1] = {a.logits + (size_t)wave * a.E};
        int id[1];
        float w[1];
        topk_rows<EJ, 1>(L, a.bias, a.E, a.k, a.sigmoid, id, w);
        token(wave, id[0], w[0]);
    }
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
__device__ __forceinline__ void combine_block(const FewArgs& a, const FewPlan& s, int fb) {
    const int lane = threadIdx.x & 63;
    const int c = 32 * fb + 4 * (lane & 7);
    for (int t = lane >> 3; t < a.T; t += 8) {
        uint4 p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < a.k) p[j] = get16(a.y_slot + (size_t)(t * a.k + j) * a.H + c);
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
        if (a.out_bf16) {
            uint2 o;
            o.x = (uint32_t)float_to_bf16_rne(acc[0]) | ((uint32_t)float_to_bf16_rne(acc[1]) << 16);
            o.y = (uint32_t)float_to_bf16_rne(acc[2]) | ((uint32_t)float_to_bf16_rne(acc[3]) << 16);
            *(uint2*)((uint16_t*)a.y + (size_t)t * a.H + c) = o;
        } else {
            *(v4f*)((float*)a.y + (size_t)t * a.H + c) = acc;
        }
    }
}

template <int FMT, bool PK, int EJ>
__global__ void __launch_bounds__(64 * kFewWaves, 2) few_layer_kernel(FewArgs a) {
    __shared__ FewPlan s;
    const int U = few_plan<EJ>(a, s);
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int KBI = a.I / kFp8Block;
    uint32_t* ticket = a.counters;
    uint32_t* ready = a.counters + kFewCounterPad;                        // [U] quantised blocks
    uint32_t* fb_count = ready + kFewSlots;                               // [H / 32] down items
    const int f1 = a.I / 16, n1 = U * f1;                                 // gate/up items (runs: 128-channel blocks)
    const int f2 = a.H / 32, n2 = U * f2;                                 // down items
    const uint32_t xs_row = (a.H / kFp8Block) * (FMT ? 4 : 1), hs_row = KBI * (FMT ? 4 : 1);

    int place;
    int item = draw(ticket, s, place);
    while (item < n1) {
        const int u = item / f1, f = item - u * f1;
        const int e = uniform(s.expert[u]), n = __popc(uniform(s.mask[e]));
        const uint32_t slot = s.slot[u][min(r, n - 1)];
        FewPtrs P;
        few_lane_offsets<FMT, PK>(P, a.H);
        few_tile<FMT>(P, 0, a.w13, a.w13_scale, (size_t)e * 2 * a.I + 16 * f, a.H);
        few_tile<FMT>(P, 1, a.w13, a.w13_scale, (size_t)e * 2 * a.I + a.I + 16 * f, a.H);
        const uint32_t t = slot / (uint32_t)a.k;
        P.x = a.xq;
        P.xs = (const uint8_t*)a.xs;
        P.xo = t * a.H;
        P.xso = t * xs_row;
        v4f acc[2];
        few_item<FMT, PK, false>(P, acc, [] {});
        if (r < n) {
            // silu(gate) * up of features 16 f + 4 g ..
            v4f h;
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = silu_f32(acc[0][i]) * acc[1][i];
            *(v4f*)&s.h[place][r][16 * (f % 8) + 4 * g] = h;
        }
        // LDS serves a wave's accesses in order: the h of 8 counted items is there
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        uint32_t before = 0;
        if (lane == 0) before = lds_add(&s.finished[place]);
        if (uniform((int)before) % kFewWaves == kFewWaves - 1) {
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
            quantise_h_block<FMT == 1>(a, s, place, u, n, f / 8);
            wave_done();
            count(ready + u);
            if (lane == 0) lds_add(&s.freed[place]);
        }
        item = draw(ticket, s, place);
    }
    item -= n1;
    while (item < n2) {
        // the run is over for its place once its 8 waves have read it
        if (lane == 0 && lds_add(&s.read[place]) % kFewWaves == kFewWaves - 1) lds_add(&s.freed[place]);
        const int u = item / f2, f = item - u * f2;
        const int e = uniform(s.expert[u]), n = __popc(uniform(s.mask[e]));
        const uint32_t slot = s.slot[u][min(r, n - 1)];
        FewPtrs P;
        few_lane_offsets<FMT, PK>(P, a.I);
        few_tile<FMT>(P, 0, a.w2, a.w2_scale, (size_t)e * a.H + 32 * f, a.I);
        few_tile<FMT>(P, 1, a.w2, a.w2_scale, (size_t)e * a.H + 32 * f + 16, a.I);
        P.x = a.hq;
        P.xs = (const uint8_t*)a.hs;
        P.xo = slot * a.I;
        P.xso = slot * hs_row;
        v4f acc[2];
        few_item<FMT, PK, true>(P, acc, [&] { wait_for(ready + u, (uint32_t)KBI, a.err); });
        if (r < n) {
            float* o = a.y_slot + (size_t)slot * a.H + 32 * f + 4 * g;
            put16(o, acc[0]);
            put16(o + 16, acc[1]);
        }
        wave_done();
        if (count(fb_count + f) == (uint32_t)(U - 1)) combine_block(a, s, f);
        item = draw(ticket, s, place) - n1;
    }
}

template <int FMT, bool PK>
hipError_t launch_layer(const FewArgs& a, hipStream_t stream) {
    const dim3 grid(kFewGrid), block(64 * kFewWaves);
    if (a.E <= 256) hipLaunchKernelGGL((few_layer_kernel<FMT, PK, 4>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((few_layer_kernel<FMT, PK, 8>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few_layer(const FewArgs& a, int packed, int fp8_block, hipStream_t stream) {
    if (a.T < 1 || a.T > kFewMaxT || a.n_counters < few_counters(a.H)) return hipErrorInvalidValue;
    const dim3 grid((a.E + 15) / 16 + a.T + 1), block(64 * kRouteWaves);
    if (fp8_block) hipLaunchKernelGGL(few_route_kernel<true>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(few_route_kernel<false>, grid, block, 0, stream, a);
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
    if (fp8_block) return packed ? launch_layer<1, true>(a, stream) : launch_layer<1, false>(a, stream);
    return packed ? launch_layer<0, true>(a, stream) : launch_layer<0, false>(a, stream);
}

}  // namespace moe
