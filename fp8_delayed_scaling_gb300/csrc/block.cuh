// block.cuh — what the block-scaled FP8 kernels share: a block's scale, the ragged groups' tables and
// the host checks of their arguments.
#pragma once

#include "common.cuh"

namespace fp8dl {

// Lets a kernel take up to `bytes` of dynamic shared memory: once per device (`done` holds a bit for each), and always
// the most that any call of it needs, so that calls of several threads cannot lower it for one another.
template <typename... KArgs>
fp8dl_status allow_smem(void (*kernel)(KArgs...), size_t bytes, int dev, std::atomic<uint64_t> &done, const char *what) {
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return FP8DL_OK;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return fail(FP8DL_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    done.fetch_or(bit, std::memory_order_release);
    return FP8DL_OK;
}

constexpr int kMaxGroups = 1024;

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool block_tokens_ok(int64_t n) { return n >= 0 && n < (int64_t(1) << 31); }

// offsets/n_groups of a call; `optional`: NULL and 0 stand for no groups.
inline fp8dl_status check_block_groups(const int32_t *offsets, int32_t n_groups, bool optional) {
    if (optional && !offsets) {
        FP8DL_CHECK_ARG(n_groups == 0, "n_groups (%d) without offsets", n_groups);
        return FP8DL_OK;
    }
    FP8DL_CHECK_ARG(offsets, "offsets is NULL");
    FP8DL_CHECK_ARG(n_groups >= 1 && n_groups <= kMaxGroups, "n_groups must be in [1, %d]", kMaxGroups);
    if (reinterpret_cast<uintptr_t>(offsets) & 3u) return fail(FP8DL_ERR_ALIGN, "offsets must be 4-byte aligned");
    return FP8DL_OK;
}

// Group g's rows, clamped to the tensor (the host does not see the offsets).
__device__ __forceinline__ void group_rows(const int32_t *offsets, int g, int64_t rows, int64_t &first, int64_t &end) {
    first = min(max((int64_t)offsets[g], (int64_t)0), rows);
    end = min(max((int64_t)offsets[g + 1], first), rows);
}

__device__ __forceinline__ int64_t warp_inclusive_sum(int64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// (scale, stored factor) of a block whose largest finite magnitude is amax: both are
// correctly rounded divisions.  A maximum below 2^-100 counts as 2^-100, so that the scale
// stays finite; an all-zero block has scale 1.
template <int FMT>
__device__ __forceinline__ float2 block_scale(float amax) {
    constexpr float FMAX = FMT == FP8DL_E4M3 ? 448.0f : 57344.0f;
    const float sc = amax > 0.0f ? __fdiv_rn(FMAX, fmaxf(amax, 7.888609052210118e-31f)) : 1.0f;
    return make_float2(sc, __frcp_rn(sc));
}

// The same two figures, bit for bit, in fewer instructions: Markstein's division (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34, 1990): a reciprocal refined by one step is
// the correctly rounded one or next to it, and a quotient corrected by its exact remainder is correctly rounded.
// No step leaves the normal numbers for maxima of 2^-100 to the largest finite one: dividend and divisor are taken a
// fourth, so that the divisor's reciprocal stays above 2^-126.  The tests compare both figures with the divisions for every
// maximum of six binades, both formats: the hardware's first estimate decides the last bit of a handful of mantissas.
__device__ __forceinline__ float refined_rcp(float b) {
    const float y = rcp_approx_ftz(b);
    return __fmaf_rn(y, __fmaf_rn(-b, y, 1.0f), y);
}
template <int FMT>
__device__ __forceinline__ float2 block_scale_fast(float amax) {
    constexpr float FMAX4 = FMT == FP8DL_E4M3 ? 112.0f : 14336.0f;
    const float b = 0.25f * fmaxf(amax, 7.888609052210118e-31f), y = refined_rcp(b), q = FMAX4 * y;
    const float sc = amax > 0.0f ? __fmaf_rn(__fmaf_rn(-b, q, FMAX4), y, q) : 1.0f;
    return make_float2(sc, refined_rcp(sc));
}

// |v|, or 0 if v is not finite (blocks that hold infinities or NaN only).
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a <= 3.402823466e38f ? a : 0.0f;
}

// Called by all 256 threads of a block: the rows behind 128-row block `block` of the padded order (every
// group rounded up to a multiple of 128): first row and how many (0 behind the last group).  A
// thread takes up to four groups, so every offset is loaded at once and few instructions are issued
// (a search by every warp for itself cost twice the time with 200 groups).  Offsets in disorder may make
// groups overlap: a warp's 128 groups then have up to 2^30 blocks (every other group 2^24), and all 1024 up
// to 2^33.  So that 32 bits hold the sums, a warp counts for 2^28 at most, which is more than there are blocks to
// look for (2^25): the warps after it find nothing, as they should.  One thread at most answers; two answers
// could mix into rows behind the tensor's end.
__device__ __forceinline__ void group_of_block(const int32_t *offsets, int n_groups, int64_t rows, uint32_t block,
                                               int64_t &first_row, int &count) {
    __shared__ uint32_t warp_sum[8];
    __shared__ int32_t found[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (int)rows;
    const int per = (n_groups + 255) / 256, g0 = (int)threadIdx.x * per;
    int32_t first[4], length[4];
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        first[i] = length[i] = 0;
        if (i < per && g0 + i < n_groups) {
            first[i] = min(max(offsets[g0 + i], 0), n);
            length[i] = min(max(offsets[g0 + i + 1], first[i]), n) - first[i];
        }
        mine += ((uint32_t)length[i] + 127) >> 7;
    }
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 31) warp_sum[warp] = min(sum, 1u << 28);
    if (threadIdx.x == 0) found[1] = 0;
    __syncthreads();
    uint32_t at = block - (sum - mine);  // within this thread's blocks, if below `mine`
#pragma unroll
    for (int w = 0; w < 7; w++) at -= w < warp ? warp_sum[w] : 0;
    if (at < mine) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t blocks = ((uint32_t)length[i] + 127) >> 7;
            if (at < blocks) {
                found[0] = first[i] + (int32_t)(at * 128);
                found[1] = min(length[i] - (int32_t)(at * 128), 128);
                break;
            }
            at -= blocks;
        }
    }
    __syncthreads();
    first_row = found[0];
    count = found[1];
}

// Four fp32 values -> four codes, v0 in byte 0, the halves joined by the conversions themselves.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(float v0, float v1, float v2, float v3) {
    uint32_t r;
    if (FMT == FP8DL_E4M3)
        asm("{.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};}"
            : "=r"(r) : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
    else
        asm("{.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};}"
            : "=r"(r) : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
    return r;
}

// The largest of |a|, |b| and |c| (NaN does not count): one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float m;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// 32 x 32 -> 64 bits in one instruction: every extent fits 32 bits, no tensor's size does.
__device__ __forceinline__ uint64_t wide_mul(uint32_t a, uint32_t b) { return (uint64_t)a * b; }

// The padded order's 128-row blocks in shared memory, for kernels that look up many of them: before[g] blocks
// lie before group g, first[g] and length[g] are its rows.  Built once by a block of THREADS >= 256 threads, which meet
// at a barrier at its end; sums are limited as in group_of_block.
struct GroupTable {
    uint32_t *before;  // [n_groups + 1]
    int32_t *first, *length;
    uint32_t *warp_sum;  // [8]
};
inline size_t group_table_bytes(int n_groups) { return n_groups ? (3 * (size_t)n_groups + 9) * 4 : 0; }
__device__ __forceinline__ GroupTable group_table(void *smem, int n_groups) {
    uint32_t *p = static_cast<uint32_t *>(smem);
    return {p, reinterpret_cast<int32_t *>(p + n_groups + 1), reinterpret_cast<int32_t *>(p + 2 * n_groups + 1), p + 3 * n_groups + 1};
}

__device__ __forceinline__ void build_group_table(const GroupTable &t, const int32_t *offsets, int n_groups, int64_t rows) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (int)rows;
    const int per = (n_groups + 255) / 256, g0 = (int)threadIdx.x * per;
    uint32_t mine = 0;
    if (warp < 8) {
        for (int i = 0; i < per && g0 + i < n_groups; i++) {
            const int32_t f = min(max(offsets[g0 + i], 0), n), l = min(max(offsets[g0 + i + 1], f), n) - f;
            t.first[g0 + i] = f, t.length[g0 + i] = l;
            mine += ((uint32_t)l + 127) >> 7;
        }
    }
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 31 && warp < 8) t.warp_sum[warp] = min(sum, 1u << 28);
    __syncthreads();
    if (warp < 8) {
        uint32_t at = sum - mine;
        for (int w = 0; w < warp; w++) at += t.warp_sum[w];
        for (int i = 0; i < per && g0 + i < n_groups; i++) {
            t.before[g0 + i] = at;
            at += ((uint32_t)t.length[g0 + i] + 127) >> 7;
            if (g0 + i == n_groups - 1) t.before[n_groups] = at;
        }
    }
    __syncthreads();
}

// Block `block` of the table, block < before[n_groups]: its first row and how many.  `group`: where the search starts,
// 0 or what it left for an earlier block (before[group] <= block); a walk's next block is few groups on.
__device__ __forceinline__ void find_group(const GroupTable &t, uint32_t block, int &group, int64_t &first_row, int &count) {
    while (t.before[group + 1] <= block) group++;
    const int32_t skip = (int32_t)(block - t.before[group]) * 128;
    first_row = (int64_t)t.first[group] + skip;
    count = min(t.length[group] - skip, 128);
}

}  // namespace fp8dl
