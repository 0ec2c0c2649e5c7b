// block.cuh — what the block-scaled FP8 kernels share: the ragged groups' tables and the
// host checks of their arguments.
#pragma once

#include "common.cuh"

namespace fp8dl {

constexpr int kMaxGroups = 1024;

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

// Called by one whole warp: the rows behind 128-row block `block` of the padded order (every
// group rounded up to a multiple of 128): first row and how many (0 behind the last group).
__device__ __forceinline__ void group_of_block(const int32_t *offsets, int n_groups, int64_t rows, int64_t block,
                                               int64_t &first_row, int64_t &count) {
    const int lane = threadIdx.x & 31;
    int64_t before = 0;  // blocks of the groups already passed
    for (int g0 = 0; g0 < n_groups; g0 += 32) {
        int64_t first = 0, end = 0;
        if (g0 + lane < n_groups) group_rows(offsets, g0 + lane, rows, first, end);
        const int64_t blocks = (end - first + 127) / 128;
        const int64_t sum = before + warp_inclusive_sum(blocks, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, block < sum);
        if (hit) {
            const int src = __ffs((int)hit) - 1;
            const int64_t r = first + (block - (sum - blocks)) * 128;
            first_row = __shfl_sync(0xffffffffu, r, src);
            count = min(__shfl_sync(0xffffffffu, end, src) - first_row, (int64_t)128);
            return;
        }
        before = __shfl_sync(0xffffffffu, sum, 31);
    }
    first_row = 0;
    count = 0;
}

}  // namespace fp8dl
