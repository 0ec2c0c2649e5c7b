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

}  // namespace fp8dl
