// blockgemm.cu — block-scaled FP8 products on the tcgen05 tensor cores: one matrix, the
// ragged groups of an expert layer, and the groups' weight gradients.
//
//   D[m,n] = sum_b s[b] * P_b[m,n],  P_b = sum over the 128 k of block b of A[m,k] B[n,k],
//   s[b] = fl32(a_s[b][m] * b_s[b][n or n / 128])
//
// The factors differ from block to block along the reduction axis, so the tensor cores
// cannot sum over blocks: every P_b (four MMAs of K = 32) goes to its own tensor-memory
// buffer, and the epilogue warps multiply it into fp32 registers while the next block's MMAs
// run.  The tile's whole sum lives in registers; tensor memory only passes the blocks on.
#include <cuda_bf16.h>

#include "block.cuh"
#include "tc.cuh"

namespace fp8dl {

enum { BG_DENSE = 0, BG_ROWS = 1, BG_REDUCE = 2 };  // one matrix; ragged rows of A; ragged reduction

struct BlockGemmArgs {
    int kind;
    int64_t M, N, K;         // D is [M x N] (BG_REDUCE: per group); K = T for BG_REDUCE
    const float *a_s, *b_s;
    int64_t b_ld;            // entries of one block row of b_s
    const int32_t *offsets;
    int n_groups;
    const void *bias;
    int bias_dtype;          // -1 none
    void *D;
    int d_dtype;
    int32_t *status;
    uint32_t idesc;
    int along_n;     // tile order: bands along the columns (1) or rows (0) of D
    uint32_t band;
    uint32_t first, end;  // the launch's tiles (256 x 256)
};

// The groups' tables in shared memory: off = the offsets clamped to the tensor, in order
// (group g owns rows off[g] .. off[g+1]-1); pre[g] = units (row tiles, or token blocks) of
// the groups before g.
struct GroupTables {
    int32_t *off, *pre;
};
constexpr int kGroupTableBytes = 2 * 4 * (kMaxGroups + 4);

__device__ __forceinline__ GroupTables group_tables(uint8_t *smem) {
    int32_t *p = reinterpret_cast<int32_t *>(smem);
    return {p, p + kMaxGroups + 4};
}

// All threads of the block; `limit` caps the running sum (a reduction never reads past T).
__device__ __forceinline__ void build_groups(const GroupTables &t, const int32_t *offsets, int n_groups, int64_t rows,
                                             int unit, int64_t limit) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int64_t before = 0;
        int32_t from = 0;  // the running maximum: disordered offsets make empty groups, not overlaps
        if (lane == 0) {
            t.off[0] = from = (int32_t)min(max((int64_t)offsets[0], (int64_t)0), rows);
            t.pre[0] = 0;
        }
        from = __shfl_sync(0xffffffffu, from, 0);
        for (int g0 = 0; g0 < n_groups; g0 += 32) {
            const int g = g0 + lane;
            int32_t end = g < n_groups ? (int32_t)min(max((int64_t)offsets[g + 1], (int64_t)0), rows) : 0;
            end = max(end, from);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t u = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end = max(end, u);
            }
            int32_t first = __shfl_up_sync(0xffffffffu, end, 1);
            if (lane == 0) first = from;
            const int64_t sum = min(before + warp_inclusive_sum(((int64_t)end - first + unit - 1) / unit, lane), limit);
            if (g < n_groups) {
                t.off[g + 1] = end;
                t.pre[g + 1] = (int32_t)sum;
            }
            from = __shfl_sync(0xffffffffu, end, 31);
            before = __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    __syncthreads();
}

// The group that holds unit u: pre[g] <= u < pre[g + 1].
__device__ __forceinline__ int find_group(const GroupTables &t, int n_groups, uint32_t u) {
    int lo = 0, hi = n_groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((uint32_t)t.pre[mid] <= u)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Tiles in bands of `band` tiles along one dimension, which varies fastest inside a band: the
// tiles in flight form a block whose operand panels are shared through L2.  32-bit arithmetic
// (the host checks the tile count): a 64-bit division is a long subroutine, and every role of
// the kernel decodes every tile.
__device__ __forceinline__ void band_order(uint32_t tile, uint32_t tiles_m, uint32_t tiles_n, int along_n, uint32_t band,
                                           uint32_t &tm, uint32_t &tn) {
    const uint32_t inner = along_n ? tiles_n : tiles_m, outer = along_n ? tiles_m : tiles_n;
    band = min(band, inner);
    const uint32_t first = tile / (band * outer) * band;
    const uint32_t width = min(band, inner - first), r = tile - first * outer;
    const uint32_t o = r / width, i = first + r - o * width;
    tm = along_n ? o : i;
    tn = along_n ? i : o;
}

// One tile's work.
struct BlockTile {
    int64_t a_row, a_end;  // first row of A, and the end of the rows that are the tile's to write
    int64_t n0;            // first column of D
    int64_t b_row;         // its row of B
    int kb0, kbs;          // reduction blocks
    const float *b_s;      // factors of B of the tile's matrix
    int64_t d_row;         // a_row's row of D (BG_REDUCE: within all groups' matrices)
};

template <int TM, int TN>
__device__ __forceinline__ uint32_t block_tiles(const BlockGemmArgs &a, const GroupTables &t) {
    const uint32_t tiles_n = (uint32_t)((a.N + TN - 1) / TN), tiles_m = (uint32_t)((a.M + TM - 1) / TM);
    if (a.kind == BG_DENSE) return tiles_m * tiles_n;
    if (a.kind == BG_ROWS) return (uint32_t)t.pre[a.n_groups] * tiles_n;
    return (uint32_t)a.n_groups * tiles_m * tiles_n;
}

// Reduction blocks of a tile, or of share `share` of `split` (of one product only).
template <int TM, int TN>
__device__ __forceinline__ int block_tile_kbs(const BlockGemmArgs &a, const GroupTables &t, uint32_t tile, int split = 1,
                                              int share = 0) {
    if (a.kind != BG_REDUCE) {
        const int kbs = (int)((a.K + 127) / 128);
        return kbs * (share + 1) / split - kbs * share / split;
    }
    const uint32_t per = (uint32_t)((a.N + TN - 1) / TN) * (uint32_t)((a.M + TM - 1) / TM);
    const uint32_t g = tile / per;
    return t.pre[g + 1] - t.pre[g];
}

template <int TM, int TN>
__device__ __forceinline__ BlockTile block_tile(const BlockGemmArgs &a, const GroupTables &t, uint32_t tile, int split = 1,
                                                int share = 0) {
    const uint32_t tiles_n = (uint32_t)((a.N + TN - 1) / TN), tiles_m = (uint32_t)((a.M + TM - 1) / TM);
    BlockTile w;
    uint32_t tm, tn;
    const int kbs = (int)((a.K + 127) / 128);
    w.kb0 = 0;
    w.kbs = kbs;
    w.b_s = a.b_s;
    if (a.kind == BG_DENSE) {
        band_order(tile, tiles_m, tiles_n, a.along_n, a.band, tm, tn);
        w.a_row = w.d_row = (int64_t)tm * TM;
        w.a_end = a.M;
        w.n0 = w.b_row = (int64_t)tn * TN;
        w.kb0 = kbs * share / split;
        w.kbs = kbs * (share + 1) / split - w.kb0;
    } else if (a.kind == BG_ROWS) {
        const int g = find_group(t, a.n_groups, tile / tiles_n);
        band_order(tile - t.pre[g] * tiles_n, t.pre[g + 1] - t.pre[g], tiles_n, a.along_n, a.band, tm, tn);
        w.a_row = w.d_row = t.off[g] + (int64_t)tm * TM;
        w.a_end = t.off[g + 1];
        w.n0 = (int64_t)tn * TN;
        w.b_row = g * a.N + w.n0;
        w.b_s = a.b_s + (int64_t)g * kbs * a.b_ld;
    } else {
        const uint32_t g = tile / (tiles_m * tiles_n);
        band_order(tile - g * tiles_m * tiles_n, tiles_m, tiles_n, a.along_n, a.band, tm, tn);
        w.a_row = (int64_t)tm * TM;
        w.a_end = a.M;
        w.d_row = g * a.M + w.a_row;
        w.n0 = w.b_row = (int64_t)tn * TN;
        w.kb0 = t.pre[g];
        w.kbs = t.pre[g + 1] - t.pre[g];
    }
    return w;
}

// mbar_wait by a whole warp, with one answer for all its lanes: where a wait runs out, lanes that
// saw the abort and lanes that saw the phase complete would part, and the warp-wide operations
// that follow wait for lanes that never come.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
}

// One k-block of the pair's tile by one elected lane of a converged warp: four MMAs (K = 32 each,
// 32 bytes further into the swizzled rows, two descriptor units), the first one overwriting D,
// and the commits that hand the buffer to the epilogue and the stage to the producer.
__device__ __forceinline__ void umma_block_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t tfull,
                                                uint32_t empty, uint16_t ctas) {
    asm volatile(
        "{\n\t.reg .pred e, t, f;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 f, 0, 0;\n\t\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, f;\n\t"
        "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%4], %6;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], %6;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(tfull), "r"(empty), "h"(ctas)
        : "memory");
}

// The same on one CTA.
__device__ __forceinline__ void umma_block(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t tfull,
                                                uint32_t empty) {
    asm volatile(
        "{\n\t.reg .pred e, t, f;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.eq.u32 t, 0, 0;\n\tsetp.ne.u32 f, 0, 0;\n\t\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n\t"
        "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 4;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(tfull), "r"(empty)
        : "memory");
}

// Arrive on an mbarrier of this CTA from the lanes with `who`, without a branch.
__device__ __forceinline__ void arrive_if(uint32_t bar, bool who) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
                 "r"((uint32_t)who)
                 : "memory");
}

// The same on another CTA's mbarrier (a shared::cluster address).  What it announces is that this
// warp's tensor-memory loads are done, which tcgen05.wait::ld and the tcgen05 fence order; no
// ordinary memory is handed over, so the release stays within the CTA: a release at cluster
// scope waits for every global access in flight, once per k-block here (16384 x 16384 x 4096:
// 1.92 ms with it, 0.92 without).
__device__ __forceinline__ void arrive_remote_if(uint32_t cluster_addr, bool who) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];\n\t}" ::"r"(
            cluster_addr),
        "r"((uint32_t)who)
        : "memory");
}

// No use of r moves above this point: r belongs to a tcgen05.ld that has just been waited for.
template <int L>
__device__ __forceinline__ void regs_ready(uint32_t (&r)[L]) {
#pragma unroll
    for (int i = 0; i < L; i++) asm volatile("" : "+r"(r[i]));
}

// 32 lanes x 16 consecutive 32-bit columns of tensor memory.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Loads from shared memory of a CTA of the cluster (addresses from mapa_shared).
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// 4- and 16-byte copies from global to shared memory.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival on an mbarrier of this CTA when the thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ float load_bias1(const BlockGemmArgs &a, int64_t n) {
    return a.bias_dtype == FP8DL_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.bias)[n])
                                      : static_cast<const float *>(a.bias)[n];
}
__device__ __forceinline__ void store1(const BlockGemmArgs &a, int64_t at, float v) {
    if (a.d_dtype == FP8DL_BF16)
        static_cast<__nv_bfloat16 *>(a.D)[at] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(a.D)[at] = v;
}

// Sixteen consecutive columns' bias (in shared memory) added to the sums.
__device__ __forceinline__ void add_bias16(const float *bias, float2 (&v)[8]) {
#pragma unroll
    for (int g = 0; g < 4; g++) {
        const float4 u = *reinterpret_cast<const float4 *>(bias + 4 * g);
        v[2 * g] = __fadd2_rn(v[2 * g], make_float2(u.x, u.y));
        v[2 * g + 1] = __fadd2_rn(v[2 * g + 1], make_float2(u.z, u.w));
    }
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles on CTA pairs (tcgen05 cta_group::2, M 256, N 256, K 32).
//   warp 0      TMA producer: 128 rows of A and 128 of B per CTA and k-block
//   warp 1      the leader's MMA thread: four MMAs per block into one of two 256-column
//               tensor-memory buffers
//   warp 2      copies the blocks' factors into a shared-memory ring, blocks ahead
//   warp 3      adds "the factors are there" to "the MMAs are done", so that the epilogue waits
//               once per block: an mbarrier wait costs about 90 cycles even when it is over
//   warps 4-11  epilogue: warp w drains lane quarter w & 3 of column half (w - 4) / 4; a thread
//               holds one row x 128 columns of the sum (64 fp32 pairs)
// Every block's sums go to the epilogue and the buffer back to the MMAs, about 1270 cycles for the
// two buffers with an epilogue that does nothing: 638 a block, where the MMAs alone take 566.
// This kernel takes 742 (8192 x 8192 x 16384, 3050 TFLOP/s in a burst, 2630 under the power cap).  What got it there:
//   - a release at CTA scope on the leader's barrier (1.92 -> 0.92 ms at 16384 x 16384 x 4096),
//   - MMAs issued by one elected lane of the whole warp, without a branch on the lane (10 %),
//   - one wait per block for sums and factors, no branches in the loop (a wait costs 90 cycles),
//   - the buffer given back before the last three eighths of the multiply-adds,
//   - no spilled register in the kernels of whole tiles: 128 sums, 48 loads and 40 others are what 216
//     registers hold (the SPLIT kernels spill 20 bytes),
//   - the store, the tile's decoding and its bias out of the epilogue's way (see store_tile).
// A tile costs 0.376 us a block (0.545 with BROWS) and 2.0 us (2.2) beside them, for its first block's way through
// and its store (8192 x 4864, eight tiles a pair, K 512 to 8192): 14 % of it at K = 4096, 25 % at 2048.
// Tried and slower: 128 x 256 tiles on single CTAs (shared memory: 96 KB written and read a block,
// 750 cycles at 128 bytes a clock; 826-900 measured), 256 x 160 tiles with three buffers (the
// fixed 500 cycles an MMA thread spends per block weigh more: 990 per 256 columns).
// FP32 pipe: with 128 x 128 weight factors one packed multiply-add per two values (2.25 cycles each: 290
// a block); with factors per row of B (BROWS, weight gradients) one packed multiply more, and the
// columns' factors from shared memory: 1141 cycles a block.  Reading tensor memory in shapes that
// give a thread four rows and a quarter of the columns (16x128b, 16x256b: half and a quarter of
// the 32x32b shape's speed) needs fewer factors but came out no faster.
// ---------------------------------------------------------------------------
namespace bp {
constexpr int TM = 256, TN = 256, HALF = 128, BK = 128, STAGES = 4, BUFS = 2;
constexpr int A_BYTES = 128 * BK, B_ROWS = TN / 2, STAGE_BYTES = A_BYTES + B_ROWS * BK;
constexpr int THREADS = 384, EPI_WARPS = 8;
constexpr int REGS_LAUNCH = 168, REGS_IO = 72, REGS_EPI = 216;  // 128 * 72 + 256 * 216 = 384 * 168
static_assert(128 * REGS_IO + 256 * REGS_EPI <= THREADS * REGS_LAUNCH, "register split");
constexpr int TMEM_COLS = 512;
// The factors of the next blocks, FB blocks per ring slot: 128 of A's, then one per column half
// of B's (padded to 16 bytes), or, BROWS, 256.
template <bool BROWS>
struct Ring {
    static constexpr int FB = BROWS ? 2 : 4, SLOTS = 2, BLOCK = 128 + (BROWS ? TN : 4);
    static constexpr int SLOT = FB * BLOCK;
};
constexpr int RING_BYTES = Ring<true>::SLOTS * Ring<true>::SLOT * 4;
// One warp's 32 rows x 256 bytes of D on their way out, as two boxes of 128 bytes.
constexpr int OUT_BOX = 32 * 128, OUT_WARP = 2 * OUT_BOX, OUT_BYTES = EPI_WARPS * OUT_WARP;
// What the epilogue needs of a tile, decoded by the relay warp (the decoding's divisions took
// 600-900 cycles at each tile's end): the CTA's first row of D, how many rows are its to write,
// the first column.  The relay writes a tile's entry at most five blocks ahead of the last one
// that the epilogue has loaded (it waits for block i - 3 before it gets to block i, whose MMAs
// waited for the release of block i - 5): five tiles if each has one block.  Tiles without
// blocks take no entry.
struct TileOut {
    int64_t d_row, n0;
    int64_t rows;
};
constexpr int TILE_RING = 8;
constexpr int BIAS_BYTES = TILE_RING * TN * 4;  // and the tile's bias as fp32, if there is one
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + OUT_BYTES + 1024 + RING_BYTES + BIAS_BYTES + kGroupTableBytes + 1024;
static_assert(SMEM_BYTES <= 227 * 1024 && Ring<false>::SLOTS * Ring<false>::SLOT * 4 <= RING_BYTES, "shared memory");
}  // namespace bp

__device__ __forceinline__ bp::TileOut tile_out_of(const BlockTile &w, uint32_t rank) {
    return {w.d_row + rank * 128, w.n0, w.a_end - (w.a_row + rank * 128)};
}

// One warp's 32 rows x 128 columns of D (lane = row): rounded once, laid out in shared memory as
// boxes of 128 bytes a row (16-byte chunk j of row r at j ^ (r & 7): the TMA's 128-byte
// swizzle, free of bank conflicts) and stored by the TMA while the next tile is summed.  All
// CTAs finish their tiles together, so stores that the epilogue waits for come in bursts at the
// speed of L2: with stores from registers, or through 4 KB a warp, a tile's end cost 4000-7200
// cycles, an eighth to a fifth of a tile with K = 4096.  Rows at a ragged group's end are
// written by the warp itself.  The box is free once the TMA has read it: the wait is at the
// next tile's end (two boxes hold 128 columns of bf16; fp32 takes two turns).
__device__ __forceinline__ void store_tile(const BlockGemmArgs &a, const CUtensorMap *tmap_d, uint8_t *stage, int lane,
                                           int64_t d_row, int rows, int64_t n0, const float *bias,
                                           float2 (&acc)[64]) {
    using namespace bp;
    const bool bf = a.d_dtype == FP8DL_BF16;
    const int esz = bf ? 2 : 4;
    uint8_t *mine = stage + lane * 128;
    const int swz = lane & 7;
    auto flush = [&](uint8_t *box, int64_t n) {  // a box whose first column is n
        if (rows == 32) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && n < a.N) {
                tma_store_2d(tmap_d, smem_u32(box), (int32_t)(n * esz), (int32_t)d_row);
                bulk_commit();
            }
        } else {
            __syncwarp();
            const int sub = lane >> 3, ch = lane & 7;
            uint8_t *to = static_cast<uint8_t *>(a.D) + ((d_row + sub) * a.N + n) * esz + 16 * ch;
            const bool ok = n + ch * (16 / esz) < a.N;
            for (int r = sub; r < rows; r += 4, to += 4 * a.N * esz)
                if (ok) *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(box + r * 128 + ((ch ^ (r & 7)) << 4));
            __syncwarp();
        }
    };
    auto wait_free = [&] {
        if (lane == 0) bulk_wait_read();
        __syncwarp();
    };
    wait_free();
#pragma unroll
    for (int c = 0; c < 8; c++) {
        float2 v[8];
#pragma unroll
        for (int p = 0; p < 8; p++) v[p] = acc[8 * c + p];
        if (a.bias_dtype >= 0) add_bias16(bias + 16 * c, v);
        if (bf) {
#pragma unroll
            for (int g = 0; g < 2; g++) {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[4 * g + q].x, v[4 * g + q].y);
                    w[q] = *reinterpret_cast<const uint32_t *>(&h);
                }
                *reinterpret_cast<uint4 *>(mine + (c >> 2) * OUT_BOX + (((2 * (c & 3) + g) ^ swz) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
            if ((c & 3) == 3) flush(stage + (c >> 2) * OUT_BOX, n0 + 64 * (c >> 2));
        } else {
            if (c == 4) wait_free();
#pragma unroll
            for (int g = 0; g < 4; g++)
                *reinterpret_cast<float4 *>(mine + ((c >> 1) & 1) * OUT_BOX + (((4 * (c & 1) + g) ^ swz) << 4)) =
                    make_float4(v[2 * g].x, v[2 * g].y, v[2 * g + 1].x, v[2 * g + 1].y);
            if (c & 1) flush(stage + ((c >> 1) & 1) * OUT_BOX, n0 + 32 * (c >> 1));
        }
    }
}

// Eight columns' factors from shared memory, in program order with the other volatile accesses.
__device__ __forceinline__ void load_factors(float4 (&f)[2], const float *p) {
#pragma unroll
    for (int i = 0; i < 2; i++)
        asm volatile("ld.volatile.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(f[i].x), "=f"(f[i].y), "=f"(f[i].z), "=f"(f[i].w)
                     : "r"(smem_u32(p + 4 * i)));
}

// acc[C .. C+L) += r * factor: the factor sc, or (BROWS) sc times the columns' own, of which f0 and f1
// hold the next sixteen; they are loaded sixteen columns ahead of their use, which with two
// warps a scheduler hides most of it (1205 cycles a block with the loads at their use, 1141 so,
// 907 if there were none).
template <bool BROWS, int C, int L>
__device__ __forceinline__ void add_block(float2 (&acc)[64], const uint32_t (&r)[L], float2 sc, const float *fb,
                                          float4 (&f0)[2], float4 (&f1)[2]) {
#pragma unroll
    for (int g = 0; g < L / 8; g++) {
        float2 m[4] = {sc, sc, sc, sc};
        if constexpr (BROWS) {
            float4(&f)[2] = ((C / 8 + g) & 1) ? f1 : f0;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                m[2 * i] = __fmul2_rn(sc, make_float2(f[i].x, f[i].y));
                m[2 * i + 1] = __fmul2_rn(sc, make_float2(f[i].z, f[i].w));
            }
            if (C + 8 * g + 16 < bp::HALF) load_factors(f, fb + C + 8 * g + 16);
        }
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int j = 8 * g + 2 * k;
            float2 &a = acc[(C + j) / 2];
            a = __ffma2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), m[k], a);
        }
    }
}

// A split tile's end: one thread's row, the 128 / SPLIT columns that its share stores; the shares' sums
// (sixteen bytes at 512 k from `sums`, in the CTAs of the same rank of every pair) are added in
// order.  Sixteen columns' loads are under way at once: one at a time their latency
// made the join as long as the products it saved.
template <int SPLIT>
__device__ __forceinline__ void join_shares(const BlockGemmArgs &a, uint32_t sums, uint32_t rank, int share, int64_t row,
                                            int64_t n0, const float *bias) {
    constexpr int PIECES = 32 / SPLIT;
    uint32_t from[SPLIT];
#pragma unroll
    for (int o = 0; o < SPLIT; o++) from[o] = mapa_shared(sums + 512 * PIECES * share, 2 * o + rank);
    for (int k = 0; k < PIECES; k += 4) {
        const int col = 4 * (PIECES * share + k);
        const int64_t n = n0 + col;
        if (n >= a.N) break;
        float4 v[SPLIT][4];
#pragma unroll
        for (int o = 0; o < SPLIT; o++)
#pragma unroll
            for (int i = 0; i < 4; i++) v[o][i] = ld_cluster_f32x4(from[o] + 512 * (k + i));
        float y[16];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float4 s = v[0][i];
#pragma unroll
            for (int o = 1; o < SPLIT; o++) s.x += v[o][i].x, s.y += v[o][i].y, s.z += v[o][i].z, s.w += v[o][i].w;
            if (a.bias_dtype >= 0) {
                const float4 u = *reinterpret_cast<const float4 *>(bias + col + 4 * i);
                s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
            }
            y[4 * i] = s.x, y[4 * i + 1] = s.y, y[4 * i + 2] = s.z, y[4 * i + 3] = s.w;
        }
        if (a.d_dtype == FP8DL_BF16) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
            uint4 *d = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.D) + row * a.N + n);
            d[0] = make_uint4(w[0], w[1], w[2], w[3]);
            d[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(a.D) + row * a.N + n);
#pragma unroll
            for (int i = 0; i < 4; i++) d[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        }
    }
}

// SPLIT: the cluster's pairs share a tile (a kernel of its own: with the shares as run-time numbers
// the others lost 3 %).
template <bool BROWS, bool SPLIT>
__global__ void __launch_bounds__(bp::THREADS, 1)
    block_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                      const __grid_constant__ CUtensorMap tmap_d, const BlockGemmArgs args) {
    using namespace bp;
    using R = Ring<BROWS>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
    uint8_t *out_stage = smem + STAGES * STAGE_BYTES;
    uint8_t *bar_area = out_stage + OUT_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(bar_area);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;
    uint64_t *tempty = tfull + BUFS;
    uint64_t *ffull = tempty + BUFS;
    uint64_t *fempty = ffull + R::SLOTS;
    TileOut *tile_out = reinterpret_cast<TileOut *>(bar_area + 512);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fempty + R::SLOTS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *ring = reinterpret_cast<float *>(bar_area + 1024);
    float *bias_ring = reinterpret_cast<float *>(bar_area + 1024 + RING_BYTES);
    const GroupTables tab = group_tables(bar_area + 1024 + RING_BYTES + BIAS_BYTES);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // A cluster is one pair, or (SPLIT) several that share a tile, each with a part of its blocks.
    const uint32_t cluster_rank = cluster_ctarank(), cluster_size = SPLIT ? cluster_nctarank() : 2u;
    const uint32_t rank = SPLIT ? cluster_rank & 1 : cluster_rank, leader_rank = SPLIT ? cluster_rank & ~1u : 0u;
    const bool leader = rank == 0;
    const int split = SPLIT ? (int)(cluster_size >> 1) : 1, share = SPLIT ? (int)(cluster_rank >> 1) : 0;
    const uint32_t pair = args.first + blockIdx.x / cluster_size, npairs = gridDim.x / cluster_size;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < BUFS; a++) {
            mbar_init(smem_u32(&tfull[a]), 2);  // the MMAs' commit, and the relay's word for the factors
            mbar_init(smem_u32(&tempty[a]), 2 * EPI_WARPS);
        }
        for (int a = 0; a < R::SLOTS; a++) {
            mbar_init(smem_u32(&ffull[a]), 32);  // every lane of the copying warp
            mbar_init(smem_u32(&fempty[a]), EPI_WARPS);
        }
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_map(&tmap_a);
        tma_prefetch_map(&tmap_b);
        tma_prefetch_map(&tmap_d);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are initialised before any signal crosses
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();
    if (args.kind == BG_ROWS) build_groups(tab, args.offsets, args.n_groups, args.M, TM, 0x7fffffffll);
    if (args.kind == BG_REDUCE)
        build_groups(tab, args.offsets, args.n_groups, 0x7fffffffll, 128, args.K / 128);
    const uint32_t tiles = min(block_tiles<TM, TN>(args, tab), args.end);

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_IO));
        if (warp == 0 && lane == 0) {  // ------------------------------------- producer (both CTAs)
            int s = 0;
            uint32_t ph = 0;
            int64_t issued = 0;
            bool ok = true;
            for (uint32_t tile = pair; tile < tiles && ok; tile += npairs) {
                const BlockTile w = block_tile<TM, TN>(args, tab, tile, split, share);
                const int32_t ra = (int32_t)(w.a_row + rank * 128), rb = (int32_t)(w.b_row + rank * B_ROWS);
                for (int kb = 0; kb < w.kbs; kb++) {
                    if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    // both CTAs' loads complete on the leader's barrier
                    const uint32_t fb = smem_u32(&full[s]), lb = mapa_shared(fb, leader_rank);
                    const uint32_t sa = smem_u32(smem + s * STAGE_BYTES);
                    if (leader) mbar_expect_tx(fb, 2 * STAGE_BYTES);
                    tma_load_2d_pair(sa, &tmap_a, lb, (w.kb0 + kb) * BK, ra);
                    tma_load_2d_pair(sa + A_BYTES, &tmap_b, lb, (w.kb0 + kb) * BK, rb);
                    issued++;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok && leader)
                for (int64_t i = issued - 1; i >= 0 && i >= issued - STAGES; i--)
                    mbar_drain(smem_u32(&full[i % STAGES]), (uint32_t)((i / STAGES) & 1));
        } else if (warp == 1 && leader) {  // ----------------------------------- MMA issuer (leader only)
            // The whole warp runs the loop and one elected lane issues, so that the operands are the same
            // for all lanes and no branch on the lane stands before an MMA, on a scheduler shared with
            // two epilogue warps: 10 % of the kernel.
            int s = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true, any = false;
            uint32_t last_bar = 0, last_par = 0;
            const SDesc desc0 = sdesc_k_sw128_split(smem_u32(smem));
            for (uint32_t tile = pair; tile < tiles && ok; tile += npairs) {
                const int kbs = block_tile_kbs<TM, TN>(args, tab, tile, split, share);
                for (int kb = 0; kb < kbs; kb++) {
                    // the operands first: they are there early, the buffer comes back last
                    if (!warp_wait(smem_u32(&full[s]), ph, abort_flag, args.status) ||
                        !warp_wait(smem_u32(&tempty[buf]), bph ^ 1, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t lo_a = desc0.lo + (uint32_t)s * (STAGE_BYTES >> 4);
                    umma_block_pair(tmem_base + (uint32_t)(buf * TN), sdesc_join(lo_a, desc0.hi),
                                    sdesc_join(lo_a + (A_BYTES >> 4), desc0.hi), args.idesc, smem_u32(&tfull[0]) + 8 * buf,
                                    smem_u32(&empty[0]) + 8 * s, (uint16_t)(0x3u << leader_rank));
                    any = true;
                    last_bar = smem_u32(&empty[s]);
                    last_par = ph;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                    if (++buf == BUFS) {
                        buf = 0;
                        bph ^= 1;
                    }
                }
            }
            if (!ok && any) mbar_drain(last_bar, last_par);
        } else if (warp == 2) {  // --------------------------------------------- factors (both CTAs)
            // Rows and columns outside the matrix take a valid address: their sums are not stored.
            int slot = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (uint32_t tile = pair; tile < tiles && ok; tile += npairs) {
                const BlockTile w = block_tile<TM, TN>(args, tab, tile, split, share);
                const int64_t row = w.a_row + rank * 128 + lane;
                const float *pa = args.a_s + (int64_t)w.kb0 * args.M + w.a_row;
                const float *pb = w.b_s + (int64_t)w.kb0 * args.b_ld + (BROWS ? w.n0 : w.n0 >> 7);
                int oa[4], ob[2];  // from those: four rows, and (BROWS) two times four columns, or one block
#pragma unroll
                for (int j = 0; j < 4; j++) oa[j] = row + 32 * j < w.a_end ? (int)(rank * 128) + lane + 32 * j : 0;
                if (BROWS) {
#pragma unroll
                    for (int h = 0; h < 2; h++) ob[h] = w.n0 + 128 * h + 4 * lane < args.N ? 128 * h + 4 * lane : 0;
                } else {
                    ob[0] = (w.n0 >> 7) + lane < args.b_ld ? lane : 0;
                }
                for (int kb = 0; kb < w.kbs; kb += R::FB) {
                    if (!warp_wait(smem_u32(&fempty[slot]), ph ^ 1, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    uint32_t dst = smem_u32(ring + slot * R::SLOT);
                    for (int f = 0; f < R::FB && kb + f < w.kbs; f++, dst += 4 * R::BLOCK) {
#pragma unroll
                        for (int j = 0; j < 4; j++) cp_async4(dst + 4 * (32 * j + lane), pa + oa[j]);
                        if (BROWS) {
                            cp_async16(dst + 512 + 16 * lane, pb + ob[0]);
                            cp_async16(dst + 1024 + 16 * lane, pb + ob[1]);
                        } else if (lane < 2) {
                            cp_async4(dst + 512 + 4 * lane, pb + ob[0]);
                        }
                        pa += args.M;
                        pb += args.b_ld;
                    }
                    cp_async_arrive(smem_u32(&ffull[slot]));
                    if (++slot == R::SLOTS) {
                        slot = 0;
                        ph ^= 1;
                    }
                }
            }
            cp_async_wait_all();
        } else if (warp == 3) {  // --------------------------------------------- relay (both CTAs)
            // A block reaches the epilogue in one wait: its buffer is full when the MMAs have
            // committed and this warp, which waits for the factors, has said so.  It arrives for
            // a block once the buffer's last block is complete, well before the MMAs do.
            int slot = 0, buf = 0;
            uint32_t fph = 0, bph = 0;
            bool ok = true;
            uint32_t seq = 0;
            for (uint32_t tile = pair; tile < tiles && ok; tile += npairs) {
                const BlockTile w = block_tile<TM, TN>(args, tab, tile, split, share);
                const int kbs = w.kbs;
                if (kbs > 0) {  // handed over with the first block's arrival
                    if (lane == 0) tile_out[seq % TILE_RING] = tile_out_of(w, rank);
                    if (args.bias_dtype >= 0) {
#pragma unroll
                        for (int j = 0; j < TN / 32; j++)
                            if (w.n0 + 32 * j + lane < args.N)
                                bias_ring[seq % TILE_RING * TN + 32 * j + lane] = load_bias1(args, w.n0 + 32 * j + lane);
                    }
                    __syncwarp();
                    seq++;
                }
                for (int kb = 0; kb < kbs; kb++) {
                    if (kb % R::FB == 0) {
                        ok = warp_wait(smem_u32(&ffull[slot]), fph, abort_flag, args.status);
                        if (++slot == R::SLOTS) {
                            slot = 0;
                            fph ^= 1;
                        }
                    }
                    if (!ok || !(ok = warp_wait(smem_u32(&tfull[buf]), bph ^ 1, abort_flag, args.status))) break;
                    if (lane == 0) mbar_arrive(smem_u32(&tfull[buf]));
                    __syncwarp();
                    if (++buf == BUFS) {
                        buf = 0;
                        bph ^= 1;
                    }
                }
            }
        }
    } else {  // ------------------------------------------------------------ epilogue (both CTAs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t taddr0 = tmem_base + (uint32_t)(HALF * half) + ((uint32_t)(32 * q) << 16);
        uint8_t *stage = out_stage + (warp - 4) * OUT_WARP;
        const float *my_a = ring + 32 * q + lane, *my_b = ring + 128 + (BROWS ? HALF : 1) * half;
        const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), leader_rank);
        int slot = 0, buf = 0;
        uint32_t bph = 0, seq = 0;  // seq: tiles with blocks so far, as the relay counts them
        for (uint32_t tile = pair; tile < tiles; tile += npairs) {
            const int kbs = block_tile_kbs<TM, TN>(args, tab, tile, split, share);
            float2 acc[64];
#pragma unroll
            for (int p = 0; p < 64; p++) acc[p] = make_float2(0.0f, 0.0f);
            bool ok = true;
            for (int kb = 0; ok && kb < kbs; kb++) {
                // after a wait that ran out this block's sums are garbage and the loop ends
                ok = warp_wait(smem_u32(&tfull[0]) + 8 * buf, bph, abort_flag, args.status);
                tc_fence_after();
                const uint32_t ta = taddr0 + (uint32_t)(buf * TN);
                // Columns 0-31, 32-47, 48-79, 80-95, 96-127 through two sets of registers (48 beside
                // the 128 sums: with 64 the compiler spills).  The buffer goes back as soon as the last
                // ones are loaded, before their multiply-adds and those of columns 80-95.
                uint32_t ra[32], rb[16];
                tmem_ld_32x32b_x32(ta, ra);
                tmem_ld_32x32b_x16(ta + 32, rb);
                const int at = slot * R::SLOT + (kb % R::FB) * R::BLOCK;
                const float *fb = my_b + at;  // BROWS: the block's column factors
                const float2 sc = f2(BROWS ? my_a[at] : __fmul_rn(my_a[at], fb[0]));
                float4 f0[2], f1[2];
                if (BROWS) {
                    load_factors(f0, fb);
                    load_factors(f1, fb + 8);
                }
                tmem_ld_wait_regs(ra);
                regs_ready(rb);
                add_block<BROWS, 0>(acc, ra, sc, fb, f0, f1);
                tmem_ld_32x32b_x32(ta + 48, ra);
                add_block<BROWS, 32>(acc, rb, sc, fb, f0, f1);
                tmem_ld_32x32b_x16(ta + 80, rb);
                tmem_ld_wait_regs(ra);
                regs_ready(rb);
                add_block<BROWS, 48>(acc, ra, sc, fb, f0, f1);
                tmem_ld_32x32b_x32(ta + 96, ra);
                tmem_ld_wait_regs(ra);
                tc_fence_before();
                __syncwarp();
                arrive_remote_if(tempty0 + 8 * buf, lane == 0);
                add_block<BROWS, 80>(acc, rb, sc, fb, f0, f1);
                add_block<BROWS, 96>(acc, ra, sc, fb, f0, f1);
                const bool last = kb % R::FB == R::FB - 1 || kb == kbs - 1;  // of the factor slot
                __syncwarp();
                arrive_if(smem_u32(&fempty[0]) + 8 * slot, lane == 0 && last);
                slot = last ? (slot + 1) % R::SLOTS : slot;
                bph ^= buf == BUFS - 1;
                buf = buf == BUFS - 1 ? 0 : buf + 1;
            }
            if (SPLIT) {
                // this share's sums, where the operands were (all its MMAs are done): sixteen bytes of
                // lane l's row at 512 k + 16 l, free of bank conflicts for the writer and the readers
#pragma unroll
                for (int k = 0; k < 32; k++)
                    *reinterpret_cast<float4 *>(smem + (warp - 4) * 16384 + 512 * k + 16 * lane) =
                        make_float4(acc[2 * k].x, acc[2 * k].y, acc[2 * k + 1].x, acc[2 * k + 1].y);
                break;  // the cluster's one tile; joined below
            }
            if (!ok) break;
            const TileOut out = kbs > 0 ? tile_out[seq % TILE_RING]
                                        : tile_out_of(block_tile<TM, TN>(args, tab, tile, split, share), rank);  // nothing to sum: zeros
            const int64_t rows = out.rows - 32 * q, n0 = out.n0 + HALF * half;
            if (rows > 0 && n0 < args.N)
                store_tile(args, &tmap_d, stage, lane, out.d_row + 32 * q, (int)min(rows, (int64_t)32), n0,
                           bias_ring + seq % TILE_RING * TN + HALF * half, acc);
            seq += kbs > 0;
        }
        if (lane == 0) bulk_wait_all();
    }

    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (SPLIT) {
        cluster_sync();  // every share's sums are there
        if (warp >= 4 && pair < tiles) {
            const TileOut out = tile_out[0];
            const int q = warp & 3, half = (warp - 4) >> 2;
            const uint8_t *sums = smem + (warp - 4) * 16384 + 16 * lane;
            if (32 * q + lane < out.rows && split == 2)
                join_shares<2>(args, smem_u32(sums), rank, share, out.d_row + 32 * q + lane, out.n0 + HALF * half,
                               bias_ring + HALF * half);
            if (32 * q + lane < out.rows && split == 4)
                join_shares<4>(args, smem_u32(sums), rank, share, out.d_row + 32 * q + lane, out.n0 + HALF * half,
                               bias_ring + HALF * half);
        }
        __syncwarp();
    }
    cluster_sync();  // the peers' shared memory and TMEM stay live until the cluster is done
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// Few rows of A (decoding, small groups of tokens): the weight takes the MMA's M side, 128 of its
// rows a tile, and BT rows of A (16, 32 or 64) its N side, so that a tile computes little
// more than the rows there are and the kernel runs at the speed the weight arrives.
//   warp 0      TMA producer: 128 weight rows and BT rows of A per k-block
//   warp 1      MMA thread: four MMAs (M 128, N BT, K 32) per block into one of NB buffers
//   warp 2      multiplies the blocks' factors (one per row of A with the weight's) into a ring
//   warp 3      relay: a block's one signal to the epilogue, as in the tile kernel
//   warps 4-7   epilogue: a thread holds one weight row x BT rows of A
// Split: where the tiles alone would leave SMs without a weight to read, the CTAs of a cluster
// share a tile, each with a contiguous part of the blocks, and add their sums in rank order
// through distributed shared memory: no workspace, one launch, the same bits every time.
// Two CTAs fit an SM: one's start and end hide behind the other's loads.
// ---------------------------------------------------------------------------
namespace bf {
constexpr int TW = 128, BK = 128, MOST_SHARES = 6;  // CTAs of a weight tile
template <int BT>
struct Shape {
    static constexpr int EPI_WARPS = 4, THREADS = 32 * (4 + EPI_WARPS);
    static constexpr int STAGE_BYTES = TW * BK + BT * BK;
    static constexpr int STAGES = BT <= 32 ? 5 : 4;
    static constexpr int NB = 4, TMEM_COLS = NB * BT;
    static constexpr int RING = 8, SLOT = BT;                  // the factors of eight blocks, BT each
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + RING * SLOT * 4 + kGroupTableBytes + 1024;
    static_assert(2 * SMEM_BYTES <= 227 * 1024 && 2 * TMEM_COLS <= 512, "two CTAs per SM");
    static_assert(STAGES * STAGE_BYTES >= BT * TW * 4, "the sums of a split tile take the operands' place");
};
}  // namespace bf

// A split tile's end: the cluster's sums (row t of A at 512 t bytes from `sums` in every CTA) are added in
// rank order; rank r stores every split-th row, four columns a thread, the loads of all ranks
// under way at once.
__device__ __forceinline__ void join_few(const BlockGemmArgs &a, uint32_t sums, int split, int rank, const BlockTile &w,
                                         int rows) {
    const int col = 4 * (threadIdx.x & 31);
    const int64_t n = w.n0 + col;
    if (n >= a.N) return;
    for (int t = split * (int)(threadIdx.x >> 5) + rank; t < rows; t += split * 8) {
        float4 v[bf::MOST_SHARES];
#pragma unroll
        for (int o = 0; o < bf::MOST_SHARES; o++)
            if (o < split) v[o] = ld_cluster_f32x4(mapa_shared(sums, o) + 4 * (t * bf::TW + col));
#pragma unroll
        for (int o = 1; o < bf::MOST_SHARES; o++)
            if (o < split) v[0].x += v[o].x, v[0].y += v[o].y, v[0].z += v[o].z, v[0].w += v[o].w;
        if (a.bias_dtype >= 0)
            v[0].x += load_bias1(a, n), v[0].y += load_bias1(a, n + 1), v[0].z += load_bias1(a, n + 2), v[0].w += load_bias1(a, n + 3);
        const int64_t at = (w.d_row + t) * a.N + n;
        if (a.d_dtype == FP8DL_BF16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0].x, v[0].y), hi = __floats2bfloat162_rn(v[0].z, v[0].w);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.D) + at) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(a.D) + at) = v[0];
        }
    }
}

template <int BT>
__global__ void __launch_bounds__(bf::Shape<BT>::THREADS, 2)
    block_gemm_few_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                          const BlockGemmArgs args) {
    using namespace bf;
    using S = Shape<BT>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
    uint8_t *bar_area = smem + S::STAGES * S::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(bar_area);
    uint64_t *empty = full + S::STAGES;
    uint64_t *tfull = empty + S::STAGES;
    uint64_t *tempty = tfull + S::NB;
    uint64_t *ffull = tempty + S::NB;
    uint64_t *fempty = ffull + S::RING;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fempty + S::RING);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *ring = reinterpret_cast<float *>(bar_area + 1024);
    const GroupTables tab = group_tables(bar_area + 1024 + S::RING * S::SLOT * 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t split = cluster_nctarank(), rank = cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::STAGES; i++) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), 1);
        }
        for (int i = 0; i < S::NB; i++) {
            mbar_init(smem_u32(&tfull[i]), 2);  // the MMAs' commit, and the relay's word for the factors
            mbar_init(smem_u32(&tempty[i]), S::EPI_WARPS);
        }
        for (int i = 0; i < S::RING; i++) {
            mbar_init(smem_u32(&ffull[i]), 1);
            mbar_init(smem_u32(&fempty[i]), S::EPI_WARPS);
        }
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_map(&tmap_a);
        tma_prefetch_map(&tmap_b);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), S::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();
    if (args.kind == BG_ROWS) build_groups(tab, args.offsets, args.n_groups, args.M, BT, 0x7fffffffll);
    const uint32_t tiles = block_tiles<BT, TW>(args, tab);
    const uint32_t tile0 = blockIdx.x / split, step = gridDim.x / split;  // a split launch has a tile per cluster at most
    const int all_kbs = (int)((args.K + BK - 1) / BK);
    const int kb0 = (int)((int64_t)all_kbs * rank / split), kb1 = (int)((int64_t)all_kbs * (rank + 1) / split);

    if (warp == 0) {
        if (lane == 0) {  // ---------------------------------------------------- producer
            int s = 0;
            uint32_t ph = 0;
            int64_t issued = 0;
            bool ok = true;
            for (uint32_t tile = tile0; tile < tiles && ok; tile += step) {
                const BlockTile w = block_tile<BT, TW>(args, tab, tile);
                for (int kb = kb0; kb < kb1; kb++) {
                    if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&full[s]), dst = smem_u32(smem + s * S::STAGE_BYTES);
                    mbar_expect_tx(fb, S::STAGE_BYTES);
                    tma_load_2d(dst, &tmap_b, fb, kb * BK, (int32_t)w.b_row);
                    tma_load_2d(dst + TW * BK, &tmap_a, fb, kb * BK, (int32_t)w.a_row);
                    issued++;
                    if (++s == S::STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok)
                for (int64_t i = issued - 1; i >= 0 && i >= issued - S::STAGES; i--)
                    mbar_drain(smem_u32(&full[i % S::STAGES]), (uint32_t)((i / S::STAGES) & 1));
        }
    } else if (warp == 1) {  // ------------------------------------------------- MMA issuer
        int s = 0, buf = 0;
        uint32_t ph = 0, bph = 0;
        bool ok = true, any = false;
        uint32_t last_bar = 0, last_par = 0;
        const SDesc desc0 = sdesc_k_sw128_split(smem_u32(smem));
        for (uint32_t tile = tile0; tile < tiles && ok; tile += step) {
            for (int kb = kb0; kb < kb1; kb++) {
                if (!warp_wait(smem_u32(&full[s]), ph, abort_flag, args.status) ||
                    !warp_wait(smem_u32(&tempty[buf]), bph ^ 1, abort_flag, args.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t lo = desc0.lo + (uint32_t)s * (S::STAGE_BYTES >> 4);
                umma_block(tmem_base + (uint32_t)(buf * BT), sdesc_join(lo, desc0.hi),
                           sdesc_join(lo + (TW * BK >> 4), desc0.hi), args.idesc, smem_u32(&tfull[0]) + 8 * buf,
                           smem_u32(&empty[0]) + 8 * s);
                any = true;
                last_bar = smem_u32(&empty[s]);
                last_par = ph;
                if (++s == S::STAGES) {
                    s = 0;
                    ph ^= 1;
                }
                if (++buf == S::NB) {
                    buf = 0;
                    bph ^= 1;
                }
            }
        }
        if (!ok && any) mbar_drain(last_bar, last_par);
    } else if (warp == 2) {  // ------------------------------------------------- factors
        // The two factors of every row and block, multiplied once for all the weight's rows.  Four
        // blocks' are loaded at a time, four blocks before they are needed.
        constexpr int PER = (BT + 31) / 32, AHEAD = 4;
        int slot = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (uint32_t tile = tile0; tile < tiles && ok; tile += step) {
            const BlockTile w = block_tile<BT, TW>(args, tab, tile);
            const float *pa = args.a_s + (int64_t)kb0 * args.M + w.a_row;
            const float *pb = w.b_s + (int64_t)kb0 * args.b_ld + (w.n0 >> 7);
            float fa[AHEAD][PER], fb[AHEAD], na[AHEAD][PER], nb[AHEAD];
            auto load = [&](int kb, float(&a)[AHEAD][PER], float(&b)[AHEAD]) {
#pragma unroll
                for (int i = 0; i < AHEAD; i++, pa += args.M, pb += args.b_ld) {
                    b[i] = kb + i < kb1 ? __ldg(pb) : 0.0f;
#pragma unroll
                    for (int t = 0; t < PER; t++)  // rows behind the last: zeros, not stored
                        a[i][t] = kb + i < kb1 && 32 * t + lane < BT && w.a_row + 32 * t + lane < w.a_end
                                      ? __ldg(pa + 32 * t + lane)
                                      : 0.0f;
                }
            };
            load(kb0, fa, fb);
            for (int kb = kb0; kb < kb1 && ok; kb += AHEAD) {
                load(kb + AHEAD, na, nb);
#pragma unroll
                for (int i = 0; i < AHEAD; i++) {
                    if (kb + i >= kb1 || !(ok = warp_wait(smem_u32(&fempty[slot]), ph ^ 1, abort_flag, args.status))) break;
#pragma unroll
                    for (int t = 0; t < PER; t++)
                        if (32 * t + lane < BT) ring[slot * S::SLOT + 32 * t + lane] = __fmul_rn(fa[i][t], fb[i]);
                    __syncwarp();
                    arrive_if(smem_u32(&ffull[slot]), lane == 0);
                    if (++slot == S::RING) {
                        slot = 0;
                        ph ^= 1;
                    }
                }
#pragma unroll
                for (int i = 0; i < AHEAD; i++) {
                    fb[i] = nb[i];
#pragma unroll
                    for (int t = 0; t < PER; t++) fa[i][t] = na[i][t];
                }
            }
        }
    } else if (warp == 3) {  // ------------------------------------------------- relay (as in the tile kernel)
        int slot = 0, buf = 0;
        uint32_t fph = 0, bph = 0;
        bool ok = true;
        for (uint32_t tile = tile0; tile < tiles && ok; tile += step)
            for (int kb = kb0; kb < kb1; kb++) {
                ok = warp_wait(smem_u32(&ffull[slot]), fph, abort_flag, args.status) &&
                     warp_wait(smem_u32(&tfull[buf]), bph ^ 1, abort_flag, args.status);
                if (!ok) break;
                arrive_if(smem_u32(&tfull[buf]), lane == 0);
                if (++slot == S::RING) {
                    slot = 0;
                    fph ^= 1;
                }
                if (++buf == S::NB) {
                    buf = 0;
                    bph ^= 1;
                }
            }
    } else if (warp >= 4) {  // ------------------------------------------------- epilogue
        const int q = warp & 3;
        const int row = 32 * q + lane;  // of the weight tile
        const uint32_t taddr0 = tmem_base + ((uint32_t)(32 * q) << 16);
        int slot = 0, buf = 0;
        uint32_t bph = 0;
        for (uint32_t tile = tile0; tile < tiles; tile += step) {
            float2 acc[BT / 2];
#pragma unroll
            for (int p = 0; p < BT / 2; p++) acc[p] = make_float2(0.0f, 0.0f);
            bool ok = true;
            for (int kb = kb0; kb < kb1; kb++) {
                if (!warp_wait(smem_u32(&tfull[buf]), bph, abort_flag, args.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ta = taddr0 + (uint32_t)(buf * BT);
                const float *fac = ring + slot * S::SLOT;
                constexpr int LD = BT < 32 ? 16 : 32;
#pragma unroll
                for (int c = 0; c < BT; c += LD) {
                    uint32_t r[LD];
                    if constexpr (LD == 16)
                        tmem_ld_32x32b_x16(ta + c, r);
                    else
                        tmem_ld_32x32b_x32(ta + c, r);
                    tmem_ld_wait();
                    regs_ready(r);
#pragma unroll
                    for (int j = 0; j < LD; j += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(fac + c + j);
                        float2 &a = acc[(c + j) / 2], &b = acc[(c + j) / 2 + 1];
                        a = __ffma2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), make_float2(f.x, f.y), a);
                        b = __ffma2_rn(make_float2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])), make_float2(f.z, f.w), b);
                    }
                }
                tc_fence_before();
                __syncwarp();
                arrive_if(smem_u32(&tempty[buf]), lane == 0);
                arrive_if(smem_u32(&fempty[slot]), lane == 0);
                if (++slot == S::RING) slot = 0;
                if (++buf == S::NB) {
                    buf = 0;
                    bph ^= 1;
                }
            }
            if (split > 1) {  // this rank's sums, where the operands were: all its MMAs are done
                float *red = reinterpret_cast<float *>(smem);
#pragma unroll
                for (int p = 0; p < BT / 2; p++) {
                    red[2 * p * TW + row] = acc[p].x;
                    red[(2 * p + 1) * TW + row] = acc[p].y;
                }
                break;  // joined below; the one tile of this cluster
            }
            if (!ok) break;
            const BlockTile w = block_tile<BT, TW>(args, tab, tile);
            const int rows = (int)min(w.a_end - w.a_row, (int64_t)BT);
            if (w.n0 + row < args.N) {
                const float bias = args.bias_dtype >= 0 ? load_bias1(args, w.n0 + row) : 0.0f;
                const int64_t at = w.d_row * args.N + w.n0 + row;
#pragma unroll
                for (int p = 0; p < BT / 2; p++) {
                    if (2 * p < rows) store1(args, at + 2 * p * args.N, acc[p].x + bias);
                    if (2 * p + 1 < rows) store1(args, at + (2 * p + 1) * args.N, acc[p].y + bias);
                }
            }
        }
    }

    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (split > 1) {
        cluster_sync();  // every rank's sums are there
        if (tile0 < tiles) {
            const BlockTile w = block_tile<BT, TW>(args, tab, tile0);
            const int rows = (int)min(w.a_end - w.a_row, (int64_t)BT);
            join_few(args, smem_u32(smem), (int)split, (int)rank, w, rows);
        }
        __syncwarp();
        cluster_sync();  // nobody's sums go away while they are read
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, S::TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static std::atomic<bool> g_block_set[64];
static int g_block_pairs[64][3];  // clusters of 2, 4 and 8 CTAs resident at once

static fp8dl_status block_gemm_setup(int dev, int sms) {
    if (g_block_set[dev].load(std::memory_order_acquire)) return FP8DL_OK;
    std::lock_guard<std::mutex> lock(init_mutex());
    if (g_block_set[dev].load(std::memory_order_relaxed)) return FP8DL_OK;
    int resident[3] = {1 << 30, 1 << 30, 1 << 30};
    const void *kernels[] = {(const void *)block_gemm_kernel<false, false>, (const void *)block_gemm_kernel<true, false>,
                             (const void *)block_gemm_kernel<false, true>, (const void *)block_gemm_kernel<true, true>};
    for (const void *k : kernels) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bp::SMEM_BYTES);
        cudaFuncAttributes fa = {};
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, k);
        if (e != cudaSuccess) return fail(FP8DL_ERR_CUDA, "block GEMM set-up: %s", cudaGetErrorString(e));
        // the epilogue's larger register share comes out of the launch's registers
        if (fa.numRegs < bp::REGS_LAUNCH)
            return fail(FP8DL_ERR_CUDA, "block GEMM: built with %d registers, %d needed", fa.numRegs, bp::REGS_LAUNCH);
        // persistent pairs: how many are resident at once
        cudaLaunchConfig_t cfg = {};
        cfg.blockDim = dim3(bp::THREADS, 1, 1);
        cfg.dynamicSmemBytes = bp::SMEM_BYTES;
        cudaLaunchAttribute at = {};
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        for (int i = 0; i < 3; i++) {
            at.val.clusterDim.x = 2u << i;
            cfg.gridDim = dim3((unsigned)(sms / (2 << i) * (2 << i)), 1, 1);
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
            if (e != cudaSuccess) {
                cudaGetLastError();
                n = 0;
            }
            if (i == 0 && n < 1) return fail(FP8DL_ERR_UNSUPPORTED_DEVICE, "the block GEMM needs resident CTA-pair clusters");
            resident[i] = n < resident[i] ? n : resident[i];
        }
    }
    for (int i = 0; i < 3; i++) g_block_pairs[dev][i] = resident[i];
    const void *few[] = {(const void *)block_gemm_few_kernel<16>, (const void *)block_gemm_few_kernel<32>,
                         (const void *)block_gemm_few_kernel<64>};
    const int bytes[] = {bf::Shape<16>::SMEM_BYTES, bf::Shape<32>::SMEM_BYTES, bf::Shape<64>::SMEM_BYTES};
    for (int i = 0; i < 3; i++) {
        const cudaError_t e = cudaFuncSetAttribute(few[i], cudaFuncAttributeMaxDynamicSharedMemorySize, bytes[i]);
        if (e != cudaSuccess) return fail(FP8DL_ERR_CUDA, "block GEMM set-up: %s", cudaGetErrorString(e));
    }
    g_block_set[dev].store(true, std::memory_order_release);
    return FP8DL_OK;
}

// How many CTAs share a tile of the few-row kernel, each with two blocks at least: as many as give every SM
// one CTA, or, where the tiles alone fill more than half the SMs, two.  More than six cost
// more than they save.  us with 1 / 2 / 3 / 4 / 5 / 6 / 8:
//   M 16, N 4096, K 4096 (32 tiles) 11.0 / 8.5 / 7.9 / 7.5 / 8.0 / 7.9 / 7.9;  M 64 14.8 / 10.8 / 9.7 / 9.0 / 10.1 / 10.1 / 10.3
//   M 64, N 2048, K 7168 (16 tiles) 21.6 / 13.9 / 11.4 / 9.9 / 9.5 / 9.2 / 10.1;  M 64, N 11008, K 4096 (86 tiles) 16.6 / 14.5 / 13.9
static int few_split(int64_t tiles, int64_t kbs, int sms) {
    const int64_t most = kbs / 2 < bf::MOST_SHARES ? kbs / 2 : bf::MOST_SHARES;
    const int64_t split = (2 * tiles > sms ? 2 * (int64_t)sms : (int64_t)sms) / tiles;
    return split < 1 || most < 1 ? 1 : (int)(split < most ? split : most);
}

// Tiles of one product that are left when every pair has had the same number, if several pairs share each of
// them (`split`: two or four, each with a part of the blocks), else 0: where the reduction is long and all
// their clusters run at once.  us with 1 / 2 / 4 pairs a tile:
//   all tiles:  M 512, N 4096, K 4096 (32 tiles) 17.9 / 16.0;  K 11008 38.4 / 26.9;  M 256, N 4096, K 11008 (16 tiles) 38.0 / 25.7,
//     37.9 with 4 (not all at once);  M 256, N 2048, K 7168 (8 tiles) 26.0 / 18.8 / 15.9;  M 512, N 1536, K 1536 (12 tiles)
//     9.8 / 10.7 / 11.5
//   the last of them, in a launch of their own, without and with:  M 1280, N 4096, K 11008 (4 of 80 tiles) 72.2, 58.2;
//     M 1536 (20 of 96) 72.2, 65.0;  M 2048, N 2560, K 8192 (4 of 80) 55.4, 46.6;  M 512, N 11008, K 4096 (10 of 86) 32.7, 33.9
static int64_t shared_tiles(int64_t tiles, int64_t kbs, const int (&resident)[3], int &split) {
    const int64_t tail = tiles % resident[0];
    split = tail <= resident[2] && kbs >= 32 ? 4 : tail <= resident[1] && kbs >= 24 ? 2 : 1;
    if (tail == 0 || (tail < tiles && kbs - (kbs + split - 1) / split < 32)) split = 1;
    return split > 1 ? tail : 0;
}

// Rows of A per tile of the few-row kernel, or 0 for the 256 x 256 tiles.
// Groups: by their mean length in A's M rows (the host sees neither the offsets nor how many rows lie behind the
// last group: 128 rows in 64 groups of a buffer of 128 to 1024 rows 84 us, of 4096 90, of 16384 118).  64 groups, N 2048, K 4096, us with
// 16 / 32 / 64 rows a tile and with 256 x 256 tiles: 16 rows a group 87 / 88 / 93, 116;  32 rows 94 / 89 /
// 95, 116;  64 rows 138 / 99 / 97, 118;  96 rows 200 / 122 / 117, 121;  128 rows - / 151 / 120, 122;  192 rows
// - / 220 / 172, 125.
// One product: by what the two kernels' times follow.  The few-row kernel's: the bytes that pass the
// SM with the most CTAs (weight and rows of A, its CTAs' share of the blocks), and the rows a
// tile (epilogue and join): 4.5 us + 7.5 us per 1000 of (KB + 6 a row).  The tiles': 0.42 us a block, 6 us
// of start and end, 2 for a join.  us, 16 / 32 / 64 rows a tile, 256 x 256 tiles:
//   N 11008, K 4096   M 16: 12.2 / 12.3 / 13.5, 20.6;  M 37: 14.7 / 15.1 / 13.1, 18.8;  M 96: 24.1 / 15.6 / 19.4, 19.3;
//                     M 128: 33.3 / 24.0 / 19.7, 19.6
//   N 4096, K 4096    M 37: 8.7 / 9.0 / 8.8, 12.5;  M 128: 13.7 / 10.5 / 10.9, 14.4;  M 256: - / 14.6 / 13.0, 14.5;  M 384: - / - / 19.0, 15.3
//   N 2048, K 7168    M 64: 10.8 / 8.7 / 9.2, 13.2;  M 256: - / 14.0 / 14.1, 15.3
//   N 2048, K 2048    M 64: 6.2 / 6.1 / 6.8, 10.7;  M 256: - / 7.7 / 8.0, 11.1
//   N 16384, K 4096   M 64: 24.8 / 17.2 / 17.6, 21.0;  M 128: - / 25.9 / 20.8, 21.6
static int few_rows(const BlockGemmArgs &a, int sms, const int (&resident)[3]) {
    if (a.kind == BG_REDUCE) return 0;
    if (a.kind == BG_ROWS) {
        const int64_t busy = a.n_groups < a.M ? a.n_groups : a.M;
        const int64_t mean = (a.M + busy - 1) / busy;
        return mean <= 16 ? 16 : mean <= 48 ? 32 : mean <= 96 ? 64 : 0;
    }
    const int64_t kbs = (a.K + 127) / 128, tiles_w = (a.N + bf::TW - 1) / bf::TW;
    const int64_t pair_tiles = ((a.M + bp::TM - 1) / bp::TM) * ((a.N + bp::TN - 1) / bp::TN);
    int share;
    const int64_t shared = shared_tiles(pair_tiles, kbs, resident, share);
    const int64_t waves = (pair_tiles - shared + resident[0] - 1) / resident[0];
    double best = 6.0 + 0.42 * (double)(waves * kbs + (shared ? (kbs + share - 1) / share : 0)) + (shared ? 2.0 : 0.0);
    int rows = 0;
    for (int bt = 16; bt <= 64; bt *= 2) {
        const int64_t tiles = (a.M + bt - 1) / bt * tiles_w;
        const int split = few_split(tiles, kbs, sms);
        const double kb = 0.125 * (double)((tiles * split + sms - 1) / sms * ((kbs + split - 1) / split) * (bf::TW + bt));
        const double us = 4.5 + 0.0075 * (kb + 6.0 * bt);
        if (us < best) {
            best = us;
            rows = bt;
        }
    }
    return rows;
}

// What a product runs as.  Groups: the tiles are the most there can be, wherever the groups' borders lie.
struct BlockPlan {
    int rows;               // of A per tile: 16, 32 or 64 (few-row kernel), or 256
    int split;              // CTAs (few-row kernel) or CTA pairs that share each of the shared tiles
    int64_t whole, shared;  // tiles that one of them computes alone, and shared ones
};

static BlockPlan plan_block_gemm(const BlockGemmArgs &a, bool brows, int sms, const int (&resident)[3]) {
    BlockPlan p = {brows ? 0 : few_rows(a, sms, resident), 1, 0, 0};
    const bool few = p.rows > 0;
    if (!few) p.rows = bp::TM;
    const int64_t tw = few ? bf::TW : bp::TN, tiles_m = (a.M + p.rows - 1) / p.rows, tiles_n = (a.N + tw - 1) / tw;
    const int64_t busy = a.n_groups < a.M ? a.n_groups : a.M;  // groups that can hold a row
    const int64_t tiles = a.kind == BG_DENSE  ? tiles_m * tiles_n
                          : a.kind == BG_ROWS ? (a.M / p.rows + busy) * tiles_n
                                              : a.n_groups * tiles_m * tiles_n;
    const int64_t kbs = (a.K + 127) / 128;
    if (few) {
        p.split = few_split(tiles, kbs, sms);
        p.shared = p.split > 1 ? tiles : 0;
    } else if (a.kind == BG_DENSE) {
        p.shared = shared_tiles(tiles, kbs, resident, p.split);
    }
    p.whole = tiles - p.shared;
    return p;
}

template <int BT>
static fp8dl_status launch_few(const uint8_t *A, int32_t a_dtype, const uint8_t *B, int32_t b_dtype, int64_t b_rows,
                               BlockGemmArgs &args, const BlockPlan &plan, int sms, cudaStream_t st, bool pdl, const char *what) {
    using S = bf::Shape<BT>;
    CUtensorMap ta, tb;
    FP8DL_TRY(encode_tmap_2d_u8(&ta, A, (uint64_t)args.K, (uint64_t)args.M, (uint64_t)args.K, bf::BK, BT,
                                CU_TENSOR_MAP_SWIZZLE_128B));
    FP8DL_TRY(encode_tmap_2d_u8(&tb, B, (uint64_t)args.K, (uint64_t)b_rows, (uint64_t)args.K, bf::BK, bf::TW,
                                CU_TENSOR_MAP_SWIZZLE_128B));
    args.idesc = (1u << 4) | ((uint32_t)b_dtype << 7) | ((uint32_t)a_dtype << 10) | ((uint32_t)(BT >> 3) << 17) |
                 ((uint32_t)(bf::TW >> 4) << 24);
    args.along_n = 0;  // the token tiles of a weight tile follow one another
    args.band = 0x7fffffffu;
    const int64_t resident = 2 * (int64_t)sms;
    const int64_t ctas = plan.shared ? plan.shared * plan.split : plan.whole < resident ? plan.whole : resident;
    (void)launch_kernel(block_gemm_few_kernel<BT>, dim3((unsigned)ctas), S::THREADS, S::SMEM_BYTES, st, plan.split, pdl, ta, tb, args);
    note_launch();
    return check_launch(what);
}

// Columns of D: a row's bytes are a 32-bit coordinate of the stores.
static bool block_cols_ok(int64_t n) { return dim_ok(n, 16) && n < (int64_t(1) << 29); }

static fp8dl_status check_block_gemm(const uint8_t *A, int32_t a_dtype, const float *a_s, const uint8_t *B,
                                     int32_t b_dtype, const float *b_s, const void *D, int32_t d_dtype, bool tokens) {
    FP8DL_CHECK_ARG((a_dtype == FP8DL_E4M3 || a_dtype == FP8DL_E5M2) && (b_dtype == FP8DL_E4M3 || b_dtype == FP8DL_E5M2),
                    "a_dtype and b_dtype must be E4M3 or E5M2");
    FP8DL_CHECK_ARG(d_dtype == FP8DL_BF16 || d_dtype == FP8DL_F32, "d_dtype must be FP8DL_BF16 or FP8DL_F32");
    FP8DL_CHECK_ARG(!tokens || (A && a_s && B && b_s && D), "A, a_s, B, b_s and D must be non-NULL");
    if (!aligned16(A) || !aligned16(a_s) || !aligned16(B) || !aligned16(b_s) || !aligned16(D))
        return fail(FP8DL_ERR_ALIGN, "A, a_s, B, b_s and D must be 16-byte aligned");
    return FP8DL_OK;
}

// rows_b: rows of B in memory (all groups'); a_rows: rows of A.
static fp8dl_status launch_block_gemm(const uint8_t *A, int32_t a_dtype, int64_t a_rows, const uint8_t *B,
                                      int32_t b_dtype, int64_t b_rows, bool brows, BlockGemmArgs &args,
                                      cudaStream_t st, bool pdl, const char *what) {
    int dev = 0, sms = 0;
    FP8DL_TRY(current_device(&dev, &sms));
    FP8DL_TRY(block_gemm_setup(dev, sms));
    const BlockPlan plan = plan_block_gemm(args, brows, sms, g_block_pairs[dev]);
    if (plan.whole + plan.shared > 0x7fffffffll) return fail(FP8DL_ERR_SHAPE, "%s: more than 2^31 - 1 output tiles", what);
    if (plan.rows == 16) return launch_few<16>(A, a_dtype, B, b_dtype, b_rows, args, plan, sms, st, pdl, what);
    if (plan.rows == 32) return launch_few<32>(A, a_dtype, B, b_dtype, b_rows, args, plan, sms, st, pdl, what);
    if (plan.rows == 64) return launch_few<64>(A, a_dtype, B, b_dtype, b_rows, args, plan, sms, st, pdl, what);
    CUtensorMap ta, tb, td;
    FP8DL_TRY(encode_tmap_2d_u8(&ta, A, (uint64_t)args.K, (uint64_t)a_rows, (uint64_t)args.K, bp::BK, 128,
                                CU_TENSOR_MAP_SWIZZLE_128B));
    FP8DL_TRY(encode_tmap_2d_u8(&tb, B, (uint64_t)args.K, (uint64_t)b_rows, (uint64_t)args.K, bp::BK, bp::B_ROWS,
                                CU_TENSOR_MAP_SWIZZLE_128B));
    const uint64_t d_ld = (uint64_t)args.N * (args.d_dtype == FP8DL_BF16 ? 2 : 4);
    FP8DL_TRY(encode_tmap_2d_u8(&td, args.D, d_ld, (uint64_t)(args.kind == BG_REDUCE ? args.n_groups * args.M : args.M), d_ld, 128,
                                32, CU_TENSOR_MAP_SWIZZLE_128B));
    args.idesc = (1u << 4) | ((uint32_t)a_dtype << 7) | ((uint32_t)b_dtype << 10) | ((uint32_t)(bp::TN >> 3) << 17) |
                 ((uint32_t)(bp::TM >> 4) << 24);
    const int64_t tiles_m = (args.M + bp::TM - 1) / bp::TM, tiles_n = (args.N + bp::TN - 1) / bp::TN;
    // Bands of 16 tiles along the dimension with fewer of them, 8 where a panel is long (16384 x 16384 x
    // 4096: 838 us with 16, 857 with 8, under the power cap; 16384 x 4096 x 16384: 833 along the
    // columns with 8, 848 with 16, 850 along the rows).  A group's row tiles are few: along the rows.
    args.along_n = args.kind != BG_ROWS && tiles_n < tiles_m;
    args.band = args.kind == BG_REDUCE || args.K <= 8192 ? 16 : 8;
    const int64_t pairs = g_block_pairs[dev][0];
    args.end = (uint32_t)plan.whole;
    if (plan.whole) {
        (void)launch_kernel(brows ? block_gemm_kernel<true, false> : block_gemm_kernel<false, false>,
                            dim3((unsigned)(2 * (plan.whole < pairs ? plan.whole : pairs))), bp::THREADS, bp::SMEM_BYTES, st, 2, pdl, ta, tb,
                            td, args);
        note_launch();
    }
    if (plan.shared) {
        args.first = (uint32_t)plan.whole;
        args.end = (uint32_t)(plan.whole + plan.shared);
        (void)launch_kernel(brows ? block_gemm_kernel<true, true> : block_gemm_kernel<false, true>,
                            dim3((unsigned)(2 * plan.split * plan.shared)), bp::THREADS, bp::SMEM_BYTES, st, 2 * plan.split,
                            pdl || plan.whole, ta, tb,
                            td, args);
        note_launch();
    }
    return check_launch(what);
}

}  // namespace fp8dl

using namespace fp8dl;

extern "C" fp8dl_status fp8_block_gemm(const uint8_t *A, int32_t a_dtype, const float *a_s, const uint8_t *B,
                                       int32_t b_dtype, const float *b_s, int32_t b_rows, int64_t M, int64_t N,
                                       int64_t K, const void *bias, int32_t bias_dtype, void *D, int32_t d_dtype,
                                       int32_t *dev_status, fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_gemm");
    if (!block_tokens_ok(M) || !block_cols_ok(N) || !dim_ok(K, 16))
        return fail(FP8DL_ERR_SHAPE, "M (%lld) must be in [0, 2^31), N (%lld) and K (%lld) positive multiples of 16, N < 2^29",
                    (long long)M, (long long)N, (long long)K);
    FP8DL_TRY(check_block_gemm(A, a_dtype, a_s, B, b_dtype, b_s, D, d_dtype, M > 0));
    FP8DL_CHECK_ARG(b_rows == 1 || b_rows == 128, "b_rows must be 1 or 128");
    FP8DL_CHECK_ARG(!bias || bias_dtype == FP8DL_BF16 || bias_dtype == FP8DL_F32,
                    "bias_dtype must be FP8DL_BF16 or FP8DL_F32");
    if (!aligned16(bias)) return fail(FP8DL_ERR_ALIGN, "bias must be 16-byte aligned");
    FP8DL_TRY(current_device(nullptr, nullptr));
    if (M == 0) return FP8DL_OK;
    BlockGemmArgs a = {};
    a.kind = BG_DENSE;
    a.M = M;
    a.N = N;
    a.K = K;
    a.a_s = a_s;
    a.b_s = b_s;
    a.b_ld = b_rows == 1 ? N : (N + 127) / 128;
    a.bias = bias;
    a.bias_dtype = bias ? bias_dtype : -1;
    a.D = D;
    a.d_dtype = d_dtype;
    a.status = dev_status;
    return launch_block_gemm(A, a_dtype, M, B, b_dtype, N, b_rows == 1, a, (cudaStream_t)stream,
                             short_call_flops(2.0 * (double)M * (double)N * (double)K), "fp8_block_gemm");
}

extern "C" fp8dl_status fp8_block_gemm_plan(int32_t b_rows, int32_t n_groups, int64_t M, int64_t N, int64_t K,
                                            int32_t *tile_rows, int32_t *shares, int64_t *whole, int64_t *shared) {
    if (!dim_ok(M, 1) || !block_tokens_ok(M) || !block_cols_ok(N) || !dim_ok(K, 16))
        return fail(FP8DL_ERR_SHAPE, "M (%lld) must be in [1, 2^31), N (%lld) and K (%lld) positive multiples of 16, N < 2^29",
                    (long long)M, (long long)N, (long long)K);
    FP8DL_CHECK_ARG(n_groups >= 0 && n_groups <= kMaxGroups, "n_groups must be in [0, %d]", kMaxGroups);
    FP8DL_CHECK_ARG(b_rows == 128 || (b_rows == 1 && n_groups == 0), "b_rows must be 128, or 1 without groups");
    FP8DL_CHECK_ARG(tile_rows && shares && whole && shared, "tile_rows, shares, whole and shared must be non-NULL");
    int dev = 0, sms = 0;
    FP8DL_TRY(current_device(&dev, &sms));
    FP8DL_TRY(block_gemm_setup(dev, sms));
    BlockGemmArgs a = {};
    a.kind = n_groups ? BG_ROWS : BG_DENSE;
    a.M = M;
    a.N = N;
    a.K = K;
    a.n_groups = n_groups;
    const BlockPlan p = plan_block_gemm(a, b_rows == 1, sms, g_block_pairs[dev]);
    *tile_rows = p.rows;
    *shares = p.split;
    *whole = p.whole;
    *shared = p.shared;
    return FP8DL_OK;
}

extern "C" fp8dl_status fp8_block_gemm_grouped(const uint8_t *A, int32_t a_dtype, const float *a_s, const uint8_t *B,
                                               int32_t b_dtype, const float *b_s, const int32_t *offsets,
                                               int32_t n_groups, int64_t M, int64_t N, int64_t K, void *D,
                                               int32_t d_dtype, int32_t *dev_status, fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_gemm_grouped");
    if (!block_tokens_ok(M) || !block_cols_ok(N) || !dim_ok(K, 16))
        return fail(FP8DL_ERR_SHAPE, "M (%lld) must be in [0, 2^31), N (%lld) and K (%lld) positive multiples of 16, N < 2^29",
                    (long long)M, (long long)N, (long long)K);
    FP8DL_TRY(check_block_groups(offsets, n_groups, false));
    FP8DL_TRY(check_block_gemm(A, a_dtype, a_s, B, b_dtype, b_s, D, d_dtype, M > 0));
    if (!block_tokens_ok(N * n_groups))
        return fail(FP8DL_ERR_SHAPE, "n_groups * N (%lld) must be below 2^31", (long long)(N * n_groups));
    FP8DL_TRY(current_device(nullptr, nullptr));
    if (M == 0) return FP8DL_OK;
    BlockGemmArgs a = {};
    a.kind = BG_ROWS;
    a.M = M;
    a.N = N;
    a.K = K;
    a.a_s = a_s;
    a.b_s = b_s;
    a.b_ld = (N + 127) / 128;
    a.offsets = offsets;
    a.n_groups = n_groups;
    a.bias_dtype = -1;
    a.D = D;
    a.d_dtype = d_dtype;
    a.status = dev_status;
    return launch_block_gemm(A, a_dtype, M, B, b_dtype, N * n_groups, false, a, (cudaStream_t)stream,
                             short_call_flops(2.0 * (double)M * (double)N * (double)K), "fp8_block_gemm_grouped");
}

extern "C" fp8dl_status fp8_block_gemm_grouped_wgrad(const uint8_t *A, int32_t a_dtype, const float *a_s,
                                                     const uint8_t *B, int32_t b_dtype, const float *b_s,
                                                     const int32_t *offsets, int32_t n_groups, int64_t M, int64_t N,
                                                     int64_t T, void *D, int32_t d_dtype, int32_t *dev_status,
                                                     fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_gemm_grouped_wgrad");
    if (!dim_ok(M, 1) || !block_tokens_ok(M) || !block_tokens_ok(M * (n_groups < 1 ? 1 : n_groups)) || !block_cols_ok(N) || !block_tokens_ok(T) || T % 128 != 0)
        return fail(FP8DL_ERR_SHAPE, "M (%lld) must be positive, n_groups * M < 2^31, N (%lld) a positive multiple of 16 < 2^29, T (%lld) a multiple of 128",
                    (long long)M, (long long)N, (long long)T);
    FP8DL_TRY(check_block_groups(offsets, n_groups, false));
    FP8DL_CHECK_ARG(D, "D is NULL");
    FP8DL_TRY(check_block_gemm(A, a_dtype, a_s, B, b_dtype, b_s, D, d_dtype, T > 0));
    FP8DL_TRY(current_device(nullptr, nullptr));
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) {
        const size_t bytes = (size_t)n_groups * (size_t)M * (size_t)N * (d_dtype == FP8DL_BF16 ? 2 : 4);
        cudaError_t e = cudaMemsetAsync(D, 0, bytes, st);
        if (e != cudaSuccess) return fail(FP8DL_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
        return FP8DL_OK;
    }
    BlockGemmArgs a = {};
    a.kind = BG_REDUCE;
    a.M = M;
    a.N = N;
    a.K = T;
    a.a_s = a_s;
    a.b_s = b_s;
    a.b_ld = N;
    a.offsets = offsets;
    a.n_groups = n_groups;
    a.bias_dtype = -1;
    a.D = D;
    a.d_dtype = d_dtype;
    a.status = dev_status;
    return launch_block_gemm(A, a_dtype, M, B, b_dtype, N, true, a, st,
                             short_call_flops(2.0 * (double)M * (double)N * (double)T), "fp8_block_gemm_grouped_wgrad");
}
