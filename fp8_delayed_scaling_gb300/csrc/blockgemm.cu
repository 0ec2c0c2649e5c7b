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
#include <stdlib.h>

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

// Reduction blocks of a tile.
template <int TM, int TN>
__device__ __forceinline__ int block_tile_kbs(const BlockGemmArgs &a, const GroupTables &t, uint32_t tile) {
    if (a.kind != BG_REDUCE) return (int)((a.K + 127) / 128);
    const uint32_t per = (uint32_t)((a.N + TN - 1) / TN) * (uint32_t)((a.M + TM - 1) / TM);
    const uint32_t g = tile / per;
    return t.pre[g + 1] - t.pre[g];
}

template <int TM, int TN>
__device__ __forceinline__ BlockTile block_tile(const BlockGemmArgs &a, const GroupTables &t, uint32_t tile) {
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

// Columns c0 .. c0 + 31 of this thread's sums, bias added (n = their first column of D).
__device__ __forceinline__ void add_bias32(const BlockGemmArgs &a, int64_t n, float2 (&v)[16]) {
    if (a.bias_dtype == FP8DL_BF16) {
        const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(a.bias) + n;
#pragma unroll
        for (int g = 0; g < 4; g++)
            if (n + 8 * g < a.N) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(b + 8 * g));
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int q = 0; q < 4; q++)
                    v[4 * g + q] = __fadd2_rn(v[4 * g + q], make_float2(bf16_lo(w[q]), bf16_hi(w[q])));
            }
    } else if (a.bias_dtype == FP8DL_F32) {
        const float *b = static_cast<const float *>(a.bias) + n;
#pragma unroll
        for (int g = 0; g < 8; g++)
            if (n + 4 * g < a.N) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(b + 4 * g));
                v[2 * g] = __fadd2_rn(v[2 * g], make_float2(u.x, u.y));
                v[2 * g + 1] = __fadd2_rn(v[2 * g + 1], make_float2(u.z, u.w));
            }
    }
}

// One warp writes its 32 rows x 128 columns of D (lane = row; the sums in acc), rounded once.
// Straight from the registers every store would touch 32 rows, a piece of a line each (the
// stores of a 256 x 256 tile took 7200 cycles, a fifth of a tile with K = 4096).  Instead 64
// bytes of each row at a time go through shared memory (16-byte chunks XOR-swizzled by row
// pairs: conflict-free both ways) and leave as two whole sectors, eight rows per instruction.
__device__ __forceinline__ void store_tile(const BlockGemmArgs &a, uint8_t *stage, int lane, int64_t d_row, int rows,
                                           int64_t n0, float2 (&acc)[64]) {
    const bool bf = a.d_dtype == FP8DL_BF16;
    const int esz = bf ? 2 : 4;
    const int sub = lane >> 2, ch = lane & 3;
    uint8_t *base = static_cast<uint8_t *>(a.D) + ((d_row + sub) * a.N + n0) * esz + ch * 16;
    const int64_t step = 8 * a.N * esz;
    uint8_t *mine = stage + lane * 64;
    const int swz = (lane >> 1) & 3, rswz = (sub >> 1) & 3;
    auto flush = [&](int off, int64_t n) {  // the staged 64 bytes of each row, from column n on
        __syncwarp();
        const bool ok = n + ch * (16 / esz) < a.N;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint4 u = *reinterpret_cast<const uint4 *>(stage + (8 * i + sub) * 64 + ((ch ^ rswz) << 4));
            if (ok && 8 * i + sub < rows) *reinterpret_cast<uint4 *>(base + i * step + off) = u;
        }
        __syncwarp();
    };
#pragma unroll
    for (int c = 0; c < 4; c++) {
        const int64_t n = n0 + 32 * c;
        if (n >= a.N) break;
        float2 v[16];
#pragma unroll
        for (int p = 0; p < 16; p++) v[p] = acc[16 * c + p];
        if (a.bias_dtype >= 0) add_bias32(a, n, v);
        if (bf) {
#pragma unroll
            for (int g = 0; g < 4; g++) {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[4 * g + q].x, v[4 * g + q].y);
                    w[q] = *reinterpret_cast<const uint32_t *>(&h);
                }
                *reinterpret_cast<uint4 *>(mine + ((g ^ swz) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            flush(64 * c, n);
        } else {
#pragma unroll
            for (int h = 0; h < 2; h++) {
#pragma unroll
                for (int g = 0; g < 4; g++)
                    *reinterpret_cast<float4 *>(mine + ((g ^ swz) << 4)) =
                        make_float4(v[8 * h + 2 * g].x, v[8 * h + 2 * g].y, v[8 * h + 2 * g + 1].x, v[8 * h + 2 * g + 1].y);
                flush(128 * c + 64 * h, n + 16 * h);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// 128 x 256 tiles, one persistent CTA per SM.
//   warp 0      TMA producer: 128 rows of A and 256 of B per k-block, four stages
//   warp 1      MMA thread: per block four MMAs (M 128, N 256, K 32) into one of two
//               256-column tensor-memory buffers
//   warp 2      copies the blocks' factors into a shared-memory ring
//   warps 4-11  epilogue: warp w drains lane quarter w & 3 of column half (w - 4) / 4; a thread
//               holds one row x 128 columns of the sum (64 fp32 pairs)
// With 128 x 128 weight factors a thread's 128 columns share one factor per block: one
// packed multiply-add per two values, half the MMAs' time on the FP32 pipe.  With factors per
// row of B (BROWS, weight gradients) each column has its own: one more packed multiply.
//
// Why not CTA pairs (256 x 256 tiles): every block's buffer goes to the epilogue and back
// through mbarriers, and between two SMs that costs more than the pair saves in operand
// traffic: PAIRFIG.
// ---------------------------------------------------------------------------
namespace bp {
constexpr int TM = 128, TN = 256, BK = 128, STAGES = 4;
constexpr int A_BYTES = TM * BK, B_BYTES = TN * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int THREADS = 384, EPI_WARPS = 8;
constexpr int REGS_LAUNCH = 168, REGS_IO = 56, REGS_EPI = 224;  // 128 * 56 + 256 * 224 = 384 * 168
static_assert(128 * REGS_IO + 256 * REGS_EPI <= THREADS * REGS_LAUNCH, "register split");
constexpr int TMEM_COLS = 512;
// The factors of the next blocks: 128 of A's, then one per column half, or (BROWS) 256, of B's.
constexpr int RING = 4, SLOT_FLOATS = 128 + 256, RING_BYTES = RING * SLOT_FLOATS * 4;
constexpr int OUT_BYTES = EPI_WARPS * 2048;        // 32 rows x 64 bytes of D per warp
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + OUT_BYTES + 1024 + RING_BYTES + kGroupTableBytes + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
}  // namespace bp

template <bool BROWS>
__global__ void __launch_bounds__(bp::THREADS, 1)
    block_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                      const BlockGemmArgs args) {
    using namespace bp;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
    uint8_t *out_stage = smem + STAGES * STAGE_BYTES;
    uint8_t *bar_area = out_stage + OUT_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(bar_area);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *ffull = tempty + 2;
    uint64_t *fempty = ffull + RING;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fempty + RING);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *ring = reinterpret_cast<float *>(bar_area + 1024);
    const GroupTables tab = group_tables(bar_area + 1024 + RING_BYTES);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < 2; a++) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), EPI_WARPS);
        }
        for (int a = 0; a < RING; a++) {
            mbar_init(smem_u32(&ffull[a]), 32);  // every lane of the copying warp
            mbar_init(smem_u32(&fempty[a]), EPI_WARPS);
        }
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_map(&tmap_a);
        tma_prefetch_map(&tmap_b);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();
    if (args.kind == BG_ROWS) build_groups(tab, args.offsets, args.n_groups, args.M, TM, 0x7fffffffll);
    if (args.kind == BG_REDUCE)
        build_groups(tab, args.offsets, args.n_groups, 0x7fffffffll, 128, args.K / 128);
    const uint32_t tiles = block_tiles<TM, TN>(args, tab);

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_IO));
        if (warp == 0 && lane == 0) {  // ------------------------------------- producer
            int s = 0;
            uint32_t ph = 0;
            int64_t issued = 0;
            bool ok = true;
            for (uint32_t tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                const BlockTile w = block_tile<TM, TN>(args, tab, tile);
                for (int kb = 0; kb < w.kbs; kb++) {
                    if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&full[s]), sa = smem_u32(smem + s * STAGE_BYTES);
                    mbar_expect_tx(fb, STAGE_BYTES);
                    tma_load_2d(sa, &tmap_a, fb, (w.kb0 + kb) * BK, (int32_t)w.a_row);
                    tma_load_2d(sa + A_BYTES, &tmap_b, fb, (w.kb0 + kb) * BK, (int32_t)w.b_row);
                    issued++;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok)
                for (int64_t i = issued - 1; i >= 0 && i >= issued - STAGES; i--)
                    mbar_drain(smem_u32(&full[i % STAGES]), (uint32_t)((i / STAGES) & 1));
        } else if (warp == 1 && lane == 0) {  // ------------------------------- MMA issuer
            int s = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true, any = false;
            uint32_t last_bar = 0, last_par = 0;
            const SDesc desc0 = sdesc_k_sw128_split(smem_u32(smem));
            for (uint32_t tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                const int kbs = block_tile_kbs<TM, TN>(args, tab, tile);
                for (int kb = 0; kb < kbs; kb++) {
                    if (!mbar_wait(smem_u32(&tempty[buf]), bph ^ 1, abort_flag, args.status) ||
                        !mbar_wait(smem_u32(&full[s]), ph, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t lo_a = desc0.lo + (uint32_t)s * (STAGE_BYTES >> 4);
                    const uint32_t lo_b = lo_a + (A_BYTES >> 4);
#pragma unroll
                    for (int kk = 0; kk < BK / 32; kk++)
                        umma_f8f6f4(tmem_base + (uint32_t)(buf * TN), sdesc_join(lo_a + 2 * kk, desc0.hi),
                                    sdesc_join(lo_b + 2 * kk, desc0.hi), args.idesc, kk != 0);
                    umma_commit(smem_u32(&tfull[buf]));
                    umma_commit(smem_u32(&empty[s]));
                    any = true;
                    last_bar = smem_u32(&empty[s]);
                    last_par = ph;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                    buf ^= 1;
                    if (buf == 0) bph ^= 1;
                }
            }
            if (!ok && any) mbar_drain(last_bar, last_par);
        } else if (warp == 2) {  // --------------------------------------------- factors
            // Rows and columns outside the matrix take a valid address: their sums are not stored.
            int slot = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (uint32_t tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                const BlockTile w = block_tile<TM, TN>(args, tab, tile);
                const float *pa[4], *pb[2];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int64_t row = w.a_row + 32 * j + lane;
                    pa[j] = args.a_s + (int64_t)w.kb0 * args.M + (row < w.a_end ? row : w.a_row);
                }
#pragma unroll
                for (int h = 0; h < 2; h++) {  // BROWS: four columns of each half per lane
                    const int64_t n = w.n0 + 128 * h + (BROWS ? 4 * lane : 0);
                    pb[h] = w.b_s + (int64_t)w.kb0 * args.b_ld + (n < args.N ? (BROWS ? n : n >> 7) : 0);
                }
                for (int kb = 0; kb < w.kbs; kb++) {
                    if (!mbar_wait(smem_u32(&fempty[slot]), ph ^ 1, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = smem_u32(ring + slot * SLOT_FLOATS);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        cp_async4(dst + 4 * (32 * j + lane), pa[j]);
                        pa[j] += args.M;
                    }
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        if (BROWS)
                            cp_async16(dst + 512 + 512 * h + 16 * lane, pb[h]);
                        else if (lane == 0)
                            cp_async4(dst + 512 + 512 * h, pb[h]);
                        pb[h] += args.b_ld;
                    }
                    cp_async_arrive(smem_u32(&ffull[slot]));
                    if (++slot == RING) {
                        slot = 0;
                        ph ^= 1;
                    }
                }
            }
            cp_async_wait_all();
        }
    } else {  // ------------------------------------------------------------ epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t taddr0 = tmem_base + (uint32_t)(128 * half) + ((uint32_t)(32 * q) << 16);
        uint8_t *stage = out_stage + (warp - 4) * 2048;
        const float *my_a = ring + 32 * q + lane, *my_b = ring + 128 + 128 * half;
        int slot = 0;
        uint32_t fph = 0;
        // The next block's factors are there (they were copied blocks ago).
        auto wait_factors = [&] { return mbar_wait(smem_u32(&ffull[slot]), fph, abort_flag, args.status); };
        auto free_factors = [&] {  // this warp has read them
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&fempty[slot]));
            if (++slot == RING) {
                slot = 0;
                fph ^= 1;
            }
        };
        int buf = 0;
        uint32_t bph = 0;
        for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
            const int kbs = block_tile_kbs<TM, TN>(args, tab, tile);
            float2 acc[64];
#pragma unroll
            for (int p = 0; p < 64; p++) acc[p] = make_float2(0.0f, 0.0f);
            bool ok = true;
            for (int kb = 0; kb < kbs; kb++) {
                if (!wait_factors()) {
                    ok = false;
                    break;
                }
                const float *fb = my_b + slot * SLOT_FLOATS;
                const float fa = my_a[slot * SLOT_FLOATS];
                const float2 sc = f2(BROWS ? fa : __fmul_rn(fa, fb[0]));
                if (!BROWS) free_factors();
                if (!mbar_wait(smem_u32(&tfull[buf]), bph, abort_flag, args.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t ta = taddr0 + (uint32_t)(buf * TN);
                uint32_t r[2][32];
                tmem_ld_32x32b_x32(ta, r[0]);
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    tmem_ld_wait_regs(r[c & 1]);
                    if (c < 3) {
                        tmem_ld_32x32b_x32(ta + 32 * (c + 1), r[(c + 1) & 1]);
                    } else {  // the buffer is read: the next block's MMAs may overwrite it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&tempty[buf]));
                    }
#pragma unroll
                    for (int p = 0; p < 16; p += 2) {
                        float2 f0 = sc, f1 = sc;
                        if (BROWS) {
                            const float4 u = *reinterpret_cast<const float4 *>(fb + 32 * c + 2 * p);
                            f0 = __fmul2_rn(sc, make_float2(u.x, u.y));
                            f1 = __fmul2_rn(sc, make_float2(u.z, u.w));
                        }
                        const uint32_t *t = r[c & 1] + 2 * p;
                        acc[16 * c + p] =
                            __ffma2_rn(make_float2(__uint_as_float(t[0]), __uint_as_float(t[1])), f0, acc[16 * c + p]);
                        acc[16 * c + p + 1] =
                            __ffma2_rn(make_float2(__uint_as_float(t[2]), __uint_as_float(t[3])), f1, acc[16 * c + p + 1]);
                    }
                }
                if (BROWS) free_factors();
                buf ^= 1;
                if (buf == 0) bph ^= 1;
            }
            if (!ok) break;
            const BlockTile w = block_tile<TM, TN>(args, tab, tile);
            const int64_t first = 32 * q;
            const int64_t rows = w.a_end - (w.a_row + first);  // the warp's rows to write
            store_tile(args, stage, lane, w.d_row + first, (int)max(min(rows, (int64_t)32), (int64_t)0), w.n0 + 128 * half, acc);
        }
    }

    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static std::atomic<bool> g_block_set[64];

static fp8dl_status block_gemm_setup(int dev) {
    if (g_block_set[dev].load(std::memory_order_acquire)) return FP8DL_OK;
    std::lock_guard<std::mutex> lock(init_mutex());
    if (g_block_set[dev].load(std::memory_order_relaxed)) return FP8DL_OK;
    const void *kernels[] = {(const void *)block_gemm_kernel<false>, (const void *)block_gemm_kernel<true>};
    for (const void *k : kernels) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bp::SMEM_BYTES);
        cudaFuncAttributes fa = {};
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, k);
        if (e != cudaSuccess) return fail(FP8DL_ERR_CUDA, "block GEMM set-up: %s", cudaGetErrorString(e));
        // the epilogue's larger register share comes out of the launch's registers
        if (fa.numRegs < bp::REGS_LAUNCH)
            return fail(FP8DL_ERR_CUDA, "block GEMM: built with %d registers, %d needed", fa.numRegs, bp::REGS_LAUNCH);
    }
    g_block_set[dev].store(true, std::memory_order_release);
    return FP8DL_OK;
}

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
                                      int32_t b_dtype, int64_t b_rows, bool brows, int64_t tiles_bound,
                                      BlockGemmArgs &args, cudaStream_t st, bool pdl, const char *what) {
    int dev = 0, sms = 0;
    FP8DL_TRY(current_device(&dev, &sms));
    FP8DL_TRY(block_gemm_setup(dev));
    CUtensorMap ta, tb;
    FP8DL_TRY(encode_tmap_2d_u8(&ta, A, (uint64_t)args.K, (uint64_t)a_rows, (uint64_t)args.K, bp::BK, bp::TM,
                                CU_TENSOR_MAP_SWIZZLE_128B));
    FP8DL_TRY(encode_tmap_2d_u8(&tb, B, (uint64_t)args.K, (uint64_t)b_rows, (uint64_t)args.K, bp::BK, bp::TN,
                                CU_TENSOR_MAP_SWIZZLE_128B));
    args.idesc = (1u << 4) | ((uint32_t)a_dtype << 7) | ((uint32_t)b_dtype << 10) | ((uint32_t)(bp::TN >> 3) << 17) |
                 ((uint32_t)(bp::TM >> 4) << 24);
    const int64_t tiles_m = (args.M + bp::TM - 1) / bp::TM, tiles_n = (args.N + bp::TN - 1) / bp::TN;
    args.along_n = 0;
    args.band = 16;
    if (tiles_bound > 0x7fffffffll) return fail(FP8DL_ERR_SHAPE, "%s: more than 2^31 - 1 output tiles", what);
    (void)launch_kernel(brows ? block_gemm_kernel<true> : block_gemm_kernel<false>,
                        dim3((unsigned)(tiles_bound < sms ? tiles_bound : sms)), bp::THREADS, bp::SMEM_BYTES, st, 0, pdl, ta,
                        tb, args);
    note_launch();
    return check_launch(what);
}

}  // namespace fp8dl

using namespace fp8dl;

extern "C" fp8dl_status fp8_block_gemm(const uint8_t *A, int32_t a_dtype, const float *a_s, const uint8_t *B,
                                       int32_t b_dtype, const float *b_s, int32_t b_rows, int64_t M, int64_t N,
                                       int64_t K, const void *bias, int32_t bias_dtype, void *D, int32_t d_dtype,
                                       int32_t *dev_status, fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_gemm");
    if (!block_tokens_ok(M) || !dim_ok(N, 16) || !dim_ok(K, 16))
        return fail(FP8DL_ERR_SHAPE, "M (%lld) must be in [0, 2^31), N and K (%lld, %lld) positive multiples of 16",
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
    const int64_t tiles = ((M + bp::TM - 1) / bp::TM) * ((N + bp::TN - 1) / bp::TN);
    return launch_block_gemm(A, a_dtype, M, B, b_dtype, N, b_rows == 1, tiles, a, (cudaStream_t)stream,
                             short_call_flops(2.0 * (double)M * (double)N * (double)K), "fp8_block_gemm");
}

extern "C" fp8dl_status fp8_block_gemm_grouped(const uint8_t *A, int32_t a_dtype, const float *a_s, const uint8_t *B,
                                               int32_t b_dtype, const float *b_s, const int32_t *offsets,
                                               int32_t n_groups, int64_t M, int64_t N, int64_t K, void *D,
                                               int32_t d_dtype, int32_t *dev_status, fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_gemm_grouped");
    if (!block_tokens_ok(M) || !dim_ok(N, 16) || !dim_ok(K, 16))
        return fail(FP8DL_ERR_SHAPE, "M (%lld) must be in [0, 2^31), N and K (%lld, %lld) positive multiples of 16",
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
    const int64_t busy = n_groups < M ? n_groups : M;  // groups that can hold a row
    const int64_t tiles = (M / bp::TM + busy) * ((N + bp::TN - 1) / bp::TN);
    return launch_block_gemm(A, a_dtype, M, B, b_dtype, N * n_groups, false, tiles, a, (cudaStream_t)stream,
                             short_call_flops(2.0 * (double)M * (double)N * (double)K), "fp8_block_gemm_grouped");
}

extern "C" fp8dl_status fp8_block_gemm_grouped_wgrad(const uint8_t *A, int32_t a_dtype, const float *a_s,
                                                     const uint8_t *B, int32_t b_dtype, const float *b_s,
                                                     const int32_t *offsets, int32_t n_groups, int64_t M, int64_t N,
                                                     int64_t T, void *D, int32_t d_dtype, int32_t *dev_status,
                                                     fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_gemm_grouped_wgrad");
    if (!dim_ok(M, 1) || !block_tokens_ok(M) || !dim_ok(N, 16) || !block_tokens_ok(T) || T % 128 != 0)
        return fail(FP8DL_ERR_SHAPE, "M (%lld) must be positive, N (%lld) a positive multiple of 16 and T (%lld) a multiple of 128",
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
    const int64_t tiles = n_groups * ((M + bp::TM - 1) / bp::TM) * ((N + bp::TN - 1) / bp::TN);
    return launch_block_gemm(A, a_dtype, M, B, b_dtype, N, true, tiles, a, st,
                             short_call_flops(2.0 * (double)M * (double)N * (double)T), "fp8_block_gemm_grouped_wgrad");
}
