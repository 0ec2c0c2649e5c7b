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
    int raster_n;
    int64_t group;
};

// The groups' tables in shared memory: first[g], end[g] = the group's rows; pre[g] = units
// (row tiles, or token blocks) of the groups before g.
struct GroupTables {
    int32_t *first, *end, *pre;
};
constexpr int kGroupTableBytes = 3 * 4 * (kMaxGroups + 4);

__device__ __forceinline__ GroupTables group_tables(uint8_t *smem) {
    int32_t *p = reinterpret_cast<int32_t *>(smem);
    return {p, p + kMaxGroups + 4, p + 2 * (kMaxGroups + 4)};
}

// All threads of the block; `limit` caps the running sum (a reduction never reads past T).
__device__ __forceinline__ void build_groups(const GroupTables &t, const int32_t *offsets, int n_groups, int64_t rows,
                                             int unit, int64_t limit) {
    for (int g = threadIdx.x; g < n_groups; g += blockDim.x) {
        int64_t first, end;
        group_rows(offsets, g, rows, first, end);
        t.first[g] = (int32_t)first;
        t.end[g] = (int32_t)end;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int64_t before = 0;
        if (threadIdx.x == 0) t.pre[0] = 0;
        for (int g0 = 0; g0 < n_groups; g0 += 32) {
            const int g = g0 + threadIdx.x;
            const int64_t n = g < n_groups ? ((int64_t)t.end[g] - t.first[g] + unit - 1) / unit : 0;
            const int64_t sum = min(before + warp_inclusive_sum(n, threadIdx.x), limit);
            if (g < n_groups) t.pre[g + 1] = (int32_t)sum;
            before = __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    __syncthreads();
}

// The group that holds unit u: pre[g] <= u < pre[g + 1].
__device__ __forceinline__ int find_group(const GroupTables &t, int n_groups, int64_t u) {
    int lo = 0, hi = n_groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.pre[mid] <= u)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Tiles in bands of `band` tiles along one dimension, which varies fastest inside a band: the
// tiles in flight form a block whose operand panels are shared through L2.
__device__ __forceinline__ void band_order(int64_t tile, int64_t tiles_m, int64_t tiles_n, int along_n, int64_t band,
                                           int64_t &tm, int64_t &tn) {
    const int64_t inner = along_n ? tiles_n : tiles_m, outer = along_n ? tiles_m : tiles_n;
    const int64_t first = tile / (band * outer) * band;
    const int64_t width = min(band, inner - first), r = tile - first * outer;
    const int64_t i = first + r % width, o = r / width;
    tm = along_n ? o : i;
    tn = along_n ? i : o;
}

// One tile's work.
struct BlockTile {
    int64_t a_row, a_end;  // rows of A (and of D, but for BG_REDUCE) from a_row, valid below a_end
    int64_t n0;            // first column of D
    int64_t b_row;         // its row of B
    int kb0, kbs;          // reduction blocks
    const float *b_s;      // factors of B of the tile's matrix
    int64_t d_row0;        // added to A's row for D's row (BG_REDUCE)
};

template <int TM, int TN>
__device__ __forceinline__ int64_t block_tiles(const BlockGemmArgs &a, const GroupTables &t) {
    const int64_t tiles_n = (a.N + TN - 1) / TN, tiles_m = (a.M + TM - 1) / TM;
    if (a.kind == BG_DENSE) return tiles_m * tiles_n;
    if (a.kind == BG_ROWS) return (int64_t)t.pre[a.n_groups] * tiles_n;
    return a.n_groups * tiles_m * tiles_n;
}

template <int TM, int TN>
__device__ __forceinline__ BlockTile block_tile(const BlockGemmArgs &a, const GroupTables &t, int64_t tile) {
    const int64_t tiles_n = (a.N + TN - 1) / TN;
    BlockTile w;
    int64_t tm, tn;
    const int kbs = (int)((a.K + 127) / 128);
    w.kb0 = 0;
    w.kbs = kbs;
    w.b_s = a.b_s;
    w.d_row0 = 0;
    if (a.kind == BG_DENSE) {
        band_order(tile, (a.M + TM - 1) / TM, tiles_n, a.raster_n, a.group, tm, tn);
        w.a_row = tm * TM;
        w.a_end = a.M;
        w.n0 = w.b_row = tn * TN;
    } else if (a.kind == BG_ROWS) {
        const int g = find_group(t, a.n_groups, tile / tiles_n);
        band_order(tile - t.pre[g] * tiles_n, t.pre[g + 1] - t.pre[g], tiles_n, a.raster_n, a.group, tm, tn);
        w.a_row = t.first[g] + tm * TM;
        w.a_end = t.end[g];
        w.n0 = tn * TN;
        w.b_row = g * a.N + w.n0;
        w.b_s = a.b_s + (int64_t)g * kbs * a.b_ld;
    } else {
        const int64_t tiles_m = (a.M + TM - 1) / TM;
        const int64_t g = tile / (tiles_m * tiles_n);
        band_order(tile - g * tiles_m * tiles_n, tiles_m, tiles_n, a.raster_n, a.group, tm, tn);
        w.a_row = tm * TM;
        w.a_end = a.M;
        w.n0 = w.b_row = tn * TN;
        w.kb0 = t.pre[g];
        w.kbs = t.pre[g + 1] - t.pre[g];
        w.d_row0 = g * a.M;
    }
    return w;
}

// 32 consecutive columns n0 .. n0+31 of one row of D (bias added, rounded once).
__device__ __forceinline__ void store_row32(const BlockGemmArgs &a, int64_t row, int64_t n0, const float2 *v) {
    if (n0 >= a.N) return;
    float y[32];
#pragma unroll
    for (int p = 0; p < 16; p++) y[2 * p] = v[p].x, y[2 * p + 1] = v[p].y;
    if (a.bias_dtype == FP8DL_BF16) {
        const __nv_bfloat16 *b = static_cast<const __nv_bfloat16 *>(a.bias) + n0;
#pragma unroll
        for (int g = 0; g < 4; g++)
            if (n0 + 8 * g < a.N) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(b + 8 * g));
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int q = 0; q < 4; q++) y[8 * g + 2 * q] += bf16_lo(w[q]), y[8 * g + 2 * q + 1] += bf16_hi(w[q]);
            }
    } else if (a.bias_dtype == FP8DL_F32) {
        const float *b = static_cast<const float *>(a.bias) + n0;
#pragma unroll
        for (int g = 0; g < 8; g++)
            if (n0 + 4 * g < a.N) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(b + 4 * g));
                y[4 * g] += u.x, y[4 * g + 1] += u.y, y[4 * g + 2] += u.z, y[4 * g + 3] += u.w;
            }
    }
    if (a.d_dtype == FP8DL_BF16) {
        uint32_t w[16];
#pragma unroll
        for (int p = 0; p < 16; p++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * p], y[2 * p + 1]);
            w[p] = *reinterpret_cast<const uint32_t *>(&h);
        }
        __nv_bfloat16 *d = static_cast<__nv_bfloat16 *>(a.D) + row * a.N + n0;
#pragma unroll
        for (int h = 0; h < 2; h++) {  // sixteen columns at a time (N is a multiple of 16)
            if (n0 + 16 * h >= a.N) break;
            *reinterpret_cast<uint4 *>(d + 16 * h) = make_uint4(w[8 * h], w[8 * h + 1], w[8 * h + 2], w[8 * h + 3]);
            *reinterpret_cast<uint4 *>(d + 16 * h + 8) = make_uint4(w[8 * h + 4], w[8 * h + 5], w[8 * h + 6], w[8 * h + 7]);
        }
    } else {
        float *d = static_cast<float *>(a.D) + row * a.N + n0;
#pragma unroll
        for (int g = 0; g < 8; g++)
            if (n0 + 4 * g < a.N)
                *reinterpret_cast<float4 *>(d + 4 * g) = make_float4(y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]);
    }
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles on CTA pairs.
//   warp 0      TMA producer: 128 rows of A and 128 of B per CTA and k-block, six stages
//   warp 1      the leader's MMA thread: per block four MMAs (M 256, N 256, K 32) into one
//               of two 256-column tensor-memory buffers
//   warps 4-11  epilogue: warp w drains lane quarter w & 3 of column half (w - 4) / 4; a thread
//               holds one row x 128 columns of the sum (64 fp32 pairs)
// With 128 x 128 weight factors a thread's 128 columns share one factor per block: one
// packed multiply-add per two values, half the MMAs' time on the FP32 pipe.  With factors per
// row of B (BROWS, weight gradients) each column has its own: one more packed multiply.
// ---------------------------------------------------------------------------
namespace bp {
constexpr int TM = 256, TN = 256, BK = 128, STAGES = 6;
constexpr int A_BYTES = 128 * BK, B_BYTES = 128 * BK, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int THREADS = 384, EPI_WARPS = 8;
constexpr int REGS_LAUNCH = 168, REGS_IO = 40, REGS_EPI = 232;  // 128 * 40 + 256 * 232 = 384 * 168
static_assert(128 * REGS_IO + 256 * REGS_EPI <= THREADS * REGS_LAUNCH, "register split");
constexpr int TMEM_COLS = 512;
constexpr int CS_BYTES = EPI_WARPS * 2 * 128 * 4;  // column factors, double-buffered per warp
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + CS_BYTES + kGroupTableBytes + 1024;
}  // namespace bp

template <bool BROWS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(bp::THREADS, 1)
    block_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                           const BlockGemmArgs args) {
    using namespace bp;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
    uint8_t *bar_area = smem + STAGES * STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(bar_area);
    uint64_t *empty = full + STAGES;
    uint64_t *tfull = empty + STAGES;
    uint64_t *tempty = tfull + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tempty + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *cs_all = reinterpret_cast<float *>(bar_area + 1024);
    const GroupTables tab = group_tables(bar_area + 1024 + CS_BYTES);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < 2; a++) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 2 * EPI_WARPS);
        }
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_map(&tmap_a);
        tma_prefetch_map(&tmap_b);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers initialised before any cross-CTA signal
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    pdl_trigger();
    if (args.kind == BG_ROWS) build_groups(tab, args.offsets, args.n_groups, args.M, TM, 0x7fffffffll);
    if (args.kind == BG_REDUCE)
        build_groups(tab, args.offsets, args.n_groups, 0x7fffffffll, 128, args.K / 128);
    const int64_t tiles = block_tiles<TM, TN>(args, tab);

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_IO));
        if (warp == 0 && lane == 0) {  // ------------------------------------- producer (both CTAs)
            int s = 0;
            uint32_t ph = 0;
            int64_t issued = 0;
            bool ok = true;
            for (int64_t tile = pair; tile < tiles && ok; tile += npairs) {
                const BlockTile w = block_tile<TM, TN>(args, tab, tile);
                const int32_t ra = (int32_t)(w.a_row + rank * 128), rb = (int32_t)(w.b_row + rank * 128);
                for (int kb = 0; kb < w.kbs; kb++) {
                    if (!mbar_wait(smem_u32(&empty[s]), ph ^ 1, abort_flag, args.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb_local = smem_u32(&full[s]);
                    const uint32_t fb = mapa_shared(fb_local, 0);
                    if (leader) mbar_expect_tx(fb_local, 2 * STAGE_BYTES);
                    const uint32_t sa = smem_u32(smem + s * STAGE_BYTES);
                    tma_load_2d_pair(sa, &tmap_a, fb, (w.kb0 + kb) * BK, ra);
                    tma_load_2d_pair(sa + A_BYTES, &tmap_b, fb, (w.kb0 + kb) * BK, rb);
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
        } else if (warp == 1 && lane == 0 && leader) {  // --------------------- MMA issuer (leader only)
            int s = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true, any = false;
            uint32_t last_bar = 0, last_par = 0;
            const SDesc desc0 = sdesc_k_sw128_split(smem_u32(smem));
            for (int64_t tile = pair; tile < tiles && ok; tile += npairs) {
                const int kbs = block_tile<TM, TN>(args, tab, tile).kbs;
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
                        umma_f8f6f4_pair(tmem_base + (uint32_t)(buf * TN), sdesc_join(lo_a + 2 * kk, desc0.hi),
                                         sdesc_join(lo_b + 2 * kk, desc0.hi), args.idesc, kk != 0);
                    umma_commit_pair(smem_u32(&tfull[buf]), 0x3);
                    umma_commit_pair(smem_u32(&empty[s]), 0x3);
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
        }
    } else {  // ------------------------------------------------------------ epilogue (both CTAs)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t taddr0 = tmem_base + (uint32_t)(128 * half) + ((uint32_t)(32 * q) << 16);
        const uint32_t tempty_leader[2] = {mapa_shared(smem_u32(&tempty[0]), 0), mapa_shared(smem_u32(&tempty[1]), 0)};
        float *cs = cs_all + (warp - 4) * 256;
        int buf = 0;
        uint32_t bph = 0;
        bool ok = true;
        for (int64_t tile = pair; tile < tiles && ok; tile += npairs) {
            const BlockTile w = block_tile<TM, TN>(args, tab, tile);
            const int64_t row = w.a_row + rank * 128 + 32 * q + lane;
            const bool row_ok = row < w.a_end;
            const int64_t n0 = w.n0 + 128 * half;
            // factors of block kb: the row's, and the column half's (or, BROWS, the lane's four columns')
            const float *pa = args.a_s + (int64_t)w.kb0 * args.M + (row_ok ? row : 0);
            const float *pb = BROWS ? w.b_s + (int64_t)w.kb0 * args.b_ld + n0 + 4 * lane : w.b_s + n0 / 128;
            const bool b_ok = BROWS ? n0 + 4 * lane < args.N : n0 < args.N;
            auto load_a = [&](int kb) { return row_ok && kb < w.kbs ? __ldg(pa + kb * args.M) : 0.0f; };
            auto load_b = [&](int kb) -> float4 {
                if (!b_ok || kb >= w.kbs) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (BROWS) return __ldg(reinterpret_cast<const float4 *>(pb + kb * args.b_ld));
                return make_float4(__ldg(pb + kb * args.b_ld), 0.0f, 0.0f, 0.0f);
            };
            float2 acc[64];
#pragma unroll
            for (int p = 0; p < 64; p++) acc[p] = make_float2(0.0f, 0.0f);
            float sa0 = load_a(0), sa1 = load_a(1);
            float4 sb0 = load_b(0), sb1 = load_b(1);
            for (int kb = 0; kb < w.kbs; kb++) {
                const float sa2 = load_a(kb + 2);
                const float4 sb2 = load_b(kb + 2);
                float *csb = cs + (kb & 1) * 128;
                if (BROWS) {
                    *reinterpret_cast<float4 *>(csb + 4 * lane) = sb0;
                    __syncwarp();
                }
                const float2 sc = f2(BROWS ? sa0 : __fmul_rn(sa0, sb0.x));
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
                        if (lane == 0) mbar_arrive_cluster(tempty_leader[buf]);
                    }
#pragma unroll
                    for (int p = 0; p < 16; p++) {
                        const float2 t = make_float2(__uint_as_float(r[c & 1][2 * p]), __uint_as_float(r[c & 1][2 * p + 1]));
                        const float2 f = BROWS ? __fmul2_rn(sc, *reinterpret_cast<const float2 *>(csb + 32 * c + 2 * p)) : sc;
                        acc[16 * c + p] = __ffma2_rn(t, f, acc[16 * c + p]);
                    }
                }
                sa0 = sa1, sa1 = sa2;
                sb0 = sb1, sb1 = sb2;
                buf ^= 1;
                if (buf == 0) bph ^= 1;
            }
            if (ok && row_ok)
#pragma unroll
                for (int c = 0; c < 4; c++) store_row32(args, w.d_row0 + row, n0 + 32 * c, acc + 16 * c);
        }
    }

    tc_fence_before();
    __syncwarp();
    __syncthreads();
    cluster_sync();  // the peer's shared memory and TMEM stay live until the pair is done
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
static std::atomic<bool> g_block_set[64];
static int g_block_pairs[64];

static fp8dl_status block_gemm_setup(int dev, int sms) {
    if (g_block_set[dev].load(std::memory_order_acquire)) return FP8DL_OK;
    std::lock_guard<std::mutex> lock(init_mutex());
    if (g_block_set[dev].load(std::memory_order_relaxed)) return FP8DL_OK;
    const void *pairs[] = {(const void *)block_gemm_pair_kernel<false>, (const void *)block_gemm_pair_kernel<true>};
    int resident = 1 << 30;
    for (const void *k : pairs) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bp::SMEM_BYTES);
        cudaFuncAttributes fa = {};
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, k);
        if (e != cudaSuccess) return fail(FP8DL_ERR_CUDA, "block GEMM set-up: %s", cudaGetErrorString(e));
        // the epilogue's larger register share comes out of the launch's registers
        if (fa.numRegs < bp::REGS_LAUNCH)
            return fail(FP8DL_ERR_CUDA, "block GEMM: built with %d registers, %d needed", fa.numRegs, bp::REGS_LAUNCH);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(sms / 2 * 2), 1, 1);
        cfg.blockDim = dim3(bp::THREADS, 1, 1);
        cfg.dynamicSmemBytes = bp::SMEM_BYTES;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, k, &cfg);
        if (e != cudaSuccess || n < 1) {
            cudaGetLastError();
            return fail(FP8DL_ERR_UNSUPPORTED_DEVICE, "the block GEMM needs resident CTA-pair clusters");
        }
        resident = n < resident ? n : resident;
    }
    g_block_pairs[dev] = resident;
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
    FP8DL_TRY(block_gemm_setup(dev, sms));
    CUtensorMap ta, tb;
    FP8DL_TRY(encode_tmap_2d_u8(&ta, A, (uint64_t)args.K, (uint64_t)a_rows, (uint64_t)args.K, 128, 128,
                                CU_TENSOR_MAP_SWIZZLE_128B));
    FP8DL_TRY(encode_tmap_2d_u8(&tb, B, (uint64_t)args.K, (uint64_t)b_rows, (uint64_t)args.K, 128, 128,
                                CU_TENSOR_MAP_SWIZZLE_128B));
    args.idesc = (1u << 4) | ((uint32_t)a_dtype << 7) | ((uint32_t)b_dtype << 10) | ((uint32_t)(bp::TN >> 3) << 17) |
                 ((uint32_t)(bp::TM >> 4) << 24);
    const int64_t tiles_m = (args.M + bp::TM - 1) / bp::TM, tiles_n = (args.N + bp::TN - 1) / bp::TN;
    args.raster_n = tiles_n < tiles_m;
    args.group = args.K <= 8192 ? 16 : 8;
    const int64_t pairs = tiles_bound < g_block_pairs[dev] ? tiles_bound : g_block_pairs[dev];
    (void)launch_kernel(brows ? block_gemm_pair_kernel<true> : block_gemm_pair_kernel<false>, dim3((unsigned)(2 * pairs)),
                        bp::THREADS, bp::SMEM_BYTES, st, 0, pdl, ta, tb, args);
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
