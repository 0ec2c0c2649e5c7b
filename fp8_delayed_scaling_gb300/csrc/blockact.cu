// blockact.cu — activations between block-scaled products, with the argument kept in 8 bits for
// the backward pass, and transposed codes made from row-wise ones.
//
//   act      g = act(h) or act(a) * u, h = [a | u]: codes of g along the rows (the next product's
//            operand) and of h (the checkpoint), straight from fp32
//   dact     h from the checkpoint; dh = dg act'(h), or [dg u act'(a) | dg act(a)]: its codes along the rows
//            (dgrad's operand) and transposed (wgrad's); g again, transposed (the next product's wgrad operand)
//   recode   transposed codes of a matrix whose row-wise codes were kept
//
// GELU(a) = a Phi(a), GELU'(a) = Phi(a) + a phi(a) (the normal tail of common.cuh);
// SiLU(a) = a s, SiLU'(a) = s (1 + a (1 - s)), s = 1 / (1 + exp(-a)).
#include <cuda_fp16.h>

#include "block.cuh"

namespace fp8dl {

// Codes -> values, two at a time: FP8 is exact in fp16, fp16 in fp32.
__device__ __forceinline__ float2 decode2(uint32_t two, bool e4m3) {
    uint32_t h;
    if (e4m3)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    else
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// act(a) and, with D, its derivative.
template <bool SILU, bool D>
__device__ __forceinline__ void activation2(float2 a, float2 &y, float2 &d) {
    if (SILU) {
        const float2 t = __fmul2_rn(a, f2(-1.4426950409f));
        const float2 e = __fadd2_rn(make_float2(ex2_approx_ftz(t.x), ex2_approx_ftz(t.y)), f2(1.0f));
        const float2 s = make_float2(rcp_approx_ftz(e.x), rcp_approx_ftz(e.y));
        y = __fmul2_rn(a, s);
        if (D) d = __fmul2_rn(s, __ffma2_rn(a, __fadd2_rn(f2(1.0f), make_float2(-s.x, -s.y)), f2(1.0f)));
    } else {
        const NormalTail2 n = normal_tail2(a, make_float2(fabsf(a.x), fabsf(a.y)));
        const float2 up = __fadd2_rn(f2(1.0f), n.ntail);
        const float2 cdf = make_float2(a.x >= 0.0f ? up.x : -n.ntail.x, a.y >= 0.0f ? up.y : -n.ntail.y);
        y = __fmul2_rn(a, cdf);  // infinity stays infinity
        if (D) d = __ffma2_rn(__fmul2_rn(a, f2(0.3989422804f)), n.e, cdf);
    }
}

// ---------------------------------------------------------------------------
// act: blocks along the rows only, 16 lanes a block.
// ---------------------------------------------------------------------------
struct BlockActArgs {
    const void *h;
    int64_t rows, cols, wide;  // wide: columns of h
    const int32_t *offsets;
    int n_groups;
    uint8_t *g_q, *h_q;
    float *g_s, *h_s;
    uint32_t jobs;  // blocks of a row
    int split;
};

namespace ba {
constexpr int ACT_THREADS = 256, ACT_ROWS = 32;  // rows of a CTA: two for each 16 lanes
}

// Eight columns of a row in fp32; zeros where there are none.
template <int XKIND>
__device__ __forceinline__ void load8(const void *base, int64_t at, bool ok, float2 (&v)[4]) {
    if (XKIND == FP8DL_BF16) {
        const uint4 u = ok ? ldg_stream(static_cast<const char *>(base) + at * 2) : make_uint4(0u, 0u, 0u, 0u);
        v[0] = make_float2(bf16_lo(u.x), bf16_hi(u.x)), v[1] = make_float2(bf16_lo(u.y), bf16_hi(u.y));
        v[2] = make_float2(bf16_lo(u.z), bf16_hi(u.z)), v[3] = make_float2(bf16_lo(u.w), bf16_hi(u.w));
    } else {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint4 u = ok ? ldg_stream(static_cast<const char *>(base) + at * 4 + 16 * h) : make_uint4(0u, 0u, 0u, 0u);
            v[2 * h] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
            v[2 * h + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
        }
    }
}

// Codes and factor of one block held by 16 lanes, eight values each.
template <int FMT>
__device__ __forceinline__ void put_block(const float2 (&v)[4], bool ok, bool first, uint8_t *q, float *s) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) m = fmaxf(m, fmaxf(finite_abs(v[i].x), finite_abs(v[i].y)));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float2 sc = block_scale<FMT>(m);
    float2 y[4];
#pragma unroll
    for (int i = 0; i < 4; i++) y[i] = __fmul2_rn(v[i], f2(sc.x));
    if (ok)
        *reinterpret_cast<uint2 *>(q) =
            make_uint2(pack4<FMT>(y[0].x, y[0].y, y[1].x, y[1].y), pack4<FMT>(y[2].x, y[2].y, y[3].x, y[3].y));
    if (first) *s = sc.y;
}

// A CTA takes 32 rows of one block column (of a's and of u's where g is gated).  Where u's half does not start
// on a block (cols not a multiple of 128: `split`) h's blocks do not line up with g's: the codes of h
// are jobs of their own behind g's.
template <int XKIND, int FMT, bool GATED, bool SILU>
__global__ void __launch_bounds__(ba::ACT_THREADS) block_act_kernel(const BlockActArgs a) {
    using namespace ba;
    pdl_wait();
    pdl_trigger();
    const uint32_t tile = blockIdx.x / a.jobs, job = blockIdx.x % a.jobs, g_jobs = (uint32_t)((a.cols + 127) / 128);
    int64_t first = 0, end = a.rows;
    if (a.offsets) {  // blocks along the rows do not see the groups' borders
        group_rows(a.offsets, 0, a.rows, first, end);
        end = min(max((int64_t)a.offsets[a.n_groups], first), a.rows);
    }
    const int64_t r0 = first + (int64_t)tile * ACT_ROWS + (threadIdx.x >> 4);
    if (r0 - (threadIdx.x >> 4) >= end) return;
    const bool lead = (threadIdx.x & 15) == 0;
    const int64_t c = (int64_t)(job < g_jobs ? job : job - g_jobs) * 128 + 8 * (threadIdx.x & 15);
    if (job >= g_jobs) {  // h alone
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int64_t r = r0 + 16 * i;
            const bool ok = r < end && c < a.wide;
            float2 v[4];
            load8<XKIND>(a.h, r * a.wide + c, ok, v);
            put_block<FMT>(v, ok, lead && r < end, a.h_q + r * a.wide + c, a.h_s + (c >> 7) * a.rows + r);
        }
        return;
    }
    float2 va[2][4], vu[2][4];
    bool ok[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int64_t at = (r0 + 16 * i) * a.wide + c;
        ok[i] = r0 + 16 * i < end && c < a.cols;
        load8<XKIND>(a.h, at, ok[i], va[i]);
        if (GATED) load8<XKIND>(a.h, at + a.cols, ok[i], vu[i]);
    }
    const bool keep = a.h_q && !a.split;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int64_t r = r0 + 16 * i, at = r * a.wide + c;
        const bool put = lead && r < end;
        float2 y[4], none;
#pragma unroll
        for (int q = 0; q < 4; q++) {
            activation2<SILU, false>(va[i][q], y[q], none);
            if (GATED) y[q] = __fmul2_rn(y[q], vu[i][q]);
        }
        put_block<FMT>(y, ok[i], put, a.g_q + r * a.cols + c, a.g_s + (c >> 7) * a.rows + r);
        if (keep) {
            put_block<FMT>(va[i], ok[i], put, a.h_q + at, a.h_s + (c >> 7) * a.rows + r);
            if (GATED) put_block<FMT>(vu[i], ok[i], put, a.h_q + at + a.cols, a.h_s + ((c + a.cols) >> 7) * a.rows + r);
        }
    }
}

// ---------------------------------------------------------------------------
// 128 x 128 tiles with blocks along the rows and along the columns (dact, recode).
//   Threads  32 x 16, thread (rr, cc) holds rows 4rr .. 4rr+3 and columns 8cc .. 8cc+7 of each of
//            the tile's up to three matrices, in fp32 from the first computation to the codes.
//   Row      maxima over the 16 lanes that share a row by a halving exchange.
//   blocks
//   Column   maxima over 4 rows in the thread, halved over two row groups by shuffle, 16 warps
//   blocks   through shared memory.
//   Codes    transposed codes are packed along the rows (four from four registers), staged in
//            shared memory word by word, XOR-swizzled by column group (32 lanes hit 32 banks both
//            ways), and leave as whole 128-byte lines.
// ---------------------------------------------------------------------------
namespace bt {
constexpr int THREADS = 512, TILE = 128, WARPS = 16;
struct Matrix {            // shared memory of one of a tile's matrices
    uint8_t code[TILE * TILE];
    float part[WARPS][TILE];
    float scale[TILE];
};
typedef float2 Values[4][4];  // rows, pairs of columns
}

struct Where {  // a thread's place in its tile
    int64_t r0, c0;  // the tile's first row, the thread's first column
    int nrows;       // of the tile
    int rr, cc;
    bool col_ok;
};

// Codes of a tile's matrix along the rows; q, s: of the tensor, ld columns, `rows` factors in a row of s.
template <int FMT>
__device__ __forceinline__ void tile_rows(const bt::Values &v, const Where &w, uint8_t *q, float *s, int64_t ld, int64_t rows) {
    float m[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        m[i] = 0.0f;
#pragma unroll
        for (int p = 0; p < 4; p++) m[i] = fmaxf(m[i], fmaxf(fabsf(v[i][p].x), fabsf(v[i][p].y)));
    }
    if (fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) > 3.402823466e38f) {  // an infinity: over the finite values
#pragma unroll
        for (int i = 0; i < 4; i++) {
            m[i] = 0.0f;
#pragma unroll
            for (int p = 0; p < 4; p++) m[i] = fmaxf(m[i], fmaxf(finite_abs(v[i][p].x), finite_abs(v[i][p].y)));
        }
    }
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const bool up = lane & 8;
        const float send = up ? m[i] : m[i + 2], keep = up ? m[i + 2] : m[i];
        m[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 8));
    }
    const bool up = lane & 4;
    float top = fmaxf(up ? m[1] : m[0], __shfl_xor_sync(0xffffffffu, up ? m[0] : m[1], 4));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const float2 sc = block_scale<FMT>(top);  // of row (cc >> 2) of the thread's four
    const int row = 4 * w.rr + (w.cc >> 2);
    if ((w.cc & 3) == 0 && row < w.nrows) s[(w.c0 >> 7) * rows + w.r0 + row] = sc.y;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 s2 = f2(__shfl_sync(0xffffffffu, sc.x, (lane & 16) + 4 * i));
        float2 y[4];
#pragma unroll
        for (int p = 0; p < 4; p++) y[p] = __fmul2_rn(v[i][p], s2);
        if (w.col_ok && 4 * w.rr + i < w.nrows)
            *reinterpret_cast<uint2 *>(q + (w.r0 + 4 * w.rr + i) * ld + w.c0) = make_uint2(
                pack4<FMT>(y[0].x, y[0].y, y[1].x, y[1].y), pack4<FMT>(y[2].x, y[2].y, y[3].x, y[3].y));
    }
}

// The warp's column maxima into shared memory.
__device__ __forceinline__ void tile_maxima(const bt::Values &v, const Where &w, bt::Matrix &sm) {
    const int lane = threadIdx.x & 31;
    float m[8], top = 0.0f;
#pragma unroll
    for (int p = 0; p < 4; p++) {
        m[2 * p] = fmaxf(fmaxf(fabsf(v[0][p].x), fabsf(v[1][p].x)), fmaxf(fabsf(v[2][p].x), fabsf(v[3][p].x)));
        m[2 * p + 1] = fmaxf(fmaxf(fabsf(v[0][p].y), fabsf(v[1][p].y)), fmaxf(fabsf(v[2][p].y), fabsf(v[3][p].y)));
        top = fmaxf(top, fmaxf(m[2 * p], m[2 * p + 1]));
    }
    if (top > 3.402823466e38f) {
#pragma unroll
        for (int p = 0; p < 4; p++) {
            m[2 * p] = m[2 * p + 1] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                m[2 * p] = fmaxf(m[2 * p], finite_abs(v[i][p].x));
                m[2 * p + 1] = fmaxf(m[2 * p + 1], finite_abs(v[i][p].y));
            }
        }
    }
    const bool up = lane & 16;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float send = up ? m[j] : m[j + 4], keep = up ? m[j + 4] : m[j];
        m[j] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 16));
    }
    *reinterpret_cast<float4 *>(&sm.part[threadIdx.x >> 5][8 * w.cc + (up ? 4 : 0)]) = make_float4(m[0], m[1], m[2], m[3]);
}

// The warp's column sums (rows in a fixed order) into shared memory, where the codes will be.
__device__ __forceinline__ void tile_sums(const bt::Values &v, const Where &w, bt::Matrix &sm) {
    const int lane = threadIdx.x & 31;
    float m[8];
#pragma unroll
    for (int p = 0; p < 4; p++) {
        const float2 t = __fadd2_rn(__fadd2_rn(v[0][p], v[1][p]), __fadd2_rn(v[2][p], v[3][p]));
        m[2 * p] = t.x, m[2 * p + 1] = t.y;
    }
    const bool up = lane & 16;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float send = up ? m[j] : m[j + 4], keep = up ? m[j + 4] : m[j];
        m[j] = keep + __shfl_xor_sync(0xffffffffu, send, 16);
    }
    float *to = reinterpret_cast<float *>(sm.code) + (threadIdx.x >> 5) * bt::TILE + 8 * w.cc + (up ? 4 : 0);
    *reinterpret_cast<float4 *>(to) = make_float4(m[0], m[1], m[2], m[3]);
}

// Scale and factor of column c of the tile; its sum, if `sums` is not NULL.  After a barrier.
template <int FMT>
__device__ __forceinline__ void tile_scale(bt::Matrix &sm, int c, float *s, float *sums) {
    float m = sm.part[0][c];
#pragma unroll
    for (int w = 1; w < bt::WARPS; w++) m = fmaxf(m, sm.part[w][c]);
    const float2 sc = block_scale<FMT>(m);
    sm.scale[c] = sc.x;
    if (s) *s = sc.y;
    if (sums) {
        const float *from = reinterpret_cast<const float *>(sm.code);
        float t = from[c];
#pragma unroll
        for (int w = 1; w < bt::WARPS; w++) t += from[w * bt::TILE + c];
        *sums = t;
    }
}

// Transposed codes into shared memory.  After a barrier.
template <int FMT>
__device__ __forceinline__ void tile_stage(const bt::Values &v, const Where &w, bt::Matrix &sm) {
    uint32_t *words = reinterpret_cast<uint32_t *>(sm.code) + (w.rr ^ (2 * w.cc));
#pragma unroll
    for (int p = 0; p < 4; p++) {  // columns 8cc + 2p and the next
        const float2 sc = *reinterpret_cast<const float2 *>(&sm.scale[8 * w.cc + 2 * p]);
        float2 y[4];
#pragma unroll
        for (int i = 0; i < 4; i++) y[i] = __fmul2_rn(v[i][p], sc);
        words[(8 * w.cc + 2 * p) * 32] = pack4<FMT>(y[0].x, y[1].x, y[2].x, y[3].x);
        words[(8 * w.cc + 2 * p + 1) * 32] = pack4<FMT>(y[0].y, y[1].y, y[2].y, y[3].y);
    }
}

// The staged codes to their columns: q at the tile's first column, ld its row length, `cols` of the
// tile's columns exist.  After a barrier.
__device__ __forceinline__ void tile_out(const bt::Matrix &sm, uint8_t *q, int64_t ld, int cols) {
    const int ch = threadIdx.x & 7;
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const int c = (threadIdx.x >> 3) + 64 * k, g = c >> 3;
        uint4 u = *reinterpret_cast<const uint4 *>(sm.code + c * bt::TILE + ((ch ^ (g >> 1)) << 4));
        if (g & 1) u = make_uint4(u.z, u.w, u.x, u.y);
        if (c < cols) *reinterpret_cast<uint4 *>(q + c * ld + 16 * ch) = u;
    }
}

struct BlockDactArgs {
    const void *dg;
    int64_t rows, cols, wide;  // wide: columns of h
    const uint8_t *h_q;
    const float *h_s;
    const int32_t *offsets;
    int n_groups;
    uint8_t *dh_q, *dh_qt, *g_qt;
    float *dh_s, *dh_st, *g_st;
    int64_t col_ld;
    float *ws;              // column sums of dh per 128-row tile, or NULL
    uint32_t tiles, across;  // tiles down (of the padded order, at most) and across
    uint32_t row_first, row_jobs;  // blocks along the rows that block_dact_rows_kernel makes: the first, how many
    int bf16, h_e4;         // dg's type; the checkpoint's format (and g's): E4M3, else E5M2
};

// cp.async of N bytes, zeros where !ok (nothing is read then).
template <int N>
__device__ __forceinline__ void copy_async(void *smem, const void *global, bool ok) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(smem)), n = ok ? N : 0;
    if (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(global), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(global), "n"(N), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Eight codes -> fp16 pairs.  (volatile: a branch, not both conversions and a select.)
__device__ __forceinline__ void decode8(uint2 u, bool e4m3, uint32_t (&h)[4]) {
    if (e4m3) {
        asm volatile("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}"
                     : "=r"(h[0]), "=r"(h[1]) : "r"(u.x));
        asm volatile("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}"
                     : "=r"(h[2]), "=r"(h[3]) : "r"(u.y));
    } else {  // E5M2 is the upper byte of an fp16
        h[0] = __byte_perm(u.x, 0, 0x1404), h[1] = __byte_perm(u.x, 0, 0x3424);
        h[2] = __byte_perm(u.y, 0, 0x1404), h[3] = __byte_perm(u.y, 0, 0x3424);
    }
}

// dh (and g) of two elements: every caller rounds in this order, so that the same element has the same
// bits whichever kernel computes it.
template <bool GATED, bool SILU>
__device__ __forceinline__ void gradient2(uint32_t ha, float fa, uint32_t hu, float fu, float2 dg, float2 &da, float2 &du,
                                          float2 &g) {
    float2 y, d;
    activation2<SILU, true>(__fmul2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&ha)), f2(fa)), y, d);
    if (GATED) {
        const float2 u = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&hu)), f2(fu));
        g = __fmul2_rn(y, u);
        da = __fmul2_rn(__fmul2_rn(dg, u), d);
        du = __fmul2_rn(dg, y);
    } else {
        g = y;
        da = __fmul2_rn(dg, d);
    }
}

// The transposed codes, column sums and, where whole blocks line up with the tiles, the codes along the
// rows: a persistent CTA per SM walks 128 x 128 tiles of g's columns.
//   Reads    each thread copies what it will itself read of the next tile (dg and codes: 32 values of each)
//            into its own slots in shared memory, right after it has read this tile's: a tile's loads are
//            under way while the one before it is computed, without registers or a barrier for them.
//            The rows' factors (a few hundred floats) are copied by the first warps.
//   Values   of da, du and g in fp32 (96 registers) from one decoding and one activation.
//   Work     a tile of 16384 values takes 144 KB of traffic and about 25 instructions a value: HBM and the
//            issue slots are about even, so what counts is that neither waits.
// 8192 x 11008 swiglu, bf16, bias gradient: see the end of the file's entry for the figures.
template <int FMT, bool GATED, bool SILU>
__global__ void __launch_bounds__(bt::THREADS, 1) block_dact_kernel(const BlockDactArgs a) {
    using namespace bt;
    constexpr int NM = GATED ? 3 : 2, NH = NM - 1;  // matrices, those of dh
    constexpr int NF = GATED ? 3 : 1;  // factors of a row: a's block, u's, and the next where a tile of u spans two
    extern __shared__ __align__(16) uint8_t dyn[];
    Matrix *sm = reinterpret_cast<Matrix *>(dyn);                       // da, [du,] g
    uint4 *in_dg = reinterpret_cast<uint4 *>(sm + NM);                  // [8][THREADS] (bf16: half of it)
    uint2 *in_h = reinterpret_cast<uint2 *>(in_dg + 8 * THREADS);       // [4 * NH][THREADS]
    float *fac = reinterpret_cast<float *>(in_h + 4 * NH * THREADS);    // [2][NF][TILE]
    __shared__ GroupTable table;
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    uint32_t down = a.tiles;
    if (a.offsets) {
        build_group_table(table, a.offsets, a.n_groups, a.rows);
        down = min(down, table.before[a.n_groups]);
    }
    const uint32_t total = down * a.across;
    Where w;
    w.rr = tid >> 4, w.cc = tid & 15;
    int64_t next_r0 = 0;
    int next_n = 0;
    const auto place = [&](uint32_t t) {
        const uint32_t tile = t / a.across;
        if (a.offsets) {
            find_group(table, a.n_groups, tile, next_r0, next_n);
        } else {
            next_r0 = (int64_t)tile * TILE;
            next_n = (int)min((int64_t)TILE, a.rows - next_r0);
        }
    };
    const auto fetch_row = [&](int i, int64_t c) {  // row i of the thread's four, columns c ..
        const bool ok = c < a.cols && 4 * w.rr + i < next_n;
        const int64_t r = next_r0 + 4 * w.rr + i;
        if (a.bf16) {
            copy_async<16>(in_dg + i * THREADS + tid, static_cast<const char *>(a.dg) + (ok ? (r * a.cols + c) * 2 : 0), ok);
        } else {
            const char *p = static_cast<const char *>(a.dg) + (ok ? (r * a.cols + c) * 4 : 0);
            copy_async<16>(in_dg + 2 * i * THREADS + tid, p, ok);
            copy_async<16>(in_dg + (2 * i + 1) * THREADS + tid, p + 16, ok);
        }
        const uint8_t *q = a.h_q + (ok ? r * a.wide + c : 0);
        copy_async<8>(in_h + i * THREADS + tid, q, ok);
        if (GATED) copy_async<8>(in_h + (4 + i) * THREADS + tid, q + (ok ? a.cols : 0), ok);
    };
    const auto fetch_factors = [&](int slot, int64_t first) {
        if (tid < NF * TILE) {
            const int which = tid / TILE, row = tid % TILE;
            const int64_t block = ((first + (which ? a.cols : 0)) >> 7) + (which == 2);
            const bool ok = row < next_n && block * 128 < a.wide;
            copy_async<4>(fac + slot * NF * TILE + tid, a.h_s + (ok ? block * a.rows + next_r0 + row : 0), ok);
        }
    };
    uint32_t t = blockIdx.x;
    if (t < total) {
        place(t);
        const int64_t first = (int64_t)(t % a.across) * TILE;
#pragma unroll
        for (int i = 0; i < 4; i++) fetch_row(i, first + 8 * w.cc);
        fetch_factors(0, first);
    }
    for (int slot = 0; t < total; t += gridDim.x, slot ^= 1) {
        const uint32_t tile = t / a.across;
        const int64_t first = (int64_t)(t - tile * a.across) * TILE;
        w.r0 = next_r0, w.nrows = next_n;
        w.c0 = first + 8 * w.cc;
        w.col_ok = w.c0 < a.cols;
        const uint32_t u = t + gridDim.x;
        const bool more = u < total;
        const int64_t ufirst = more ? (int64_t)(u % a.across) * TILE : 0;
        copy_wait_all();
        __syncthreads();  // the factors have come, the last tile's codes have gone
        if (more) {
            place(u);
            fetch_factors(slot ^ 1, ufirst);
        }
        const float *fa_of = fac + slot * NF * TILE + 4 * w.rr;
        const float *fu_of = fa_of + (((w.c0 + a.cols) >> 7) != ((first + a.cols) >> 7) ? 2 : 1) * TILE;
        Values v[NM];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float2 dg[4];
            if (a.bf16) {
                const uint4 x = in_dg[i * THREADS + tid];
                dg[0] = make_float2(bf16_lo(x.x), bf16_hi(x.x)), dg[1] = make_float2(bf16_lo(x.y), bf16_hi(x.y));
                dg[2] = make_float2(bf16_lo(x.z), bf16_hi(x.z)), dg[3] = make_float2(bf16_lo(x.w), bf16_hi(x.w));
            } else {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const uint4 x = in_dg[(2 * i + h) * THREADS + tid];
                    dg[2 * h] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
                    dg[2 * h + 1] = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
                }
            }
            uint32_t ha[4], hu[4];
            decode8(in_h[i * THREADS + tid], a.h_e4, ha);
            if (GATED) decode8(in_h[(4 + i) * THREADS + tid], a.h_e4, hu);
            const float fa = fa_of[i], fu = GATED ? fu_of[i] : 0.0f;
            if (more) fetch_row(i, ufirst + 8 * w.cc);
#pragma unroll
            for (int p = 0; p < 4; p++)
                gradient2<GATED, SILU>(ha[p], fa, GATED ? hu[p] : 0u, fu, dg[p], v[0][i][p], v[NH - 1][i][p], v[NM - 1][i][p]);
        }
        if (a.dh_q && first < (int64_t)a.row_first * TILE) {
            tile_rows<FMT>(v[0], w, a.dh_q, a.dh_s, a.wide, a.rows);
            if (GATED && a.row_jobs == 0) {  // u's blocks line up too
                Where wu = w;
                wu.c0 += a.cols;
                tile_rows<FMT>(v[NH - 1], wu, a.dh_q, a.dh_s, a.wide, a.rows);
            }
        }
#pragma unroll
        for (int m = 0; m < NM; m++) {
            if (m < NH ? !a.dh_qt : !a.g_qt) continue;
            tile_maxima(v[m], w, sm[m]);
        }
        if (a.ws) {
#pragma unroll
            for (int m = 0; m < NH; m++) tile_sums(v[m], w, sm[m]);
        }
        __syncthreads();
        if (tid < NM * TILE) {
            const int m = tid / TILE, c = tid % TILE;
            if (first + c < a.cols) {
                if (m < NH) {
                    const int64_t at = (int64_t)tile * a.wide + first + c + (m ? a.cols : 0);
                    tile_scale<FMT>(sm[m], c, a.dh_qt ? a.dh_st + at : nullptr, a.ws ? a.ws + at : nullptr);
                } else if (a.g_qt) {
                    float *to = a.g_st + (int64_t)tile * a.cols + first + c;
                    if (a.h_e4)
                        tile_scale<FP8DL_E4M3>(sm[m], c, to, nullptr);
                    else
                        tile_scale<FP8DL_E5M2>(sm[m], c, to, nullptr);
                }
            }
        }
        __syncthreads();
        if (a.dh_qt) {
#pragma unroll
            for (int m = 0; m < NH; m++) tile_stage<FMT>(v[m], w, sm[m]);
        }
        if (a.g_qt) {
            if (a.h_e4)
                tile_stage<FP8DL_E4M3>(v[NM - 1], w, sm[NM - 1]);
            else
                tile_stage<FP8DL_E5M2>(v[NM - 1], w, sm[NM - 1]);
        }
        __syncthreads();
        const int left = (int)min((int64_t)TILE, a.cols - first);
#pragma unroll
        for (int m = 0; m < NM; m++) {
            uint8_t *q = m < NH ? a.dh_qt : a.g_qt;
            if (q) tile_out(sm[m], q + (first + (GATED && m == 1 ? a.cols : 0)) * a.col_ld + (int64_t)tile * TILE, a.col_ld, left);
        }
    }
}

// Blocks of dh along the rows, a.row_jobs of a row from a.row_first on: all of them where nothing else is
// wanted; those of u's half (and the one that holds the border) where cols is not a multiple of 128 and
// the tiles above do not hold whole blocks.  16 lanes a block, two rows of each in flight.
template <int FMT, bool GATED, bool SILU>
__global__ void __launch_bounds__(ba::ACT_THREADS) block_dact_rows_kernel(const BlockDactArgs a) {
    using namespace ba;
    pdl_wait();
    pdl_trigger();
    const uint32_t tile = blockIdx.x / a.row_jobs, job = a.row_first + blockIdx.x % a.row_jobs;
    int64_t first = 0, end = a.rows;
    if (a.offsets) {
        group_rows(a.offsets, 0, a.rows, first, end);
        end = min(max((int64_t)a.offsets[a.n_groups], first), a.rows);
    }
    const int64_t r0 = first + (int64_t)tile * ACT_ROWS + (threadIdx.x >> 4);
    if (r0 - (threadIdx.x >> 4) >= end) return;
    const bool lead = (threadIdx.x & 15) == 0;
    const int64_t at = (int64_t)job * 128 + 8 * (threadIdx.x & 15);  // of dh
    const bool right = GATED && at >= a.cols;
    const int64_t c = right ? at - a.cols : at;
    float2 dg[2][4];
    uint2 qa[2], qu[2];
    float fa[2], fu[2];
    bool ok[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int64_t r = r0 + 16 * i;
        ok[i] = r < end && at < a.wide;
        qa[i] = qu[i] = make_uint2(0u, 0u);
        fa[i] = fu[i] = 0.0f;
        if (a.bf16)
            load8<FP8DL_BF16>(a.dg, r * a.cols + c, ok[i], dg[i]);
        else
            load8<FP8DL_F32>(a.dg, r * a.cols + c, ok[i], dg[i]);
        if (ok[i]) {
            qa[i] = *reinterpret_cast<const uint2 *>(a.h_q + r * a.wide + c);
            fa[i] = a.h_s[(c >> 7) * a.rows + r];
            if (GATED && !right) {
                qu[i] = *reinterpret_cast<const uint2 *>(a.h_q + r * a.wide + c + a.cols);
                fu[i] = a.h_s[((c + a.cols) >> 7) * a.rows + r];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int64_t r = r0 + 16 * i;
        uint32_t ha[4], hu[4];
        decode8(qa[i], a.h_e4, ha);
        if (GATED) decode8(qu[i], a.h_e4, hu);
        float2 v[4], du, g;
#pragma unroll
        for (int p = 0; p < 4; p++) {
            gradient2<GATED, SILU>(ha[p], fa[i], GATED ? hu[p] : 0u, fu[i], dg[i][p], v[p], du, g);
            if (GATED && right) v[p] = du;
        }
        put_block<FMT>(v, ok[i], lead && r < end, a.dh_q + r * a.wide + at, a.dh_s + (at >> 7) * a.rows + r);
    }
}

template <int FMT, bool GATED, bool SILU>
static fp8dl_status launch_dact(const BlockDactArgs &a, bool tiles, int sms, cudaStream_t st, bool pdl) {
    using namespace bt;
    if (tiles) {
        constexpr int NM = GATED ? 3 : 2;
        constexpr size_t smem = NM * sizeof(Matrix) + 8 * THREADS * 16 + 4 * (NM - 1) * THREADS * 8 + 2 * (GATED ? 3 : 1) * TILE * 4;
        auto *kernel = block_dact_kernel<FMT, GATED, SILU>;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return fail(FP8DL_ERR_CUDA, "fp8_block_dact: %s", cudaGetErrorString(e));
        const int64_t most = (int64_t)a.tiles * a.across;
        (void)launch_kernel(kernel, dim3((unsigned)(most < sms ? most : sms)), dim3(THREADS), smem, st, 0, pdl, a);
        note_launch();
        FP8DL_TRY(check_launch("fp8_block_dact"));
    }
    if (a.dh_q && a.row_jobs) {
        const int64_t ctas = (a.rows + ba::ACT_ROWS - 1) / ba::ACT_ROWS * a.row_jobs;
        (void)launch_kernel(block_dact_rows_kernel<FMT, GATED, SILU>, dim3((unsigned)ctas), dim3(ba::ACT_THREADS), 0, st, 0, pdl, a);
        note_launch();
        FP8DL_TRY(check_launch("fp8_block_dact(rows)"));
    }
    return FP8DL_OK;
}

// The rows of tile `tile` of the padded order; false where there are none.
__device__ __forceinline__ bool tile_place(const int32_t *offsets, int n_groups, int64_t rows, uint32_t tile, Where &w) {
    w.rr = threadIdx.x >> 4;
    w.cc = threadIdx.x & 15;
    w.r0 = (int64_t)tile * bt::TILE;
    w.nrows = (int)min((int64_t)bt::TILE, rows - w.r0);
    if (offsets) group_of_block(offsets, n_groups, rows, tile, w.r0, w.nrows);
    return w.nrows > 0;
}

struct BlockRecodeArgs {
    const uint8_t *q;
    const float *s;
    int64_t src_rows, rows, cols;
    const int32_t *index, *offsets;
    int n_groups;
    uint8_t *col_q;
    float *col_s;
    int64_t col_ld;
    uint32_t jobs;
    int e4;
};

template <int FMT>
__global__ void __launch_bounds__(bt::THREADS) block_recode_kernel(const BlockRecodeArgs a) {
    using namespace bt;
    __shared__ __align__(16) Matrix sm;
    pdl_wait();
    pdl_trigger();
    const uint32_t tile = blockIdx.x / a.jobs;
    Where w;
    if (!tile_place(a.offsets, a.n_groups, a.rows, tile, w)) return;
    const int64_t first = (int64_t)(blockIdx.x % a.jobs) * TILE;
    w.c0 = first + 8 * w.cc;
    w.col_ok = w.c0 < a.cols;
    Values v;
    uint2 u[4];
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        u[i] = make_uint2(0u, 0u);
        f[i] = 0.0f;
        if (w.col_ok && 4 * w.rr + i < w.nrows) {
            int64_t r = w.r0 + 4 * w.rr + i;
            if (a.index) r = a.index[r];
            if (r >= 0 && r < a.src_rows) {
                u[i] = *reinterpret_cast<const uint2 *>(a.q + r * a.cols + w.c0);
                f[i] = a.s[(w.c0 >> 7) * a.src_rows + r];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[i][0] = __fmul2_rn(decode2(u[i].x, a.e4), f2(f[i])), v[i][1] = __fmul2_rn(decode2(u[i].x >> 16, a.e4), f2(f[i]));
        v[i][2] = __fmul2_rn(decode2(u[i].y, a.e4), f2(f[i])), v[i][3] = __fmul2_rn(decode2(u[i].y >> 16, a.e4), f2(f[i]));
    }
    tile_maxima(v, w, sm);
    __syncthreads();
    if (threadIdx.x < TILE && first + threadIdx.x < a.cols)
        tile_scale<FMT>(sm, threadIdx.x, a.col_s + (int64_t)tile * a.cols + first + threadIdx.x, nullptr);
    __syncthreads();
    tile_stage<FMT>(v, w, sm);
    __syncthreads();
    tile_out(sm, a.col_q + first * a.col_ld + (int64_t)tile * TILE, a.col_ld, (int)min((int64_t)TILE, a.cols - first));
}

static fp8dl_status check_tiles(int64_t tiles, int64_t rows, int64_t cols) {
    if (tiles > 0x7fffffffll)
        return fail(FP8DL_ERR_SHAPE, "%lld x %lld is more than 2^31 - 1 tiles", (long long)rows, (long long)cols);
    return FP8DL_OK;
}

static bool fp8_ok(int32_t f) { return f == FP8DL_E4M3 || f == FP8DL_E5M2; }
static bool act_gated(int32_t act) { return act == FP8DL_ACT_GEGLU || act == FP8DL_ACT_SWIGLU; }
static bool act_silu(int32_t act) { return act == FP8DL_ACT_SILU || act == FP8DL_ACT_SWIGLU; }

// What fp8_block_act and fp8_block_dact check alike; cols of g, h has twice as many where g is gated.
static fp8dl_status check_act(int32_t dtype, int32_t act, int64_t rows, int64_t cols, const int32_t *offsets, int32_t n_groups,
                              int32_t out_dtype) {
    FP8DL_CHECK_ARG(dtype == FP8DL_F32 || dtype == FP8DL_BF16, "the type must be FP8DL_F32 or FP8DL_BF16");
    FP8DL_CHECK_ARG(act >= FP8DL_ACT_GELU && act <= FP8DL_ACT_SWIGLU, "act must be one of fp8dl_activation");
    FP8DL_CHECK_ARG(fp8_ok(out_dtype), "out_dtype must be E4M3 or E5M2");
    if (!block_tokens_ok(rows) || !dim_ok(cols, 16) || cols > (int64_t(1) << 30))
        return fail(FP8DL_ERR_SHAPE, "rows (%lld) must be in [0, 2^31) and cols (%lld) a positive multiple of 16, at most 2^30",
                    (long long)rows, (long long)cols);
    return check_block_groups(offsets, n_groups, true);
}

}  // namespace fp8dl

using namespace fp8dl;

extern "C" fp8dl_status fp8_block_act(const void *h, int32_t h_dtype, int32_t act, int64_t rows, int64_t cols,
                                      const int32_t *offsets, int32_t n_groups, int32_t out_dtype, uint8_t *g_q,
                                      float *g_s, uint8_t *h_q, float *h_s, fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_act");
    FP8DL_TRY(check_act(h_dtype, act, rows, cols, offsets, n_groups, out_dtype));
    FP8DL_CHECK_ARG(rows == 0 || (h && g_q && g_s), "h, g_q and g_s must be non-NULL");
    FP8DL_CHECK_ARG(!h_q == !h_s, "h_q and h_s come together");
    if (!aligned16(h) || !aligned16(g_q) || !aligned16(g_s) || !aligned16(h_q) || !aligned16(h_s))
        return fail(FP8DL_ERR_ALIGN, "h, g_q, g_s, h_q and h_s must be 16-byte aligned");
    const bool gated = act_gated(act);
    BlockActArgs a = {};
    a.h = h;
    a.rows = rows;
    a.cols = cols;
    a.wide = gated ? 2 * cols : cols;
    a.offsets = offsets;
    a.n_groups = n_groups;
    a.g_q = g_q, a.h_q = h_q, a.g_s = g_s, a.h_s = h_s;
    a.split = gated && cols % 128 != 0;
    a.jobs = (uint32_t)((cols + 127) / 128 + (a.split && h_q ? (a.wide + 127) / 128 : 0));
    const int64_t ctas = (rows + ba::ACT_ROWS - 1) / ba::ACT_ROWS * a.jobs;
    FP8DL_TRY(check_tiles(ctas, rows, cols));
    FP8DL_TRY(current_device(nullptr, nullptr));
    if (rows == 0) return FP8DL_OK;
    const bool pdl = short_call_bytes((double)rows * a.wide * ((h_dtype == FP8DL_BF16 ? 2.0 : 4.0) + (h_q ? 1.0 : 0.0)) + (double)rows * cols);
    auto *kernel = &block_act_kernel<FP8DL_BF16, FP8DL_E4M3, false, false>;
#define FP8DL_ACT(X, F)                                                                                      \
    kernel = gated ? (act_silu(act) ? block_act_kernel<X, F, true, true> : block_act_kernel<X, F, true, false>) \
                   : (act_silu(act) ? block_act_kernel<X, F, false, true> : block_act_kernel<X, F, false, false>)
    if (h_dtype == FP8DL_BF16 && out_dtype == FP8DL_E4M3) FP8DL_ACT(FP8DL_BF16, FP8DL_E4M3);
    else if (h_dtype == FP8DL_BF16) FP8DL_ACT(FP8DL_BF16, FP8DL_E5M2);
    else if (out_dtype == FP8DL_E4M3) FP8DL_ACT(FP8DL_F32, FP8DL_E4M3);
    else FP8DL_ACT(FP8DL_F32, FP8DL_E5M2);
#undef FP8DL_ACT
    (void)launch_kernel(kernel, dim3((unsigned)ctas), dim3(ba::ACT_THREADS), 0, (cudaStream_t)stream, 0, pdl, a);
    note_launch();
    return check_launch("fp8_block_act");
}

extern "C" fp8dl_status fp8_block_dact(const void *dg, int32_t dg_dtype, int32_t act, int64_t rows, int64_t cols,
                                       const uint8_t *h_q, int32_t h_fp8, const float *h_s, const int32_t *offsets,
                                       int32_t n_groups, int32_t out_dtype, uint8_t *dh_q, float *dh_s, uint8_t *dh_qt,
                                       float *dh_st, uint8_t *g_qt, float *g_st, float *dbias, void *workspace,
                                       size_t workspace_bytes, fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_dact");
    FP8DL_TRY(check_act(dg_dtype, act, rows, cols, offsets, n_groups, out_dtype));
    FP8DL_CHECK_ARG(fp8_ok(h_fp8), "h_fp8 must be E4M3 or E5M2");
    FP8DL_CHECK_ARG(!offsets || !dbias, "dbias is the sum over all rows: not with offsets");
    FP8DL_CHECK_ARG(rows == 0 || (dg && h_q && h_s), "dg, h_q and h_s must be non-NULL");
    FP8DL_CHECK_ARG(rows == 0 || dh_q || dh_qt || g_qt || dbias, "dh_q, dh_qt, g_qt and dbias are all NULL");
    FP8DL_CHECK_ARG(rows == 0 || (!dh_q == !dh_s && !dh_qt == !dh_st && !g_qt == !g_st),
                    "dh_q/dh_s, dh_qt/dh_st and g_qt/g_st come in pairs");
    if (!aligned16(dg) || !aligned16(h_q) || !aligned16(h_s) || !aligned16(dh_q) || !aligned16(dh_s) || !aligned16(dh_qt) ||
        !aligned16(dh_st) || !aligned16(g_qt) || !aligned16(g_st) || !aligned16(dbias))
        return fail(FP8DL_ERR_ALIGN, "the tensors must be 16-byte aligned");
    const bool gated = act_gated(act);
    const int64_t wide = gated ? 2 * cols : cols;
    if (dbias && rows > 0) {
        if (!workspace || workspace_bytes < fp8_cast_workspace_size(rows, wide))
            return fail(FP8DL_ERR_WORKSPACE, "dbias needs a workspace of %zu bytes (got %zu)", fp8_cast_workspace_size(rows, wide),
                        workspace ? workspace_bytes : (size_t)0);
        if (!aligned16(workspace)) return fail(FP8DL_ERR_ALIGN, "workspace must be 16-byte aligned");
    }
    BlockDactArgs a = {};
    a.dg = dg;
    a.rows = rows;
    a.cols = cols;
    a.wide = wide;
    a.h_q = h_q, a.h_s = h_s;
    a.offsets = offsets;
    a.n_groups = n_groups;
    a.dh_q = dh_q, a.dh_qt = dh_qt, a.g_qt = g_qt, a.dh_s = dh_s, a.dh_st = dh_st, a.g_st = g_st;
    a.col_ld = fp8_block_padded_rows(rows, n_groups);
    a.ws = dbias ? static_cast<float *>(workspace) : nullptr;
    a.bf16 = dg_dtype == FP8DL_BF16;
    a.h_e4 = h_fp8 == FP8DL_E4M3;
    a.tiles = (uint32_t)(a.col_ld / 128);
    a.across = (uint32_t)((cols + 127) / 128);
    const bool tiles = dh_qt || g_qt || dbias, split = gated && cols % 128 != 0;
    // codes along the rows: by the tiles, but for what does not line up with them or where there are none
    a.row_first = !tiles ? 0 : split ? (uint32_t)(cols / 128) : a.across;
    a.row_jobs = tiles && !split ? 0 : (uint32_t)((wide + 127) / 128) - a.row_first;
    FP8DL_TRY(check_tiles((rows + ba::ACT_ROWS - 1) / ba::ACT_ROWS * a.row_jobs, rows, wide));
    FP8DL_TRY(check_tiles(a.col_ld / 128 * a.across, rows, wide));
    int sms = 0;
    FP8DL_TRY(current_device(nullptr, &sms));
    cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)wide * sizeof(float), st) != cudaSuccess)
            return check_launch("fp8_block_dact(empty)");
        return FP8DL_OK;
    }
    const bool pdl = short_call_bytes((double)rows * ((double)cols * (dg_dtype == FP8DL_BF16 ? 3.0 : 5.0) + 3.0 * wide));
    auto *launch = &launch_dact<FP8DL_E4M3, false, false>;
#define FP8DL_DACT(F)                                                                          \
    launch = gated ? (act_silu(act) ? launch_dact<F, true, true> : launch_dact<F, true, false>) \
                   : (act_silu(act) ? launch_dact<F, false, true> : launch_dact<F, false, false>)
    if (out_dtype == FP8DL_E4M3) FP8DL_DACT(FP8DL_E4M3);
    else FP8DL_DACT(FP8DL_E5M2);
#undef FP8DL_DACT
    FP8DL_TRY(launch(a, tiles, sms, st, pdl));
    if (dbias) {
        colsum_reduce(a.ws, (rows + 127) / 128, wide, dbias, st, pdl);
        return check_launch("fp8_block_dact(dbias reduce)");
    }
    return FP8DL_OK;
}

extern "C" fp8dl_status fp8_block_recode(const uint8_t *q, int32_t q_fp8, const float *s, int64_t src_rows, int64_t rows,
                                         int64_t cols, const int32_t *index, const int32_t *offsets, int32_t n_groups,
                                         int32_t out_dtype, uint8_t *col_q, float *col_s, fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_recode");
    FP8DL_CHECK_ARG(fp8_ok(q_fp8) && fp8_ok(out_dtype), "q_fp8 and out_dtype must be E4M3 or E5M2");
    if (!block_tokens_ok(rows) || !block_tokens_ok(src_rows) || !dim_ok(cols, 16))
        return fail(FP8DL_ERR_SHAPE, "rows (%lld) and src_rows (%lld) must be in [0, 2^31) and cols (%lld) a positive multiple of 16",
                    (long long)rows, (long long)src_rows, (long long)cols);
    if (!index && rows > src_rows)
        return fail(FP8DL_ERR_SHAPE, "rows (%lld) must not be more than src_rows (%lld) without an index", (long long)rows,
                    (long long)src_rows);
    FP8DL_TRY(check_block_groups(offsets, n_groups, true));
    FP8DL_CHECK_ARG(rows == 0 || ((src_rows == 0 || (q && s)) && col_q && col_s), "q, s, col_q and col_s must be non-NULL");
    if (!aligned16(q) || !aligned16(s) || !aligned16(col_q) || !aligned16(col_s) || !aligned4(index))
        return fail(FP8DL_ERR_ALIGN, "q, s, col_q and col_s must be 16-byte aligned, index 4-byte");
    BlockRecodeArgs a = {};
    a.q = q, a.s = s;
    a.src_rows = src_rows;
    a.rows = rows;
    a.cols = cols;
    a.index = index, a.offsets = offsets;
    a.n_groups = n_groups;
    a.col_q = col_q, a.col_s = col_s;
    a.col_ld = fp8_block_padded_rows(rows, n_groups);
    a.jobs = (uint32_t)((cols + 127) / 128);
    a.e4 = q_fp8 == FP8DL_E4M3;
    const int64_t ctas = a.col_ld / 128 * a.jobs;
    FP8DL_TRY(check_tiles(ctas, rows, cols));
    FP8DL_TRY(current_device(nullptr, nullptr));
    if (rows == 0) return FP8DL_OK;
    const bool pdl = short_call_bytes(2.0 * (double)rows * (double)cols);
    (void)launch_kernel(out_dtype == FP8DL_E4M3 ? block_recode_kernel<FP8DL_E4M3> : block_recode_kernel<FP8DL_E5M2>,
                        dim3((unsigned)ctas), dim3(bt::THREADS), 0, (cudaStream_t)stream, 0, pdl, a);
    note_launch();
    return check_launch("fp8_block_recode");
}
