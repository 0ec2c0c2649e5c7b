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
template <bool D>
__device__ __forceinline__ void activation2(float2 a, bool silu, float2 &y, float2 &d) {
    if (silu) {
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
    int silu, split;
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
template <int XKIND, int FMT, bool GATED>
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
            activation2<false>(va[i][q], a.silu, y[q], none);
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
    int64_t rows, cols, wide;
    const uint8_t *h_q;
    const float *h_s;
    const int32_t *offsets;
    int n_groups;
    uint8_t *dh_q, *dh_qt, *g_qt;
    float *dh_s, *dh_st, *g_st;
    int64_t col_ld;
    float *ws;       // column sums of dh per 128-row tile, or NULL
    uint32_t jobs;   // tiles across
    int silu, h_e4;  // SiLU, else GELU; the checkpoint's format (and g's): E4M3, else E5M2
};

// The rows of tile `tile` of the padded order; false where there are none.
__device__ __forceinline__ bool tile_place(const int32_t *offsets, int n_groups, int64_t rows, uint32_t tile, Where &w) {
    w.rr = threadIdx.x >> 4;
    w.cc = threadIdx.x & 15;
    w.r0 = (int64_t)tile * bt::TILE;
    w.nrows = (int)min((int64_t)bt::TILE, rows - w.r0);
    if (offsets) group_of_block(offsets, n_groups, rows, tile, w.r0, w.nrows);
    return w.nrows > 0;
}

// Eight values of the checkpoint from column c on (of the whole row), row r.
__device__ __forceinline__ void load_kept(const BlockDactArgs &a, int64_t r, int64_t c, bool ok, float2 (&v)[4]) {
    uint2 u = make_uint2(0u, 0u);
    float f = 0.0f;
    if (ok) {
        u = *reinterpret_cast<const uint2 *>(a.h_q + r * a.wide + c);
        f = a.h_s[(c >> 7) * a.rows + r];
    }
    v[0] = __fmul2_rn(decode2(u.x, a.h_e4), f2(f)), v[1] = __fmul2_rn(decode2(u.x >> 16, a.h_e4), f2(f));
    v[2] = __fmul2_rn(decode2(u.y, a.h_e4), f2(f)), v[3] = __fmul2_rn(decode2(u.y >> 16, a.h_e4), f2(f));
}

// One 128 x 128 tile of one matrix: of dh (its columns 0 .. wide), then of g (0 .. cols).  Right for every
// width: where u's half does not start on a block, a tile may hold columns of both halves (a
// thread's eight are always of one: cols is a multiple of 16).
template <int XKIND, int FMT, bool GATED>
__global__ void __launch_bounds__(bt::THREADS) block_dact_kernel(const BlockDactArgs a) {
    using namespace bt;
    __shared__ __align__(16) Matrix sm;
    pdl_wait();
    pdl_trigger();
    const uint32_t tile = blockIdx.x / a.jobs, job = blockIdx.x % a.jobs, dh_jobs = (uint32_t)((a.wide + 127) / 128);
    Where w;
    if (!tile_place(a.offsets, a.n_groups, a.rows, tile, w)) return;
    const bool is_g = job >= dh_jobs;
    const int64_t first = (int64_t)(is_g ? job - dh_jobs : job) * TILE, width = is_g ? a.cols : a.wide;
    w.c0 = first + 8 * w.cc;
    w.col_ok = w.c0 < width;
    const bool right = GATED && !is_g && w.c0 >= a.cols;  // of du
    const int64_t c = right ? w.c0 - a.cols : w.c0;
    Values v;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t r = w.r0 + 4 * w.rr + i;
        const bool ok = w.col_ok && 4 * w.rr + i < w.nrows;
        float2 va[4], vu[4], vd[4];
        load_kept(a, r, c, ok, va);
        if (GATED && !right) load_kept(a, r, c + a.cols, ok, vu);
        if (!is_g) load8<XKIND>(a.dg, r * a.cols + c, ok, vd);
#pragma unroll
        for (int p = 0; p < 4; p++) {
            float2 y, d;
            activation2<true>(va[p], a.silu, y, d);
            if (is_g)
                v[i][p] = GATED ? __fmul2_rn(y, vu[p]) : y;
            else if (right)
                v[i][p] = __fmul2_rn(vd[p], y);
            else
                v[i][p] = __fmul2_rn(GATED ? __fmul2_rn(vd[p], vu[p]) : vd[p], d);
        }
    }
    if (!is_g && a.dh_q) tile_rows<FMT>(v, w, a.dh_q, a.dh_s, a.wide, a.rows);
    uint8_t *qt = is_g ? a.g_qt : a.dh_qt;
    float *st = is_g ? a.g_st : a.dh_st;
    const bool sums = !is_g && a.ws;
    if (!qt && !sums) return;
    tile_maxima(v, w, sm);
    if (sums) tile_sums(v, w, sm);
    __syncthreads();
    if (threadIdx.x < TILE && first + threadIdx.x < width) {
        float *to = qt ? st + (int64_t)tile * width + first + threadIdx.x : nullptr;
        float *sum = sums ? a.ws + (int64_t)tile * width + first + threadIdx.x : nullptr;
        if (is_g && !a.h_e4)
            tile_scale<FP8DL_E5M2>(sm, threadIdx.x, to, sum);
        else if (is_g)
            tile_scale<FP8DL_E4M3>(sm, threadIdx.x, to, sum);
        else
            tile_scale<FMT>(sm, threadIdx.x, to, sum);
    }
    if (!qt) return;
    __syncthreads();
    if (is_g && !a.h_e4)
        tile_stage<FP8DL_E5M2>(v, w, sm);
    else if (is_g)
        tile_stage<FP8DL_E4M3>(v, w, sm);
    else
        tile_stage<FMT>(v, w, sm);
    __syncthreads();
    tile_out(sm, qt + first * a.col_ld + (int64_t)tile * TILE, a.col_ld, (int)min((int64_t)TILE, width - first));
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
    a.silu = act_silu(act);
    a.split = gated && cols % 128 != 0;
    a.jobs = (uint32_t)((cols + 127) / 128 + (a.split && h_q ? (a.wide + 127) / 128 : 0));
    const int64_t ctas = (rows + ba::ACT_ROWS - 1) / ba::ACT_ROWS * a.jobs;
    FP8DL_TRY(check_tiles(ctas, rows, cols));
    FP8DL_TRY(current_device(nullptr, nullptr));
    if (rows == 0) return FP8DL_OK;
    const bool pdl = short_call_bytes((double)rows * a.wide * ((h_dtype == FP8DL_BF16 ? 2.0 : 4.0) + (h_q ? 1.0 : 0.0)) + (double)rows * cols);
    auto *kernel = &block_act_kernel<FP8DL_BF16, FP8DL_E4M3, false>;
#define FP8DL_ACT(X, F) kernel = gated ? block_act_kernel<X, F, true> : block_act_kernel<X, F, false>
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
    a.silu = act_silu(act);
    a.h_e4 = h_fp8 == FP8DL_E4M3;
    a.jobs = (uint32_t)((wide + 127) / 128 + (g_qt ? (cols + 127) / 128 : 0));
    const int64_t ctas = a.col_ld / 128 * a.jobs;
    FP8DL_TRY(check_tiles(ctas, rows, wide));
    FP8DL_TRY(current_device(nullptr, nullptr));
    cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)wide * sizeof(float), st) != cudaSuccess)
            return check_launch("fp8_block_dact(empty)");
        return FP8DL_OK;
    }
    const bool pdl = short_call_bytes((double)rows * ((double)cols * (dg_dtype == FP8DL_BF16 ? 3.0 : 5.0) + 3.0 * wide));
    auto *kernel = &block_dact_kernel<FP8DL_BF16, FP8DL_E4M3, false>;
#define FP8DL_DACT(X, F) kernel = gated ? block_dact_kernel<X, F, true> : block_dact_kernel<X, F, false>
    if (dg_dtype == FP8DL_BF16 && out_dtype == FP8DL_E4M3) FP8DL_DACT(FP8DL_BF16, FP8DL_E4M3);
    else if (dg_dtype == FP8DL_BF16) FP8DL_DACT(FP8DL_BF16, FP8DL_E5M2);
    else if (out_dtype == FP8DL_E4M3) FP8DL_DACT(FP8DL_F32, FP8DL_E4M3);
    else FP8DL_DACT(FP8DL_F32, FP8DL_E5M2);
#undef FP8DL_DACT
    (void)launch_kernel(kernel, dim3((unsigned)ctas), dim3(bt::THREADS), 0, st, 0, pdl, a);
    note_launch();
    FP8DL_TRY(check_launch("fp8_block_dact"));
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
