// blockquant.cu — block-scaled FP8 quantisation: one fp32 scale per 128 values
// (activations and gradients) or per 128 x 128 block (weights).
//
// The scale is the per-tensor scale FP8_MAX / amax of "FP8 低精度训练：Transformer
// Engine 简析" §三.1, taken over a block instead of a tensor and from the block's
// own values instead of a history, so it needs no state.
#include <cuda_bf16.h>

#include "block.cuh"

namespace fp8dl {

namespace bq {
constexpr int THREADS = 256, TILE = 128;
enum { TOKENS, GROUPS, WEIGHT };
}

struct BlockQuantArgs {
    const void *x;
    int64_t rows, cols;      // of one matrix
    int64_t tiles_c;         // 128-column tiles
    int64_t row_blocks;      // 128-row tiles of one matrix (of all groups together: the padded capacity / 128)
    const int32_t *offsets;  // ragged groups, or NULL
    int n_groups;
    uint8_t *row_q, *col_q;  // row-major and transposed codes, either may be NULL
    float *row_s, *col_s;
    int64_t col_ld;          // columns of the transposed codes
    float *ws;               // column sums per 128-row tile, or NULL
};

// (scale, stored factor) of a block whose largest finite magnitude is amax: both are
// correctly rounded divisions.  A maximum below 2^-100 counts as 2^-100, so that the scale
// stays finite; an all-zero block has scale 1.
template <int FMT>
__device__ __forceinline__ float2 block_scale(float amax) {
    constexpr float FMAX = FMT == FP8DL_E4M3 ? 448.0f : 57344.0f;
    const float sc = amax > 0.0f ? __fdiv_rn(FMAX, fmaxf(amax, 7.888609052210118e-31f)) : 1.0f;
    return make_float2(sc, __frcp_rn(sc));
}

// |v|, or 0 if v is not finite (blocks that hold infinities or NaN only).
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a <= 3.402823466e38f ? a : 0.0f;
}

// A thread's 8 x 8 values as they were loaded: bf16 stays packed (32 registers instead of 64, so
// three CTAs fit an SM and their loads overlap), and its maxima are taken on the packed words.
template <int XKIND>
struct Values;
template <>
struct Values<FP8DL_BF16> {
    uint32_t w[8][4];
    __device__ __forceinline__ void load(int i, const char *p, bool ok) {
        const uint4 u = ok ? ldg_stream(p) : make_uint4(0u, 0u, 0u, 0u);
        w[i][0] = u.x, w[i][1] = u.y, w[i][2] = u.z, w[i][3] = u.w;
    }
    __device__ __forceinline__ float2 pair(int i, int q) const { return make_float2(bf16_lo(w[i][q]), bf16_hi(w[i][q])); }
    __device__ __forceinline__ void maxima(float (&rmax)[8], float (&cmax)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const uint32_t m = bf16x2_absmax(bf16x2_absmax(w[i][0], w[i][1]), bf16x2_absmax(w[i][2], w[i][3]));
            rmax[i] = fmaxf(fabsf(bf16_lo(m)), fabsf(bf16_hi(m)));
        }
#pragma unroll
        for (int q = 0; q < 4; q++) {
            uint32_t m = w[0][q];
#pragma unroll
            for (int i = 1; i < 8; i++) m = bf16x2_absmax(m, w[i][q]);
            cmax[2 * q] = fabsf(bf16_lo(m)), cmax[2 * q + 1] = fabsf(bf16_hi(m));
        }
    }
};
template <>
struct Values<FP8DL_F32> {
    float2 v[8][4];
    __device__ __forceinline__ void load(int i, const char *p, bool ok) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint4 u = ok ? ldg_stream(p + 16 * h) : make_uint4(0u, 0u, 0u, 0u);
            v[i][2 * h] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
            v[i][2 * h + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
        }
    }
    __device__ __forceinline__ float2 pair(int i, int q) const { return v[i][q]; }
    __device__ __forceinline__ void maxima(float (&rmax)[8], float (&cmax)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; i++) rmax[i] = cmax[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float a = fabsf(v[i][q].x), b = fabsf(v[i][q].y);  // fmaxf ignores NaN
                rmax[i] = fmaxf(rmax[i], fmaxf(a, b));
                cmax[2 * q] = fmaxf(cmax[2 * q], a);
                cmax[2 * q + 1] = fmaxf(cmax[2 * q + 1], b);
            }
    }
};

// One CTA converts one 128 x 128 tile: x is read once, both copies of the codes are written.
//   Threads  16 x 16, thread (rr, cc) holds rows 8rr .. 8rr+7 and columns 8cc .. 8cc+7: its
//            eight loads are 16 (bf16) or 32 (fp32) bytes and a warp covers whole 128-byte
//            lines; all eight are in flight at once.
//   Maxima   ignoring NaN; where an infinity shows up the thread takes them again over its
//            finite values.
//   Row      maxima over the 16 lanes of a half-warp by a halving exchange (8 shuffles for
//   blocks   8 rows instead of 32), after which each lane owns one row's maximum, takes its
//            scale once and the others fetch it by shuffle.
//   Column   maxima over 8 rows in the thread, two row groups by shuffle, eight warps through
//   blocks   shared memory.
//   Codes    row-wise leave as 8-byte pieces (16 lanes: one 128-byte line).  Transposed codes
//            are packed straight along the rows (the conversion takes two values from any two
//            registers, so no byte transpose is needed), staged in shared memory with the
//            8-byte chunks XOR-swizzled by column group (conflict-free both ways), and leave
//            as whole 128-byte lines.
// WEIGHT: one scale for the tile instead, for both copies.  (fp32 at three CTAs an SM spills 20 bytes.)
// GROUPS: a tile is a group's; where groups are short, most warps of a CTA would have no rows.  A tile of
// up to 16, 32 or 64 rows takes 1, 2 or 4 warps and the CTA the next 8, 4 or 2 column tiles; their
// own CTAs write the padding behind the rows' 32-byte sectors (500 rows of 200 groups, 4096 columns fp32:
// 72 us with a CTA for every tile, 43 so; 4096 rows 80 and 53; 24 groups of 2999 rows no change).
// Bound: HBM (read esz, write 2 bytes per value).  8192 x 4096 bf16, both copies: 25.1 us, 5.4 TB/s;
// weights 16384 x 4096 bf16: 44.0 us, 6.1 TB/s; 32 of 1008 x 2048 fp32: 63.9 us, 6.2 TB/s.
template <int XKIND, int FMT, int KIND>
__global__ void __launch_bounds__(bq::THREADS, XKIND == FP8DL_BF16 || KIND == bq::WEIGHT ? 3 : 2)
    block_quantize_kernel(const BlockQuantArgs args) {
    using namespace bq;
    pdl_wait();
    pdl_trigger();
    constexpr int ESZ = XKIND == FP8DL_BF16 ? 2 : 4;
    constexpr int MOST = KIND == GROUPS ? 8 : 1;    // column tiles of a CTA
    __shared__ __align__(16) uint8_t tcode[TILE * TILE];
    __shared__ __align__(16) float part[8][TILE];   // column maxima (or sums) per warp
    __shared__ __align__(16) float cscale[MOST * TILE];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cc = tid & 15;
    const uint32_t tiles_c = (uint32_t)args.tiles_c;
    const uint32_t tile_r = blockIdx.x / tiles_c, tile_c0 = blockIdx.x % tiles_c;
    const int64_t mat = blockIdx.y;
    int64_t r0 = (int64_t)tile_r * TILE;
    int nrows = (int)min((int64_t)TILE, args.rows - r0);
    int wlog = 3;  // log2 of the warps of a tile
    if (KIND == GROUPS) {
        if (args.col_q) {
            group_of_block(args.offsets, args.n_groups, args.rows, tile_r, r0, nrows);
        } else {  // rows alone: the groups' borders do not matter, where the first begins and the last ends does
            int64_t first, end;
            group_rows(args.offsets, 0, args.rows, first, end);
            end = min(max((int64_t)args.offsets[args.n_groups], first), args.rows);
            r0 += first;
            nrows = (int)min((int64_t)TILE, end - r0);
        }
        if (nrows <= 0) return;  // behind the last group
        wlog = nrows <= 16 ? 0 : nrows <= 32 ? 1 : nrows <= 64 ? 2 : 3;
        if (tile_c0 & ((8u >> wlog) - 1)) {  // another CTA's, but for the padding behind its rows' sectors
            const int ch = tid & 7;
            if (args.col_q && ch >= 2 * ((nrows + 31) / 32)) {
                uint8_t *to = args.col_q + ((int64_t)tile_c0 * TILE + (tid >> 3)) * args.col_ld + (int64_t)tile_r * TILE + 16 * ch;
                for (int64_t c = (int64_t)tile_c0 * TILE + (tid >> 3), k = 0; k < 4 && c < args.cols; k++, c += 32, to += 32 * args.col_ld)
                    *reinterpret_cast<uint4 *>(to) = make_uint4(0u, 0u, 0u, 0u);
            }
            return;
        }
    }
    const int sub = KIND == GROUPS ? warp >> wlog : 0, lw = warp - (sub << wlog);  // the warp's tile, its place there
    const int rr = KIND == GROUPS ? 2 * lw + (lane >> 4) : tid >> 4;
    const int64_t tile_c = tile_c0 + sub;
    const bool live = KIND != GROUPS || (16 * lw < nrows && tile_c < args.tiles_c);
    const int64_t c0 = tile_c * TILE + 8 * cc;
    const bool col_ok = c0 < args.cols;  // columns come in sixteens
    const char *px = static_cast<const char *>(args.x) + ((mat * args.rows + r0 + 8 * rr) * args.cols + c0) * ESZ;
    Values<XKIND> v;
#pragma unroll
    for (int i = 0; i < 8; i++) v.load(i, px + i * args.cols * ESZ, col_ok && 8 * rr + i < nrows);
    float rmax[8], cmax[8];
    v.maxima(rmax, cmax);
    float top = rmax[0];
#pragma unroll
    for (int i = 1; i < 8; i++) top = fmaxf(top, rmax[i]);
    if (top > 3.402823466e38f) {  // an infinity: the maxima over the finite values
#pragma unroll
        for (int i = 0; i < 8; i++) rmax[i] = cmax[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const float2 p = v.pair(i, q);
                const float a = finite_abs(p.x), b = finite_abs(p.y);
                rmax[i] = fmaxf(rmax[i], fmaxf(a, b));
                cmax[2 * q] = fmaxf(cmax[2 * q], a);
                cmax[2 * q + 1] = fmaxf(cmax[2 * q + 1], b);
            }
        top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) top = fmaxf(top, rmax[i]);
    }
    float tile_scale = 0.0f;
    if (KIND == WEIGHT) {
        float m = warp_max(top);
        if (lane == 0) cscale[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; w++) m = fmaxf(m, cscale[w]);
        const float2 sc = block_scale<FMT>(m);
        if (tid == 0) {
            const int64_t e = mat * args.row_blocks * args.tiles_c;
            if (args.row_s) args.row_s[e + tile_c * args.row_blocks + tile_r] = sc.y;
            if (args.col_s) args.col_s[e + tile_r * args.tiles_c + tile_c] = sc.y;
        }
        tile_scale = sc.x;
    }
    if (KIND != WEIGHT && args.col_q) {  // column maxima of the warp; joined after the row-wise stores are on their way
#pragma unroll
        for (int j = 0; j < 8; j++) {
            cmax[j] = fmaxf(cmax[j], __shfl_xor_sync(0xffffffffu, cmax[j], 16));
            if (lane < 16) part[warp][8 * cc + j] = cmax[j];
        }
    }
    if (args.row_q && live) {
        float own = tile_scale;
        if (KIND != WEIGHT) {
            // halving exchange: after steps 8, 4, 2 lane cc holds row (cc >> 1) of its eight
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const bool up = cc & 8;
                const float send = up ? rmax[i] : rmax[i + 4], keep = up ? rmax[i + 4] : rmax[i];
                rmax[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 8));
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const bool up = cc & 4;
                const float send = up ? rmax[i] : rmax[i + 2], keep = up ? rmax[i + 2] : rmax[i];
                rmax[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 4));
            }
            {
                const bool up = cc & 2;
                const float send = up ? rmax[0] : rmax[1], keep = up ? rmax[1] : rmax[0];
                rmax[0] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 2));
            }
            const float2 sc = block_scale<FMT>(fmaxf(rmax[0], __shfl_xor_sync(0xffffffffu, rmax[0], 1)));
            const int row = 8 * rr + (cc >> 1);
            if (!(cc & 1) && row < nrows) args.row_s[tile_c * args.rows + r0 + row] = sc.y;
            own = sc.x;
        }
        uint8_t *qrow = args.row_q + (mat * args.rows + r0 + 8 * rr) * args.cols + c0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 s2 = f2(KIND == WEIGHT ? own : __shfl_sync(0xffffffffu, own, (lane & 16) + 2 * i));
            float2 y[4];
#pragma unroll
            for (int q = 0; q < 4; q++) y[q] = __fmul2_rn(v.pair(i, q), s2);
            if (col_ok && 8 * rr + i < nrows)
                *reinterpret_cast<uint2 *>(qrow + i * args.cols) = make_uint2(
                    pack4<FMT>(y[0].x, y[0].y, y[1].x, y[1].y), pack4<FMT>(y[2].x, y[2].y, y[3].x, y[3].y));
        }
    }
    if (KIND != WEIGHT && args.ws) {  // column sums of the tile, rows in a fixed order
        float *sums = reinterpret_cast<float *>(tcode);  // [8][TILE], before the codes take the place
#pragma unroll
        for (int q = 0; q < 4; q++) {
            float2 s = v.pair(0, q);
#pragma unroll
            for (int i = 1; i < 8; i++) s = __fadd2_rn(s, v.pair(i, q));
            s.x += __shfl_xor_sync(0xffffffffu, s.x, 16);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, 16);
            if (lane < 16) *reinterpret_cast<float2 *>(sums + warp * TILE + 8 * cc + 2 * q) = s;
        }
        __syncthreads();
        if (tid < TILE && tile_c * TILE + tid < args.cols) {
            float s = sums[tid];
#pragma unroll
            for (int w = 1; w < 8; w++) s += sums[w * TILE + tid];
            args.ws[tile_r * args.cols + tile_c * TILE + tid] = s;
        }
    }
    if (!args.col_q) return;
    const int width = TILE << (3 - wlog);  // the CTA's columns
    if (KIND != WEIGHT) {
        __syncthreads();
        for (int c = tid; c < width; c += THREADS) {
            const int w0 = (c >> 7) << wlog, w1 = w0 + (1 << wlog);
            float m = part[w0][c & 127];
            for (int w = w0 + 1; w < w1; w++) m = fmaxf(m, part[w][c & 127]);
            const float2 sc = block_scale<FMT>(m);
            cscale[c] = sc.x;
            const int64_t col = (int64_t)tile_c0 * TILE + c;
            if (col < args.cols) args.col_s[tile_r * args.cols + col] = sc.y;
        }
        __syncthreads();
    }
    if (live) {
        const float *cs = cscale + sub * TILE + 8 * cc;
#pragma unroll
        for (int q = 0; q < 4; q++) {  // columns 8cc + 2q and the next
            const float2 s2 = KIND == WEIGHT ? f2(tile_scale) : *reinterpret_cast<const float2 *>(cs + 2 * q);
            float2 y[8];
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] = __fmul2_rn(v.pair(i, q), s2);
            uint8_t *at = tcode + (8 * cc + 2 * q) * TILE + (((tid >> 4) ^ cc) << 3);
            *reinterpret_cast<uint2 *>(at) =
                make_uint2(pack4<FMT>(y[0].x, y[1].x, y[2].x, y[3].x), pack4<FMT>(y[4].x, y[5].x, y[6].x, y[7].x));
            *reinterpret_cast<uint2 *>(at + TILE) =
                make_uint2(pack4<FMT>(y[0].y, y[1].y, y[2].y, y[3].y), pack4<FMT>(y[4].y, y[5].y, y[6].y, y[7].y));
        }
    }
    __syncthreads();
    // weights: r0 .. r0+127 of q_t's rows (sixteens); tokens: the tile's 128 padded columns, of
    // which sixteen are one warp's rows
    const int64_t out0 = (int64_t)tile_r * TILE;
    const int ch = tid & 7, first = tid >> 3, left = (int)min((int64_t)width, args.cols - (int64_t)tile_c0 * TILE);
    const bool has = KIND != GROUPS || 16 * ch < nrows;  // chunk ch holds warp ch's rows; the rest is zeros
    if (KIND == WEIGHT && out0 + 16 * ch >= args.col_ld) return;
    uint8_t *to = args.col_q + (mat * args.cols + (int64_t)tile_c0 * TILE + first) * args.col_ld + out0 + 16 * ch;
    for (int c0 = first; c0 < width; c0 += 128) {
        uint4 u[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int c = first + 32 * k, g = c >> 3, w = KIND == GROUPS ? ((c0 >> 7) << wlog) + ch : ch;
            u[k] = make_uint4(0u, 0u, 0u, 0u);
            if (has) u[k] = *reinterpret_cast<const uint4 *>(tcode + c * TILE + ((w ^ (g >> 1)) << 4));
            if (g & 1) u[k] = make_uint4(u[k].z, u[k].w, u[k].x, u[k].y);
        }
#pragma unroll
        for (int k = 0; k < 4; k++, to += 32 * args.col_ld)
            if (c0 + 32 * k < left && (KIND != GROUPS || c0 < TILE || ch < 2 * ((nrows + 31) / 32))) *reinterpret_cast<uint4 *>(to) = u[k];
    }
}

template <int KIND>
static void launch_block_quantize(int32_t x_dtype, int32_t out_dtype, dim3 grid, cudaStream_t st, bool pdl,
                                  const BlockQuantArgs &a) {
    const bool e4 = out_dtype == FP8DL_E4M3;
    if (x_dtype == FP8DL_BF16 && e4)
        (void)launch_kernel(block_quantize_kernel<FP8DL_BF16, FP8DL_E4M3, KIND>, grid, bq::THREADS, 0, st, 0, pdl, a);
    else if (x_dtype == FP8DL_BF16)
        (void)launch_kernel(block_quantize_kernel<FP8DL_BF16, FP8DL_E5M2, KIND>, grid, bq::THREADS, 0, st, 0, pdl, a);
    else if (e4)
        (void)launch_kernel(block_quantize_kernel<FP8DL_F32, FP8DL_E4M3, KIND>, grid, bq::THREADS, 0, st, 0, pdl, a);
    else
        (void)launch_kernel(block_quantize_kernel<FP8DL_F32, FP8DL_E5M2, KIND>, grid, bq::THREADS, 0, st, 0, pdl, a);
    note_launch();
}

}  // namespace fp8dl

using namespace fp8dl;

extern "C" int64_t fp8_block_padded_rows(int64_t rows, int32_t n_groups) {
    if (rows <= 0) return 0;
    const int64_t g = n_groups < 1 ? 1 : n_groups;
    return (rows + 127 * (g < rows ? g : rows)) / 128 * 128;
}

extern "C" fp8dl_status fp8_block_quantize(const void *x, int32_t x_dtype, int64_t rows, int64_t cols,
                                           const int32_t *offsets, int32_t n_groups, int32_t out_dtype,
                                           uint8_t *row_q, float *row_s, uint8_t *col_q, float *col_s, float *dbias,
                                           void *workspace, size_t workspace_bytes, fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_quantize");
    FP8DL_CHECK_ARG(x_dtype == FP8DL_F32 || x_dtype == FP8DL_BF16, "x_dtype must be FP8DL_F32 or FP8DL_BF16");
    FP8DL_CHECK_ARG(out_dtype == FP8DL_E4M3 || out_dtype == FP8DL_E5M2, "out_dtype must be E4M3 or E5M2");
    if (!block_tokens_ok(rows) || !dim_ok(cols, 16))
        return fail(FP8DL_ERR_SHAPE, "rows (%lld) must be in [0, 2^31) and cols (%lld) a positive multiple of 16",
                    (long long)rows, (long long)cols);
    FP8DL_TRY(check_block_groups(offsets, n_groups, true));
    FP8DL_CHECK_ARG(!offsets || !dbias, "dbias is the sum over all rows: not with offsets");
    FP8DL_CHECK_ARG(rows == 0 || x, "x is NULL");
    FP8DL_CHECK_ARG(rows == 0 || row_q || col_q, "row_q and col_q are both NULL");
    FP8DL_CHECK_ARG(rows == 0 || (!row_q == !row_s && !col_q == !col_s), "row_q/row_s and col_q/col_s come in pairs");
    if (!aligned16(x) || !aligned16(row_q) || !aligned16(row_s) || !aligned16(col_q) || !aligned16(col_s) || !aligned16(dbias))
        return fail(FP8DL_ERR_ALIGN, "x, row_q, row_s, col_q, col_s and dbias must be 16-byte aligned");
    if (dbias && rows > 0) {
        if (!workspace || workspace_bytes < fp8_cast_workspace_size(rows, cols))
            return fail(FP8DL_ERR_WORKSPACE, "dbias needs a workspace of %zu bytes (got %zu)",
                        fp8_cast_workspace_size(rows, cols), workspace ? workspace_bytes : (size_t)0);
        if (!aligned16(workspace)) return fail(FP8DL_ERR_ALIGN, "workspace must be 16-byte aligned");
    }
    FP8DL_TRY(current_device(nullptr, nullptr));
    cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)cols * sizeof(float), st) != cudaSuccess)
            return check_launch("fp8_block_quantize(empty)");
        return FP8DL_OK;
    }
    BlockQuantArgs a = {};
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.tiles_c = (cols + 127) / 128;
    a.row_blocks = fp8_block_padded_rows(rows, col_q ? n_groups : 0) / 128;
    a.offsets = offsets;
    a.n_groups = n_groups;
    a.row_q = row_q;
    a.row_s = row_s;
    a.col_q = col_q;
    a.col_s = col_s;
    a.col_ld = a.row_blocks * 128;
    a.ws = dbias ? static_cast<float *>(workspace) : nullptr;
    if (a.tiles_c * a.row_blocks > 0x7fffffffll)
        return fail(FP8DL_ERR_SHAPE, "%lld x %lld is more than 2^31 - 1 tiles", (long long)rows, (long long)cols);
    const bool pdl = short_call_bytes((double)rows * (double)cols * (x_dtype == FP8DL_BF16 ? 4.0 : 6.0));
    const dim3 grid((unsigned)(a.tiles_c * a.row_blocks));
    if (offsets)
        launch_block_quantize<bq::GROUPS>(x_dtype, out_dtype, grid, st, pdl, a);
    else
        launch_block_quantize<bq::TOKENS>(x_dtype, out_dtype, grid, st, pdl, a);
    FP8DL_TRY(check_launch("fp8_block_quantize"));
    if (dbias) {
        colsum_reduce(a.ws, (rows + 127) / 128, cols, dbias, st, pdl);
        return check_launch("fp8_block_quantize(dbias reduce)");
    }
    return FP8DL_OK;
}

extern "C" fp8dl_status fp8_block_quantize_weight(const void *w, int32_t w_dtype, int32_t n_mats, int64_t rows,
                                                  int64_t cols, int32_t out_dtype, uint8_t *q, float *s, uint8_t *q_t,
                                                  float *s_t, fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_quantize_weight");
    FP8DL_CHECK_ARG(w_dtype == FP8DL_F32 || w_dtype == FP8DL_BF16, "w_dtype must be FP8DL_F32 or FP8DL_BF16");
    FP8DL_CHECK_ARG(out_dtype == FP8DL_E4M3 || out_dtype == FP8DL_E5M2, "out_dtype must be E4M3 or E5M2");
    FP8DL_CHECK_ARG(n_mats >= 1 && n_mats <= 65535, "n_mats must be in [1, 65535]");
    FP8DL_CHECK_ARG(w && (q || q_t), "w and one of q and q_t must be non-NULL");
    FP8DL_CHECK_ARG(!q == !s && !q_t == !s_t, "q/s and q_t/s_t come in pairs");
    if (!dim_ok(rows, 16) || !dim_ok(cols, 16))
        return fail(FP8DL_ERR_SHAPE, "rows (%lld) and cols (%lld) must be positive multiples of 16", (long long)rows,
                    (long long)cols);
    if (!aligned16(w) || !aligned16(q) || !aligned16(s) || !aligned16(q_t) || !aligned16(s_t))
        return fail(FP8DL_ERR_ALIGN, "w, q, s, q_t and s_t must be 16-byte aligned");
    BlockQuantArgs a = {};
    a.x = w;
    a.rows = rows;
    a.cols = cols;
    a.tiles_c = (cols + 127) / 128;
    a.row_blocks = (rows + 127) / 128;
    a.row_q = q;
    a.row_s = s;
    a.col_q = q_t;
    a.col_s = s_t;
    a.col_ld = rows;
    if (a.tiles_c * a.row_blocks > 0x7fffffffll)
        return fail(FP8DL_ERR_SHAPE, "%lld x %lld is more than 2^31 - 1 tiles", (long long)rows, (long long)cols);
    FP8DL_TRY(current_device(nullptr, nullptr));
    const bool pdl = short_call_bytes((double)n_mats * (double)rows * (double)cols * (w_dtype == FP8DL_BF16 ? 4.0 : 6.0));
    launch_block_quantize<bq::WEIGHT>(w_dtype, out_dtype, dim3((unsigned)(a.tiles_c * a.row_blocks), (unsigned)n_mats),
                                (cudaStream_t)stream, pdl, a);
    return check_launch("fp8_block_quantize_weight");
}
