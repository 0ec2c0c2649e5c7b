// exchange.cu — tokens to their experts' rows and back.
//
//   dispatch     row_q[position[t,j]] = codes of x[t] (1 x 128 blocks), quantised once for all its copies
//   combine      out[t] = sum_j weight[t,j] y[position[t,j]]
//   combine_bwd  dy[position[t,j]] = weight[t,j] dout[t],  dweight[t,j] = <dout[t], y[position[t,j]]>
//
// All three walk the tokens, so that a token's values are read once whatever k is, no row needs a
// search for its token, and nothing is added with atomics.  Bound: HBM.
#include "block.cuh"

namespace fp8dl {

// Eight consecutive values of a row: 16 (bf16) or 32 (fp32) bytes.
template <int XKIND>
struct Eight;
template <>
struct Eight<FP8DL_BF16> {
    uint4 u;
    __device__ __forceinline__ void load(const void *base, int64_t at) {
        u = ldg_stream(static_cast<const char *>(base) + at * 2);
    }
    __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float2 pair(int q) const {
        const uint32_t w = q == 0 ? u.x : q == 1 ? u.y : q == 2 ? u.z : u.w;
        return make_float2(bf16_lo(w), bf16_hi(w));
    }
    static __device__ __forceinline__ void store(void *base, int64_t at, const float2 (&v)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[q].x, v[q].y);
            w[q] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(static_cast<char *>(base) + at * 2) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Eight<FP8DL_F32> {
    uint4 u[2];
    __device__ __forceinline__ void load(const void *base, int64_t at) {
        const char *p = static_cast<const char *>(base) + at * 4;
        u[0] = ldg_stream(p);
        u[1] = ldg_stream(p + 16);
    }
    __device__ __forceinline__ void zero() { u[0] = u[1] = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ float2 pair(int q) const {
        const uint4 &w = u[q >> 1];
        return q & 1 ? make_float2(__uint_as_float(w.z), __uint_as_float(w.w))
                     : make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    }
    static __device__ __forceinline__ void store(void *base, int64_t at, const float2 (&v)[4]) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<char *>(base) + at * 4);
        p[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        p[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    }
};

struct DispatchArgs {
    const void *x;
    int64_t tokens, cols, rows, chunks;  // chunks of 1024 columns in a row
    const int32_t *position;
    int k;
    uint8_t *row_q, *q;
    float *row_s, *s;
};

// A warp quantises 1024 columns of a token: four loads under way at once, 16 lanes a block of 128.
// 16384 tokens x 4096 of 2 choices, bf16, with the copy in token order: 54 us, 6.3 TB/s.
template <int XKIND, int FMT>
__global__ void __launch_bounds__(256) block_dispatch_kernel(const DispatchArgs a) {
    constexpr int U = 4;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const uint32_t w = blockIdx.x * 8 + (threadIdx.x >> 5), chunks = (uint32_t)a.chunks, tok = w / chunks;
    const int64_t t = tok, c0 = (int64_t)(w - tok * chunks) * 1024 + 8 * lane;
    if (t >= a.tokens) return;
    const int32_t at = lane < a.k ? a.position[t * a.k + lane] : -1;  // lane j: where copy j goes
    Eight<XKIND> v[U];
#pragma unroll
    for (int i = 0; i < U; i++) {
        v[i].zero();
        if (c0 + 256 * i < a.cols) v[i].load(a.x, t * a.cols + c0 + 256 * i);
    }
    // maxima of the four blocks by a halving exchange: each lane ends up with that of block (lane >> 2 & 3) of its 16 lanes
    float m[U];
#pragma unroll
    for (int i = 0; i < U; i++) {
        const float2 x = v[i].pair(0), y = v[i].pair(1), z = v[i].pair(2), w4 = v[i].pair(3);
        m[i] = max3(max3(max3(x.x, x.y, y.x), y.y, z.x), max3(z.y, w4.x, w4.y), 0.0f);
    }
    if (max3(max3(m[0], m[1], m[2]), m[3], 0.0f) > 3.402823466e38f) {  // an infinity: over the finite values
#pragma unroll
        for (int i = 0; i < U; i++) {
            m[i] = 0.0f;
#pragma unroll
            for (int q = 0; q < 4; q++) m[i] = fmaxf(m[i], fmaxf(finite_abs(v[i].pair(q).x), finite_abs(v[i].pair(q).y)));
        }
    }
    const bool up8 = lane & 8, up4 = lane & 4;
#pragma unroll
    for (int i = 0; i < 2; i++)
        m[i] = fmaxf(up8 ? m[i + 2] : m[i], __shfl_xor_sync(0xffffffffu, up8 ? m[i] : m[i + 2], 8));
    m[0] = fmaxf(up4 ? m[1] : m[0], __shfl_xor_sync(0xffffffffu, up4 ? m[0] : m[1], 4));
    m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], 2));
    m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
    const float2 sc = block_scale_fast<FMT>(m[0]);
    uint2 code[U];
#pragma unroll
    for (int i = 0; i < U; i++) {
        const float k = __shfl_sync(0xffffffffu, sc.x, (lane & 16) + 4 * i);
        const float2 x = v[i].pair(0), y = v[i].pair(1), z = v[i].pair(2), w4 = v[i].pair(3);
        code[i] = make_uint2(codes4<FMT>(x.x * k, x.y * k, y.x * k, y.y * k), codes4<FMT>(z.x * k, z.y * k, w4.x * k, w4.y * k));
    }
    // the lane that writes a block's factor: the first of four, of the block that it holds
    const int64_t cs = c0 - 8 * (lane & 15) + 256 * (lane >> 2 & 3);
    const bool lead = (lane & 3) == 0 && cs < a.cols;
    for (int j = a.q ? -1 : 0; j < a.k; j++) {
        int64_t row = t;
        if (j >= 0) row = __shfl_sync(0xffffffffu, at, j);
        if (j >= 0 && (row < 0 || row >= a.rows)) continue;
        uint8_t *q = (j < 0 ? a.q : a.row_q) + row * a.cols + c0;
        float *s = (j < 0 ? a.s : a.row_s) + row;
#pragma unroll
        for (int i = 0; i < U; i++)
            if (c0 + 256 * i < a.cols) *reinterpret_cast<uint2 *>(q + 256 * i) = code[i];
        if (lead) s[(cs >> 7) * (j < 0 ? a.tokens : a.rows)] = sc.y;
    }
}

struct CombineArgs {
    const void *y, *dout;
    int64_t rows, cols, tokens;
    const int32_t *position;
    const float *weight;
    int k;
    void *out, *dy;
    float *dweight;
};

// A warp sums 512 columns of a token, the two loads of up to J rows of y under way at once (256 columns a warp: 512 tokens x
// 2048 of 6 choices 4.0 us against 3.0).  A lane holds a choice's row and weight; the others fetch them.
// WALK: resident CTAs go on to further tokens, whose rows and weights are looked up meanwhile.  It pays for two bf16 rows only
// (16384 tokens x 4096: 62.5 us against 68.5, 6.4 TB/s), where the least is under way; with four rows 60 against 50 (8192
// tokens, 6.7 TB/s), in fp32 153 against 122: the registers for it cost CTAs.
template <int XKIND, int J, bool WALK>
__global__ void __launch_bounds__(256) moe_combine_kernel(const CombineArgs a) {
    constexpr int CH = 2;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const uint32_t per = (uint32_t)((a.cols + 256 * CH - 1) / (256 * CH)), units = (uint32_t)a.tokens * per, step = gridDim.x * 8;
    uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (unit >= units) return;
    int32_t row_next = -1;
    float w_next = 0.0f;
    const auto look = [&](uint32_t u) {
        const int64_t t = u / per;
        if (u < units && lane < a.k) {
            row_next = a.position[t * a.k + lane];
            w_next = a.weight ? a.weight[t * a.k + lane] : 1.0f;
        }
    };
    look(unit);
    do {
        const uint32_t t = unit / per;
        const int64_t c = (int64_t)(unit - t * per) * (256 * CH) + 8 * lane;
        const int32_t row = row_next < a.rows ? row_next : -1;
        const float w = w_next;
        unit += step;
        if (WALK) look(unit);
        float2 sum[CH][4];
#pragma unroll
        for (int h = 0; h < CH; h++)
#pragma unroll
            for (int q = 0; q < 4; q++) sum[h][q] = f2(0.0f);
        for (int j0 = 0; j0 < a.k; j0 += J) {
            Eight<XKIND> v[J][CH];
#pragma unroll
            for (int j = 0; j < J; j++) {
                const int32_t r = __shfl_sync(0xffffffffu, row, (j0 + j) & 31);
#pragma unroll
                for (int h = 0; h < CH; h++) {
                    v[j][h].zero();
                    if (j0 + j < a.k && r >= 0 && c + 256 * h < a.cols) v[j][h].load(a.y, r * a.cols + c + 256 * h);
                }
            }
#pragma unroll
            for (int j = 0; j < J; j++) {
                const int32_t r = __shfl_sync(0xffffffffu, row, (j0 + j) & 31);
                const float k = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
                if (j0 + j >= a.k || r < 0) continue;
#pragma unroll
                for (int h = 0; h < CH; h++)
#pragma unroll
                    for (int q = 0; q < 4; q++) sum[h][q] = __ffma2_rn(v[j][h].pair(q), f2(k), sum[h][q]);
            }
        }
#pragma unroll
        for (int h = 0; h < CH; h++)
            if (c + 256 * h < a.cols) Eight<XKIND>::store(a.out, t * a.cols + c + 256 * h, sum[h]);
    } while (WALK && unit < units);
}

// W warps walk a token's row, 256 columns a step each, two steps' loads of up to four choices under way at once or one step's
// of eight (4096 tokens x 2048 of 6 choices: 40 us, in two passes of four 46); more choices: again, dout from L1.  The sums
// run over a lane's columns in order, then over the lanes in a fixed tree, then over the warps.
// 16384 tokens x 4096 of 2 choices, bf16: 103 us, 6.5 TB/s.
template <int XKIND, int J>
__global__ void __launch_bounds__(256) moe_combine_bwd_kernel(const CombineArgs a, int wlog) {
    __shared__ float part[8][J];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = 1 << wlog, mine = warp & (W - 1);
    const int64_t t = (int64_t)blockIdx.x * (8 >> wlog) + (warp >> wlog);
    const bool here = t < a.tokens;
    int32_t row = -1;
    float w = 0.0f;
    if (here && lane < a.k) {
        row = a.position[t * a.k + lane];
        if (row >= a.rows) row = -1;
        if (a.dy && row >= 0) w = a.weight[t * a.k + lane];
    }
    for (int j0 = 0; j0 < a.k; j0 += J) {
        int32_t r[J];
        float k[J], sum[J];
#pragma unroll
        for (int j = 0; j < J; j++) {
            r[j] = __shfl_sync(0xffffffffu, row, (j0 + j) & 31);
            if (j0 + j >= a.k) r[j] = -1;
            k[j] = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
            sum[j] = 0.0f;
        }
        if (here) {
            const auto add = [&](const Eight<XKIND> &d, const Eight<XKIND> (&v)[J], int64_t c) {
#pragma unroll
                for (int j = 0; j < J; j++) {
                    if (r[j] < 0) continue;
                    float2 s[4], p = f2(0.0f);
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        s[q] = __fmul2_rn(d.pair(q), f2(k[j]));
                        p = __ffma2_rn(d.pair(q), v[j].pair(q), p);
                    }
                    if (a.dy) Eight<XKIND>::store(a.dy, r[j] * a.cols + c, s);
                    sum[j] += p.x + p.y;
                }
            };
            const auto load = [&](Eight<XKIND> &d, Eight<XKIND> (&v)[J], int64_t c) {
                d.load(a.dout, t * a.cols + c);
#pragma unroll
                for (int j = 0; j < J; j++) {
                    v[j].zero();
                    if (a.dweight && r[j] >= 0) v[j].load(a.y, r[j] * a.cols + c);
                }
            };
            const int64_t step = 256 * W;
            if (J > 4) {
                for (int64_t c = 256 * mine + 8 * lane; c < a.cols; c += step) {
                    Eight<XKIND> d, v[J];
                    load(d, v, c);
                    add(d, v, c);
                }
            } else {
                for (int64_t c = 256 * mine + 8 * lane; c < a.cols; c += 2 * step) {
                    Eight<XKIND> d0, d1, v0[J], v1[J];
                    const bool two = c + step < a.cols;
                    load(d0, v0, c);
                    if (two) load(d1, v1, c + step);
                    add(d0, v0, c);
                    if (two) add(d1, v1, c + step);
                }
            }
        }
        if (!a.dweight) continue;
#pragma unroll
        for (int j = 0; j < J; j++) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
            if (lane == 0) part[warp][j] = sum[j];
        }
        if (W > 1) __syncthreads();
        else __syncwarp();
        if (here && mine == 0 && lane < J && j0 + lane < a.k) {
            float s = part[warp][lane];
            for (int o = 1; o < W; o++) s += part[warp + o][lane];
            a.dweight[t * a.k + j0 + lane] = s;  // zero where there is no row
        }
        if (W > 1) __syncthreads();
        else __syncwarp();
    }
}

static fp8dl_status check_exchange(int32_t dtype, int64_t tokens, int64_t rows, int64_t cols, const int32_t *position,
                                   int32_t k) {
    FP8DL_CHECK_ARG(dtype == FP8DL_F32 || dtype == FP8DL_BF16, "the type must be FP8DL_F32 or FP8DL_BF16");
    FP8DL_CHECK_ARG(k >= 1 && k <= 32, "k must be in [1, 32]");
    if (!block_tokens_ok(tokens) || !block_tokens_ok(rows) || !dim_ok(cols, 16))
        return fail(FP8DL_ERR_SHAPE, "tokens (%lld) and rows (%lld) must be in [0, 2^31) and cols (%lld) a positive multiple of 16",
                    (long long)tokens, (long long)rows, (long long)cols);
    FP8DL_CHECK_ARG(tokens == 0 || position, "position is NULL");
    if (!aligned4(position)) return fail(FP8DL_ERR_ALIGN, "position must be 4-byte aligned");
    return FP8DL_OK;
}

static fp8dl_status exchange_grid(int64_t ctas) {
    if (ctas > 0x7fffffffll) return fail(FP8DL_ERR_SHAPE, "%lld blocks of threads are more than 2^31 - 1", (long long)ctas);
    return FP8DL_OK;
}

}  // namespace fp8dl

using namespace fp8dl;

extern "C" fp8dl_status fp8_block_dispatch(const void *x, int32_t x_dtype, int64_t tokens, int64_t cols, int32_t out_dtype,
                                           const int32_t *position, int32_t k, int64_t rows, uint8_t *row_q,
                                           float *row_s, uint8_t *q, float *s, fp8dl_stream_t stream) {
    FP8DL_NVTX("fp8_block_dispatch");
    FP8DL_TRY(check_exchange(x_dtype, tokens, rows, cols, position, k));
    FP8DL_CHECK_ARG(out_dtype == FP8DL_E4M3 || out_dtype == FP8DL_E5M2, "out_dtype must be E4M3 or E5M2");
    FP8DL_CHECK_ARG(tokens == 0 || x, "x is NULL");
    FP8DL_CHECK_ARG(tokens == 0 || rows == 0 || (row_q && row_s), "row_q and row_s must be non-NULL");
    FP8DL_CHECK_ARG(!q == !s, "q and s come together");
    if (!aligned16(x) || !aligned16(row_q) || !aligned16(row_s) || !aligned16(q) || !aligned16(s))
        return fail(FP8DL_ERR_ALIGN, "x, row_q, row_s, q and s must be 16-byte aligned");
    FP8DL_TRY(current_device(nullptr, nullptr));
    if (tokens == 0) return FP8DL_OK;
    DispatchArgs a = {x, tokens, cols, rows, (cols + 1023) / 1024, position, k, row_q, q, row_s, s};
    const int64_t ctas = (tokens * a.chunks + 7) / 8;
    FP8DL_TRY(exchange_grid(8 * ctas));
    const bool pdl = short_call_bytes((double)tokens * (double)cols * ((x_dtype == FP8DL_BF16 ? 2.0 : 4.0) + k));
    auto *kernel = x_dtype == FP8DL_BF16
                       ? (out_dtype == FP8DL_E4M3 ? block_dispatch_kernel<FP8DL_BF16, FP8DL_E4M3>
                                                  : block_dispatch_kernel<FP8DL_BF16, FP8DL_E5M2>)
                       : (out_dtype == FP8DL_E4M3 ? block_dispatch_kernel<FP8DL_F32, FP8DL_E4M3>
                                                  : block_dispatch_kernel<FP8DL_F32, FP8DL_E5M2>);
    (void)launch_kernel(kernel, dim3((unsigned)ctas), dim3(256), 0, (cudaStream_t)stream, 0, pdl, a);
    note_launch();
    return check_launch("fp8_block_dispatch");
}

extern "C" fp8dl_status moe_combine(const void *y, int32_t dtype, int64_t rows, int64_t cols, const int32_t *position,
                                    const float *weight, int64_t tokens, int32_t k, void *out, fp8dl_stream_t stream) {
    FP8DL_NVTX("moe_combine");
    FP8DL_TRY(check_exchange(dtype, tokens, rows, cols, position, k));
    FP8DL_CHECK_ARG(tokens == 0 || (out && (y || rows == 0)), "y and out must be non-NULL");
    if (!aligned16(y) || !aligned16(out) || !aligned4(weight))
        return fail(FP8DL_ERR_ALIGN, "y and out must be 16-byte aligned, weight 4-byte");
    int sms = 0;
    FP8DL_TRY(current_device(nullptr, &sms));
    if (tokens == 0) return FP8DL_OK;
    CombineArgs a = {y, nullptr, rows, cols, tokens, position, weight, k, out, nullptr, nullptr};
    const int64_t per = (cols + 511) / 512, ctas = (tokens * per + 7) / 8;
    FP8DL_TRY(exchange_grid(8 * ctas));
    const bool pdl = short_call_bytes((double)tokens * (double)cols * (dtype == FP8DL_BF16 ? 2.0 : 4.0) * (k + 1));
    const int64_t resident = 4 * (int64_t)sms;
    const bool walk = dtype == FP8DL_BF16 && k <= 2 && ctas > resident;
    auto *kernel = walk                  ? moe_combine_kernel<FP8DL_BF16, 2, true>
                   : dtype == FP8DL_BF16 ? (k <= 2 ? moe_combine_kernel<FP8DL_BF16, 2, false> : moe_combine_kernel<FP8DL_BF16, 4, false>)
                                         : (k <= 2 ? moe_combine_kernel<FP8DL_F32, 2, false> : moe_combine_kernel<FP8DL_F32, 4, false>);
    (void)launch_kernel(kernel, dim3((unsigned)(walk ? resident : ctas)), dim3(256), 0, (cudaStream_t)stream, 0, pdl, a);
    note_launch();
    return check_launch("moe_combine");
}

extern "C" fp8dl_status moe_combine_bwd(const void *dout, const void *y, int32_t dtype, int64_t rows, int64_t cols,
                                        const int32_t *position, const float *weight, int64_t tokens, int32_t k,
                                        void *dy, float *dweight, fp8dl_stream_t stream) {
    FP8DL_NVTX("moe_combine_bwd");
    FP8DL_TRY(check_exchange(dtype, tokens, rows, cols, position, k));
    FP8DL_CHECK_ARG(tokens == 0 || dout, "dout is NULL");
    FP8DL_CHECK_ARG(tokens == 0 || rows == 0 || dy || dweight, "dy and dweight are both NULL");
    FP8DL_CHECK_ARG(tokens == 0 || rows == 0 || ((!dy || weight) && (!dweight || y)), "dy needs weight, dweight needs y");
    if (!aligned16(dout) || !aligned16(y) || !aligned16(dy) || !aligned4(weight) || !aligned4(dweight))
        return fail(FP8DL_ERR_ALIGN, "dout, y and dy must be 16-byte aligned, weight and dweight 4-byte");
    int sms = 0;
    FP8DL_TRY(current_device(nullptr, &sms));
    if (tokens == 0) return FP8DL_OK;
    CombineArgs a = {y, dout, rows, cols, tokens, position, weight, k, nullptr, dy, dweight};
    // warps a token: more where tokens are few (x 4096 of 2 choices: 64 tokens 5.8 us with one warp, 2.2 with eight; 1024
    // tokens 6.6 and 5.9, 5.2 with four; 4096 tokens 23.0 with one, 25.4 with eight; x 2048 of 6 choices, fewer of whose
    // warps fit an SM: 512 tokens 7.6, 4.4 with four, 5.4 with eight; 2048 tokens 15.5 with one, 16.9 with two)
    int wlog = 0;
    while (wlog < 3 && (tokens << wlog) < (k <= 4 ? 16 : 8) * (int64_t)sms && (int64_t(256) << wlog) < cols) wlog++;
    const int64_t ctas = ((tokens << wlog) + 7) / 8;
    const bool pdl = short_call_bytes((double)tokens * (double)cols * (dtype == FP8DL_BF16 ? 2.0 : 4.0) * (2 * k + 1));
    auto *kernel = dtype == FP8DL_BF16
                       ? (k <= 2 ? moe_combine_bwd_kernel<FP8DL_BF16, 2> : k <= 4 ? moe_combine_bwd_kernel<FP8DL_BF16, 4> : moe_combine_bwd_kernel<FP8DL_BF16, 8>)
                       : (k <= 2 ? moe_combine_bwd_kernel<FP8DL_F32, 2> : k <= 4 ? moe_combine_bwd_kernel<FP8DL_F32, 4> : moe_combine_bwd_kernel<FP8DL_F32, 8>);
    (void)launch_kernel(kernel, dim3((unsigned)ctas), dim3(256), 0, (cudaStream_t)stream, 0, pdl, a, wlog);
    note_launch();
    return check_launch("moe_combine_bwd");
}
