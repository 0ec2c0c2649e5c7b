// blockact.cu — activations between block-scaled products, with the argument kept in 8 bits for
// the backward pass, and transposed codes made from row-wise ones.
//
//   act      g = act(h) or act(a) * u, h = [a | u]: codes of g along the rows (the next product's
//            operand) and of h (the checkpoint), straight from fp32
//   dact     h from the checkpoint; dh = dg act'(h), or [dg u act'(a) | dg act(a)]: its codes along the rows
//            (dgrad's operand) and transposed (wgrad's); g again, transposed (the next product's wgrad operand)
//   recode   transposed codes of a matrix whose row-wise codes were kept
//
// GELU(a) = a Phi(a), GELU'(a) = Phi(a) + a phi(a);
// SiLU(a) = a s, SiLU'(a) = s (1 + a (1 - s)), s = 1 / (1 + exp(-a)).
#include <cuda_fp16.h>

#include "block.cuh"

namespace fp8dl {

// -R(x) of two values x >= 0, Phi(-x) = exp(-x^2 / 2) R(x): t S(1 - t), t = 1 / (1 + p x), S a polynomial of degree 8 that is
// 1/2 at x = 0, fitted here by weighted least squares until the relative error was even over x in [0, 14.6] (3.6e-8; 2.5e-7
// in fp32).  In 1 - t, which is p x t, what the rounding of 1 + p x does to S goes with x; a polynomial in t was 4.7e-7 off near
// 0, where activations are.  Relative, because a block may hold nothing but small results: a column of a group of one row.
__device__ __forceinline__ float2 normal_ratio2(float2 x) {
    const float2 d = __ffma2_rn(f2(0.35f), x, f2(1.0f)), t = make_float2(rcp_approx_ftz(d.x), rcp_approx_ftz(d.y));
    const float2 u = __fmul2_rn(__fmul2_rn(f2(0.35f), x), t);
    float2 poly = __ffma2_rn(u, f2(0.02892103901855419f), f2(-0.08838456601291317f));
    poly = __ffma2_rn(u, poly, f2(0.06279255146641106f));
    poly = __ffma2_rn(u, poly, f2(0.01707466298726712f));
    poly = __ffma2_rn(u, poly, f2(0.06372926568268843f));
    poly = __ffma2_rn(u, poly, f2(-0.102527480416411f));
    poly = __ffma2_rn(u, poly, f2(-0.2610602466252296f));
    poly = __ffma2_rn(u, poly, f2(0.639832909834862f));
    poly = __ffma2_rn(u, poly, f2(-0.5f));
    return __fmul2_rn(poly, t);
}

// |a|, at most 32, where exp(-a^2 / 2) has long been zero: finite, so that what it is multiplied by stays zero.  NaN stays NaN.
__device__ __forceinline__ float magnitude(float a) {
    float x;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(fabsf(a)), "f"(32.0f));
    return x;
}

// act(a) and, with D, its derivative.  Relative errors in units of 2^-24, at most: GELU 1.25 a^2 + 23 where a < 0 (the
// exponent's two roundings and its constant; 8 and 1 for the squared 2^x, 12 for the ratio, 2 products), SiLU 1.25 |a| + 9.
// Measured: GELU 7 within |a| <= 1, 43 at -7, 121 at -11.5, SiLU 6 within |a| <= 4, 61 at -70; fp32 codes of gradients differ
// from 64 bits as rarely as those of a plain fp32 form (2999 x 1408, E5M2: 27 and 32 of 8 x 4 M).  An exact exponent (its
// remainder applied to 2^x) would cost 22 us on 140 for GELU of 8192 x 16384, 16 on 263 for its gradient, 22 on 207 for SiLU's,
// for results that are rounded to 3 or 4 significant bits.
template <bool SILU, bool D>
__device__ __forceinline__ void activation2(float2 a, float2 &y, float2 &d) {
    if (SILU) {  // constants in scalar instructions, which hold them (a packed one wants them in registers)
        const float2 e = make_float2(ex2_approx_ftz(a.x * -1.4426950409f), ex2_approx_ftz(a.y * -1.4426950409f));
        const float2 s = make_float2(rcp_approx_ftz(e.x + 1.0f), rcp_approx_ftz(e.y + 1.0f));
        y = make_float2(a.x * s.x, a.y * s.y);
        // s + y (1 - s): 1 - s first, which is nothing where s is 1 (s + y - y s loses s beside y from 2^24 on)
        if (D) d = make_float2(fmaf(y.x, 1.0f - s.x, s.x), fmaf(y.y, 1.0f - s.y, s.y));
    } else {
        // with e = exp(-a^2 / 2), x = |a|: Phi(a) = e R, or 1 - e R; the derivative e (R - phi(0) x), or 1 less that.  e is the
        // square of its root, so that it reaches the subnormal numbers (2^x itself flushes them: a block of nothing but such
        // results had the factor of a block of zeros)
        const float2 x = make_float2(magnitude(a.x), magnitude(a.y)), q = __fmul2_rn(__fmul2_rn(a, a), f2(-0.3606737602f));
        const float2 root = make_float2(ex2_approx_ftz(q.x), ex2_approx_ftz(q.y)), r = normal_ratio2(x), e = __fmul2_rn(root, root);
        const float2 tail = __fmul2_rn(e, r), up = __fadd2_rn(f2(1.0f), tail);
        y = __fmul2_rn(a, make_float2(a.x >= 0.0f ? up.x : -tail.x, a.y >= 0.0f ? up.y : -tail.y));  // infinity stays infinity
        if (D) {
            const float2 w = __fmul2_rn(e, __ffma2_rn(x, f2(0.3989422804f), r)), v = __fadd2_rn(f2(1.0f), w);
            d = make_float2(a.x >= 0.0f ? v.x : -w.x, a.y >= 0.0f ? v.y : -w.y);
        }
    }
}

// cp.async of N bytes; none and zeros where !ok.
template <int N, bool PAST_L1 = false>
__device__ __forceinline__ void copy_async(void *smem, const void *global, bool ok) {
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    if (PAST_L1)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(global), "r"(ok ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(global), "n"(N), "r"(ok ? N : 0) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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
};

namespace ba {
constexpr int ACT_THREADS = 256, ACT_ROWS = 32;  // rows of a CTA: two for each 16 lanes
constexpr int ACT_CTAS = 3;                       // CTAs an SM holds
}

// Eight columns of a row in fp32; unit(i): their i-th 16 bytes as they lie in memory.
template <int XKIND, typename Unit>
__device__ __forceinline__ void widen8(const Unit &unit, float2 (&v)[4]) {
    if (XKIND == FP8DL_BF16) {
        const uint4 u = unit(0);
        v[0] = make_float2(bf16_lo(u.x), bf16_hi(u.x)), v[1] = make_float2(bf16_lo(u.y), bf16_hi(u.y));
        v[2] = make_float2(bf16_lo(u.z), bf16_hi(u.z)), v[3] = make_float2(bf16_lo(u.w), bf16_hi(u.w));
    } else {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint4 u = unit(h);
            v[2 * h] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
            v[2 * h + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
        }
    }
}
// The same from memory; zeros where there are none.
template <int XKIND>
__device__ __forceinline__ void load8(const void *base, int64_t at, bool ok, float2 (&v)[4]) {
    const char *p = static_cast<const char *>(base) + at * (XKIND == FP8DL_BF16 ? 2 : 4);
    widen8<XKIND>([&](int h) { return ok ? ldg_stream(p + 16 * h) : make_uint4(0u, 0u, 0u, 0u); }, v);
}

// The blocks along the rows that 16 lanes hold together, eight values each: NA matrices, two rows of each.  Their maxima
// are joined by a halving exchange (8 shuffles for six blocks instead of 24), after which each lane works out
// one block's scale and the others fetch it.  q: a matrix's code of the thread's first value in the first row; the second
// row lies `ld` further on.  Returns the factor of the lane's block, (lane & 15) / S of [row][matrix], S lanes each.
template <int FMT, int NA>
__device__ __forceinline__ float put_blocks(const float2 (&v)[2][NA][4], uint8_t *const (&q)[NA], const uint32_t (&ld)[NA], bool ok0, bool ok1) {
    constexpr int N = 2 * NA, P = N <= 2 ? 2 : N <= 4 ? 4 : 8, S = 16 / P;
    const int lane = threadIdx.x & 31;
    float m[P];
#pragma unroll
    for (int n = 0; n < P; n++) {
        m[n] = 0.0f;
        if (n >= N) continue;
        const float2(&w)[4] = v[n / NA][n % NA];
        m[n] = max3(max3(max3(w[0].x, w[0].y, w[1].x), w[1].y, w[2].x), max3(w[2].y, w[3].x, w[3].y), 0.0f);
    }
    float top = m[0];
#pragma unroll
    for (int n = 1; n < N; n++) top = fmaxf(top, m[n]);
    if (top > 3.402823466e38f) {  // an infinity: over the finite values
#pragma unroll
        for (int n = 0; n < N; n++) {
            m[n] = 0.0f;
#pragma unroll
            for (int p = 0; p < 4; p++)
                m[n] = fmaxf(m[n], fmaxf(finite_abs(v[n / NA][n % NA][p].x), finite_abs(v[n / NA][n % NA][p].y)));
        }
    }
    int o = 8;
#pragma unroll
    for (int h = P / 2; h > 0; h /= 2, o /= 2) {
#pragma unroll
        for (int k = 0; k < h; k++) {
            const bool up = lane & o;
            const float send = up ? m[k] : m[k + h], keep = up ? m[k + h] : m[k];
            m[k] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
#pragma unroll
    for (; o > 0; o /= 2) m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    const float2 sc = block_scale_fast<FMT>(m[0]);
#pragma unroll
    for (int n = 0; n < N; n++) {
        const float k = __shfl_sync(0xffffffffu, sc.x, (lane & 16) + n * S);
        const float2(&w)[4] = v[n / NA][n % NA];
        const uint2 u = make_uint2(codes4<FMT>(w[0].x * k, w[0].y * k, w[1].x * k, w[1].y * k),
                                   codes4<FMT>(w[2].x * k, w[2].y * k, w[3].x * k, w[3].y * k));
        if (q[n % NA] && (n < NA ? ok0 : ok1)) *reinterpret_cast<uint2 *>(q[n % NA] + (n < NA ? 0 : ld[n % NA])) = u;
    }
    return sc.y;
}

// Persistent CTAs, a job of 32 rows of one block column (of a's and of u's where g is gated) after the other, two
// neighbouring rows for 16 lanes.  Each thread copies its values of the next job into its own slots of shared memory
// while it works on this one's (no barrier, no registers).
// Where u's half does not start on a block (cols not a multiple of 128) h's blocks do not line up with
// g's: the codes of h are jobs of their own behind g's.  KEEP: with the codes of h.
// Bound: HBM, SwiGLU of 8192 x 11008 in bf16 with the checkpoint: 100 us, 6.4 TB/s, without it 69 us, 6.6 TB/s (a CTA a
// job, loads into registers: 118 and 79); GELU of 8192 x 16384 140 us, 3.8 TB/s: the issue slots.
// The 16 bytes of a thread go past L1 where they are whole sectors' worth; two halves of fp32 values go through it (past
// it every sector is fetched twice: 8192 x 8192 182 us against 112).
template <int XKIND, int FMT, bool GATED, bool SILU, bool KEEP>
__global__ void __launch_bounds__(ba::ACT_THREADS, ba::ACT_CTAS) block_act_kernel(const BlockActArgs a) {
    using namespace ba;
    constexpr int NA = KEEP ? (GATED ? 3 : 2) : 1, NH = GATED ? 2 : 1, UNITS = XKIND == FP8DL_BF16 ? 1 : 2, ESZ = XKIND == FP8DL_BF16 ? 2 : 4;
    __shared__ uint4 in[2 * NH * UNITS][ACT_THREADS];  // [row][a, u][unit]
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    const uint32_t g_jobs = (uint32_t)((a.cols + 127) / 128), cols = (uint32_t)a.cols, wide = (uint32_t)a.wide, rows = (uint32_t)a.rows;
    int64_t first = 0, end = a.rows;
    if (a.offsets) {  // blocks along the rows do not see the groups' borders
        group_rows(a.offsets, 0, a.rows, first, end);
        end = min(max((int64_t)a.offsets[a.n_groups], first), a.rows);
    }
    const uint32_t last = (uint32_t)end, tiles = (uint32_t)((end - first + ACT_ROWS - 1) / ACT_ROWS), jobs = a.jobs;
    const auto row_of = [&](uint32_t tile) { return (uint32_t)first + tile * ACT_ROWS + 2 * (tid >> 4); };  // below 2^31 + 32
    const auto col_of = [&](uint32_t job) { return (job < g_jobs ? job : job - g_jobs) * 128 + 8 * (tid & 15); };
    const auto fetch = [&](uint32_t tile, uint32_t job) {
        const uint32_t r = row_of(tile), c = col_of(job);
        const bool there = c < (job < g_jobs ? cols : wide);
        const char *p = static_cast<const char *>(a.h) + (wide_mul(r, wide) + c) * ESZ;
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int n = 0; n < NH; n++) {
                if (n && job >= g_jobs) continue;
                const bool ok = r + i < last && there;
#pragma unroll
                for (int u = 0; u < UNITS; u++)
                    copy_async<16, UNITS == 1>(&in[(i * NH + n) * UNITS + u][tid], ok ? p + ((i ? wide : 0) + (uint64_t)(n ? cols : 0)) * ESZ + 16 * u : a.h, ok);
            }
    };
    uint32_t tile = blockIdx.x / jobs, job = blockIdx.x - tile * jobs;
    const uint32_t tile_step = gridDim.x / jobs, job_step = gridDim.x - tile_step * jobs;
    if (tile < tiles) fetch(tile, job);
    while (tile < tiles) {
        const uint32_t r = row_of(tile), c = col_of(job);
        const bool row0 = r < last, row1 = r + 1 < last, alone = job >= g_jobs;
        copy_wait_all();
        float2 h[2][NH][4];
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int n = 0; n < NH; n++) widen8<XKIND>([&](int u) { return in[(i * NH + n) * UNITS + u][tid]; }, h[i][n]);
        tile += tile_step, job += job_step;
        if (job >= jobs) job -= jobs, tile++;
        if (tile < tiles) fetch(tile, job);
        if (alone) {  // h alone
            float2 v[2][1][4];
#pragma unroll
            for (int p = 0; p < 4; p++) v[0][0][p] = h[0][0][p], v[1][0][p] = h[1][0][p];
            const bool there = c < wide;
            uint8_t *const q[1] = {a.h_q + wide_mul(r, wide) + c};
            const uint32_t ld[1] = {wide};
            const float f = put_blocks<FMT, 1>(v, q, ld, row0 && there, row1 && there);
            if ((tid & 7) == 0 && (tid & 8 ? row1 : row0)) a.h_s[wide_mul(c >> 7, rows) + r + (tid >> 3 & 1)] = f;
            continue;
        }
        float2 v[2][NA][4];
        const bool there = c < cols, ok0 = row0 && there, ok1 = row1 && there;
        const uint64_t at = wide_mul(r, wide) + c;
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int p = 0; p < 4; p++) {
                float2 none;
                activation2<SILU, false>(h[i][0][p], v[i][0][p], none);
                if (GATED) v[i][0][p] = make_float2(v[i][0][p].x * h[i][NH - 1][p].x, v[i][0][p].y * h[i][NH - 1][p].y);
                if (NA > 1) v[i][NA > 1 ? 1 : 0][p] = h[i][0][p];
                if (NA > 2) v[i][NA > 2 ? 2 : 0][p] = h[i][NH - 1][p];
            }
        uint8_t *q[NA];
        uint32_t ld[NA];
        q[0] = a.g_q + wide_mul(r, cols) + c, ld[0] = cols;
        if (NA > 1) q[NA > 1 ? 1 : 0] = a.h_q + at, ld[NA > 1 ? 1 : 0] = wide;
        if (NA > 2) q[NA > 2 ? 2 : 0] = a.h_q + at + cols, ld[NA > 2 ? 2 : 0] = wide;
        uint8_t *const(&qc)[NA] = reinterpret_cast<uint8_t *const(&)[NA]>(q);
        // a block's factor is written even by a lane that has none of its columns (the last block may be short)
        const float f = put_blocks<FMT, NA>(v, qc, ld, ok0, ok1);
        constexpr int N = 2 * NA, P = N <= 2 ? 2 : N <= 4 ? 4 : 8, S = 16 / P;
        const int mine = (tid & 15) / S, i = mine >= NA, n = mine - i * NA;
        if ((tid & (S - 1)) == 0 && mine < N && (i ? row1 : row0)) {
            float *s = n == 0 ? a.g_s : a.h_s;
            s[wide_mul((c + (n == 2 ? cols : 0)) >> 7, rows) + r + i] = f;
        }
    }
}

// ---------------------------------------------------------------------------
// 128 x 128 tiles with blocks along the rows and along the columns (dact, recode).
// ---------------------------------------------------------------------------
// Eight codes -> fp16 pairs (FP8 is exact in fp16).  volatile: a branch, not both conversions and a select.
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
__device__ __forceinline__ float2 half_pair(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }

// A persistent CTA's walk over tiles, `across` of a tile row side by side, CTAs one tile apart.  One thread walks,
// two tiles ahead of the work, and leaves what it finds in shared memory, where every phase reads what it
// needs: the values fill the registers.
struct Step {
    int64_t r0;          // the tile's first row
    uint32_t tile, col;  // the tile row of the padded order, the tile in it
    int n;               // rows; 0 behind the last tile
};
struct Walk {
    Step step[3];
    uint32_t down;
    int group;
};
__device__ __forceinline__ void walk_place(Walk &w, const GroupTable &table, bool grouped, int64_t rows, uint32_t tile, uint32_t col,
                                           int at) {
    Step s = {0, tile, col, 0};
    if (tile < w.down) {
        if (grouped) {
            int g = w.group;
            find_group(table, tile, g, s.r0, s.n);
            w.group = g;
        } else {
            s.r0 = (int64_t)tile * 128;
            s.n = (int)min((int64_t)128, rows - s.r0);
        }
    }
    w.step[at] = s;
}
__device__ __forceinline__ void walk_on(Walk &w, const GroupTable &table, bool grouped, int64_t rows, uint32_t across, int from, int to) {
    const uint32_t t = gridDim.x / across;
    uint32_t tile = w.step[from].tile + t, col = w.step[from].col + gridDim.x - t * across;
    if (col >= across) col -= across, tile++;
    if (w.step[from].n) walk_place(w, table, grouped, rows, tile, col, to);
    else w.step[to].n = 0;
}
// The first two steps.  The caller's next barrier shows them.
__device__ __forceinline__ void walk_start(Walk &w, const GroupTable &table, bool grouped, int n_groups, int64_t rows, uint32_t tiles,
                                           uint32_t across) {
    w.down = grouped ? min(tiles, table.before[n_groups]) : tiles;
    w.group = 0;
    walk_place(w, table, grouped, rows, blockIdx.x / across, blockIdx.x % across, 0);
    walk_on(w, table, grouped, rows, across, 0, 1);
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

// dh (and g) of two elements: every caller rounds in this order, so that the same element has the same
// bits whichever kernel computes it.
template <bool GATED, bool SILU>
__device__ __forceinline__ void gradient2(uint32_t ha, float fa, uint32_t hu, float fu, float2 dg, float2 &da, float2 &du,
                                          float2 &g) {
    const float2 p = half_pair(ha), q = half_pair(hu);
    float2 y, d;
    activation2<SILU, true>(make_float2(__fmul_rn(p.x, fa), __fmul_rn(p.y, fa)), y, d);
    if (GATED) {
        const float2 u = make_float2(__fmul_rn(q.x, fu), __fmul_rn(q.y, fu));
        g = make_float2(__fmul_rn(y.x, u.x), __fmul_rn(y.y, u.y));
        da = make_float2(__fmul_rn(__fmul_rn(dg.x, u.x), d.x), __fmul_rn(__fmul_rn(dg.y, u.y), d.y));
        du = make_float2(__fmul_rn(dg.x, y.x), __fmul_rn(dg.y, y.y));
    } else {
        g = y;
        da = make_float2(__fmul_rn(dg.x, d.x), __fmul_rn(dg.y, d.y));
    }
}

// Codes of N (one or two) matrices along the rows: two rows of eight values a thread, 16 lanes a row.  q, s: the first
// matrix's code and factor of the thread's first row; the second's lie q1, s1 further on, and are left out unless
// `both`.  Each lane works out one scale: of row (lane >> 3 & 1), of matrix (lane >> 2 & 1) where there are two.
template <int FMT, int N>
__device__ __forceinline__ void put_rows(const float2 (&v)[N][2][4], uint8_t *q, uint32_t q1, uint32_t ld, float *s, uint64_t s1, int rows,
                                         bool cols, bool both) {
    const int lane = threadIdx.x & 31;
    float m[N][2];
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float2(&w)[4] = v[n][i];
            m[n][i] = max3(max3(max3(w[0].x, w[0].y, w[1].x), w[1].y, w[2].x), max3(w[2].y, w[3].x, w[3].y), 0.0f);
        }
    if (max3(max3(m[0][0], m[0][1], 0.0f), m[N - 1][0], m[N - 1][1]) > 3.402823466e38f) {  // an infinity: over the finite values
#pragma unroll
        for (int n = 0; n < N; n++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                m[n][i] = 0.0f;
#pragma unroll
                for (int p = 0; p < 4; p++) m[n][i] = fmaxf(m[n][i], fmaxf(finite_abs(v[n][i][p].x), finite_abs(v[n][i][p].y)));
            }
    }
    const bool up8 = lane & 8, up4 = lane & 4;
    float top[N];
#pragma unroll
    for (int n = 0; n < N; n++) top[n] = fmaxf(up8 ? m[n][1] : m[n][0], __shfl_xor_sync(0xffffffffu, up8 ? m[n][0] : m[n][1], 8));
    float mine = N == 2 && up4 ? top[N - 1] : top[0];
    mine = fmaxf(mine, __shfl_xor_sync(0xffffffffu, N == 2 && !up4 ? top[N - 1] : top[0], 4));
    mine = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, 2));
    mine = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, 1));
    const float2 sc = block_scale_fast<FMT>(mine);
    if ((lane & 3) == 0 && (lane >> 3 & 1) < rows && (up4 ? N == 2 && both : true)) s[(lane >> 3 & 1) + (up4 ? s1 : 0)] = sc.y;
#pragma unroll
    for (int n = 0; n < N; n++) {
        if (n && !both) continue;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float k = __shfl_sync(0xffffffffu, sc.x, (lane & 16) + 8 * i + 4 * n);
            const float2(&w)[4] = v[n][i];
            const uint2 u = make_uint2(codes4<FMT>(w[0].x * k, w[0].y * k, w[1].x * k, w[1].y * k),
                                       codes4<FMT>(w[2].x * k, w[2].y * k, w[3].x * k, w[3].y * k));
            if (cols && i < rows) *reinterpret_cast<uint2 *>(q + (n ? q1 : 0) + (i ? ld : 0)) = u;
        }
    }
}

// Codes of a column's sixteen values (row pairs), its factor, and its sum where one is wanted; a column's eight lanes
// are neighbours.
template <int FMT>
__device__ __forceinline__ uint4 put_column(const float2 (&v)[8], float &factor) {
    float t = max3(v[0].x, v[0].y, v[1].x);
    t = max3(t, v[1].y, v[2].x);
#pragma unroll
    for (int k = 2; k < 7; k++) t = max3(t, v[k].y, v[k + 1].x);
    t = max3(t, v[7].y, 0.0f);
    if (t > 3.402823466e38f) {  // an infinity: over the finite values
        t = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; k++) t = fmaxf(t, fmaxf(finite_abs(v[k].x), finite_abs(v[k].y)));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
    const float2 sc = block_scale_fast<FMT>(t);
    factor = sc.y;
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float2 a = __fmul2_rn(v[2 * k], f2(sc.x)), b = __fmul2_rn(v[2 * k + 1], f2(sc.x));
        u[k] = codes4<FMT>(a.x, a.y, b.x, b.y);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// The transposed codes, column sums and, where whole blocks line up with the tiles, the codes along the
// rows: a persistent CTA of 1024 threads per SM walks 128 x 128 tiles of g's columns, in two phases.
//   Rows     thread (rr, cc) of 64 x 16 computes rows 2rr, 2rr+1 and columns 8cc .. 8cc+7 of da, du and g in fp32 from
//            one decoding and one activation, leaves all three in shared memory in fp32, and writes da's
//            and du's codes along the rows (maxima by shuffle over the 16 lanes of a row).
//   Columns  thread (c, k) of 128 x 8 takes column c, rows 16k .. 16k+15 of each: maxima and sums over its
//            values, then over the 8 lanes of a column, one scale, 16 codes, one 16-byte store (8 lanes: a
//            whole 128-byte line).  The next tile's values are loaded into registers meanwhile.
// Shared memory holds pairs of rows, so that the column phase reads two values at once; 16-byte units are XORed by
// unit / 8 and by row / 16: both phases hit 32 banks.
// Bound: the issue slots (71% in use, 60 instructions a value of g).  SwiGLU of 8192 x 11008 in bf16 with dbias: 199 us,
// 4.2 TB/s; GELU of 8192 x 16384 263 us; 2999 x 1408 in 24 groups, GELU 18 us (three rounds of tiles).  Slower at the
// first of these: values kept in registers by 512 threads (305 us), CTA pairs that share the rows' maxima over distributed
// shared memory with two CTAs an SM (421), short tiles with fewer lanes a column (205), packed products (207).
namespace bd {
constexpr int THREADS = 1024, TILE = 128;
}

template <int XKIND, int FMT, bool GATED, bool SILU>
__global__ void __launch_bounds__(bd::THREADS, 1) block_dact_kernel(const BlockDactArgs a) {
    using namespace bd;
    constexpr int NM = GATED ? 3 : 2, NH = NM - 1;  // matrices, those of dh
    extern __shared__ __align__(16) float2 val[];   // [NM][TILE / 2][TILE] pairs of rows
    const GroupTable table = group_table(val + NM * TILE * TILE / 2, a.n_groups);  // only with offsets
    __shared__ Walk walk;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int rr = tid >> 4, cc = tid & 15;        // rows
    const int col = tid >> 3, chunk = tid & 7;     // columns
    const uint32_t cols = (uint32_t)a.cols, wide = (uint32_t)a.wide, rows = (uint32_t)a.rows, ld = (uint32_t)a.col_ld;
    pdl_wait();
    pdl_trigger();
    if (a.offsets) build_group_table(table, a.offsets, a.n_groups, a.rows);
    if (tid == 0) walk_start(walk, table, a.offsets, a.n_groups, a.rows, a.tiles, a.across);
    __syncthreads();
    uint4 x[2][XKIND == FP8DL_BF16 ? 1 : 2];  // as loaded: dg, the codes of a and u, their factors
    uint2 qa[2], qu[2];
    float fa[2], fu[2];
    const auto load = [&](const Step &s, int i) {  // row i of the thread's two
        const uint32_t c = s.col * TILE + 8 * cc, r = (uint32_t)s.r0 + 2 * rr + i;
        const int have = c < cols ? s.n - 2 * rr : 0;
        const char *p = static_cast<const char *>(a.dg) + (wide_mul(r, cols) + c) * (XKIND == FP8DL_BF16 ? 2 : 4);
        const uint8_t *q = a.h_q + wide_mul(r, wide) + c;
        const float *f = a.h_s + wide_mul(c >> 7, rows) + r, *g = a.h_s + wide_mul((c + cols) >> 7, rows) + r;
        x[i][0] = make_uint4(0u, 0u, 0u, 0u);
        if (XKIND == FP8DL_F32) x[i][XKIND == FP8DL_F32] = make_uint4(0u, 0u, 0u, 0u);
        qa[i] = qu[i] = make_uint2(0u, 0u);
        fa[i] = fu[i] = 0.0f;
        if (i < have) {
            x[i][0] = ldg_stream(p);
            if (XKIND == FP8DL_F32) x[i][XKIND == FP8DL_F32] = ldg_stream(p + 16);
            qa[i] = __ldg(reinterpret_cast<const uint2 *>(q));
            fa[i] = __ldg(f);
            if (GATED) {
                qu[i] = __ldg(reinterpret_cast<const uint2 *>(q + cols));
                fu[i] = __ldg(g);
            }
        }
    };
    load(walk.step[0], 0);
    load(walk.step[0], 1);
    for (int cur = 0; walk.step[cur].n;) {
        const int next = cur == 2 ? 0 : cur + 1, after = next == 2 ? 0 : next + 1, n = walk.step[cur].n;
        if (4 * warp < ((n + 15) & ~15)) {  // rows up to the last sixteen: those that are not there are zeros
            float2 v[NH][2][4];
            uint32_t ha[2][4], hu[2][4];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                decode8(qa[i], a.h_e4, ha[i]);
                if (GATED) decode8(qu[i], a.h_e4, hu[i]);
            }
            float4 *to = reinterpret_cast<float4 *>(val + rr * TILE);
#pragma unroll
            for (int p = 0; p < 4; p++) {
                float2 g[2];
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    float2 dg;
                    if (XKIND == FP8DL_BF16) {
                        const uint32_t w = p == 0 ? x[i][0].x : p == 1 ? x[i][0].y : p == 2 ? x[i][0].z : x[i][0].w;
                        dg = make_float2(bf16_lo(w), bf16_hi(w));
                    } else {
                        const uint4 &w = x[i][XKIND == FP8DL_F32 ? p >> 1 : 0];
                        dg = p & 1 ? make_float2(__uint_as_float(w.z), __uint_as_float(w.w)) : make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
                    }
                    gradient2<GATED, SILU>(ha[i][p], fa[i], GATED ? hu[i][p] : 0u, fu[i], dg, v[0][i][p], v[NH - 1][i][p], g[i]);
                }
                const int unit = 4 * cc + p, at = unit ^ (unit >> 3 & 7) ^ (rr >> 3);
#pragma unroll
                for (int m = 0; m < NH; m++) to[m * (TILE * TILE / 4) + at] = make_float4(v[m][0][p].x, v[m][1][p].x, v[m][0][p].y, v[m][1][p].y);
                to[NH * (TILE * TILE / 4) + at] = make_float4(g[0].x, g[1].x, g[0].y, g[1].y);
            }
            load(walk.step[next], 0);  // zeros behind the last tile
            const Step &s = walk.step[cur];
            if (a.dh_q && s.col < a.row_first) {
                const uint32_t c = s.col * TILE + 8 * cc, r = (uint32_t)s.r0 + 2 * rr;
                const bool both = GATED && a.row_jobs == 0;  // u's blocks line up too; otherwise they are the other kernel's
                put_rows<FMT, NH>(v, a.dh_q + wide_mul(r, wide) + c, cols, wide, a.dh_s + wide_mul(s.col, rows) + r,
                                  wide_mul(cols >> 7, rows), n - 2 * rr, c < cols, both);
            }
        }
        else load(walk.step[next], 0);
        if (tid == THREADS - 1) walk_on(walk, table, a.offsets, a.rows, a.across, next, after);
        __syncthreads();
        const uint32_t first = walk.step[cur].col * TILE + col, tile = walk.step[cur].tile;
        const bool has = 16 * chunk < n, there = first < cols;
        const int unit = col >> 1;
        const float2 *from = val + 8 * chunk * TILE + 2 * (unit ^ (unit >> 3 & 7) ^ chunk) + (col & 1);
        const uint64_t code = wide_mul(first, ld) + tile * TILE + 16 * chunk, factor = wide_mul(tile, wide) + first;
#pragma unroll
        for (int m = 0; m < NM; m++) {
            uint8_t *q = m < NH ? a.dh_qt : a.g_qt;
            const bool sum = m < NH && a.ws, right = GATED && m == 1;
            if (m == NM - 2) load(walk.step[next], 1);
            if (!q && !sum) continue;
            asm volatile("" ::: "memory");  // one matrix after the other: the registers hold one's values
            float2 v[8];
#pragma unroll
            for (int k = 0; k < 8; k++) v[k] = has ? from[m * (TILE * TILE / 2) + k * TILE] : f2(0.0f);
            if (sum) {  // over the rows, in a fixed order
                float2 t2 = v[0];
#pragma unroll
                for (int k = 1; k < 8; k++) t2 = __fadd2_rn(t2, v[k]);
                float t = t2.x + t2.y;
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                if (chunk == 0 && there) a.ws[factor + (right ? cols : 0)] = t;
            }
            if (!q) continue;
            float f;
            uint4 u;
            if (m < NH)
                u = put_column<FMT>(v, f);
            else if (a.h_e4)
                u = put_column<FP8DL_E4M3>(v, f);
            else
                u = put_column<FP8DL_E5M2>(v, f);
            if (there) {
                *reinterpret_cast<uint4 *>(q + code + (right ? wide_mul(cols, ld) : 0)) = u;
                if (chunk == 0) (m < NH ? a.dh_st + factor : a.g_st + wide_mul(tile, cols) + first)[right ? cols : 0] = f;
            }
        }
        __syncthreads();
        cur = next;
    }
}

// Blocks of dh along the rows, a.row_jobs of a row from a.row_first on: all of them where nothing else is
// wanted; those of u's half (and the one that holds the border) where cols is not a multiple of 128 and
// the tiles above do not hold whole blocks.  16 lanes a block, two rows of each in flight.  (8192 x 11024: 310 us for both
// kernels, 190 where the blocks line up.)
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
    if (first + (int64_t)tile * ACT_ROWS >= end) return;
    const uint32_t cols = (uint32_t)a.cols, wide = (uint32_t)a.wide, rows = (uint32_t)a.rows;
    const uint32_t r = (uint32_t)first + tile * ACT_ROWS + 2 * (threadIdx.x >> 4);
    const uint32_t at = job * 128 + 8 * (threadIdx.x & 15);  // of dh
    const bool right = GATED && at >= cols;
    const uint32_t c = right ? at - cols : at;
    const bool row[2] = {r < (uint32_t)end, r + 1 < (uint32_t)end};
    float2 dg[2][4], v[2][1][4];
    uint2 qa[2], qu[2];
    float fa[2], fu[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const bool ok = row[i] && at < wide;
        qa[i] = qu[i] = make_uint2(0u, 0u);
        fa[i] = fu[i] = 0.0f;
        if (a.bf16)
            load8<FP8DL_BF16>(a.dg, wide_mul(r + i, cols) + c, ok, dg[i]);
        else
            load8<FP8DL_F32>(a.dg, wide_mul(r + i, cols) + c, ok, dg[i]);
        if (ok) {
            const uint8_t *q = a.h_q + wide_mul(r + i, wide) + c;
            qa[i] = __ldg(reinterpret_cast<const uint2 *>(q));
            fa[i] = __ldg(a.h_s + wide_mul(c >> 7, rows) + r + i);
            if (GATED && !right) {
                qu[i] = __ldg(reinterpret_cast<const uint2 *>(q + cols));
                fu[i] = __ldg(a.h_s + wide_mul((c + cols) >> 7, rows) + r + i);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        uint32_t ha[4], hu[4];
        decode8(qa[i], a.h_e4, ha);
        if (GATED) decode8(qu[i], a.h_e4, hu);
        float2 du, g;
#pragma unroll
        for (int p = 0; p < 4; p++) {
            gradient2<GATED, SILU>(ha[p], fa[i], GATED ? hu[p] : 0u, fu[i], dg[i][p], v[i][0][p], du, g);
            if (GATED && right) v[i][0][p] = du;
        }
    }
    uint8_t *const q[1] = {a.dh_q + wide_mul(r, wide) + at};
    const uint32_t ld[1] = {wide};
    const float f = put_blocks<FMT, 1>(v, q, ld, row[0] && at < wide, row[1] && at < wide);
    if ((threadIdx.x & 7) == 0 && row[threadIdx.x >> 3 & 1]) a.dh_s[wide_mul(at >> 7, rows) + r + (threadIdx.x >> 3 & 1)] = f;
}

template <int XKIND, int FMT, bool GATED, bool SILU>
static fp8dl_status launch_dact_tiles(const BlockDactArgs &a, int dev, int sms, cudaStream_t st, bool pdl) {
    static std::atomic<uint64_t> done{0};
    constexpr size_t values = (GATED ? 3 : 2) * bd::TILE * bd::TILE * sizeof(float);
    auto *kernel = block_dact_kernel<XKIND, FMT, GATED, SILU>;
    FP8DL_TRY(allow_smem(kernel, values + group_table_bytes(kMaxGroups), dev, done, "fp8_block_dact"));
    const int64_t most = (int64_t)a.tiles * a.across;
    (void)launch_kernel(kernel, dim3((unsigned)(most < sms ? most : sms)), dim3(bd::THREADS), values + group_table_bytes(a.n_groups), st, 0,
                        pdl, a);
    note_launch();
    return check_launch("fp8_block_dact");
}

template <int FMT, bool GATED, bool SILU>
static fp8dl_status launch_dact(const BlockDactArgs &a, bool tiles, int dev, int sms, cudaStream_t st, bool pdl) {
    if (tiles)
        FP8DL_TRY((a.bf16 ? launch_dact_tiles<FP8DL_BF16, FMT, GATED, SILU>(a, dev, sms, st, pdl)
                          : launch_dact_tiles<FP8DL_F32, FMT, GATED, SILU>(a, dev, sms, st, pdl)));
    if (a.dh_q && a.row_jobs) {
        const int64_t ctas = (a.rows + ba::ACT_ROWS - 1) / ba::ACT_ROWS * a.row_jobs;
        (void)launch_kernel(block_dact_rows_kernel<FMT, GATED, SILU>, dim3((unsigned)ctas), dim3(ba::ACT_THREADS), 0, st, 0, pdl, a);
        note_launch();
        FP8DL_TRY(check_launch("fp8_block_dact(rows)"));
    }
    return FP8DL_OK;
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
    uint32_t tiles, across;
};

// Two codes (the lower or upper half of a word) -> their values times f.
template <bool E4, bool UPPER>
__device__ __forceinline__ float2 value2(uint32_t word, float f) {
    uint32_t h;
    if (E4 && UPPER)
        asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;}" : "=r"(h) : "r"(word));
    else if (E4)
        asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(h) : "r"(word));
    else
        h = __byte_perm(word, 0, UPPER ? 0x3424 : 0x1404);  // E5M2 is the upper byte of an fp16
    return __fmul2_rn(half_pair(h), f2(f));
}
// The same of pair p of eight codes.
template <bool E4>
__device__ __forceinline__ float2 pair_of(uint2 u, int p, float f) {
    return p == 0 ? value2<E4, false>(u.x, f) : p == 1 ? value2<E4, true>(u.x, f) : p == 2 ? value2<E4, false>(u.y, f) : value2<E4, true>(u.y, f);
}

// Row-wise codes to transposed ones: persistent CTAs, four per SM, walk 128 x 128 tiles.  Thread (rr, cc) of 16 x 16 holds
// the codes of rows 8rr .. 8rr+7, columns 8cc .. 8cc+7 and decodes them twice, for the column maxima (8 rows in the
// thread, two row groups by shuffle, eight warps through shared memory) and for the new codes: kept as fp32 they
// would take 64 registers and leave two CTAs an SM.  The new codes go through shared memory in 8-byte pieces XORed by
// column group and leave as whole 128-byte lines.  Neighbours copy the next tile's codes into each other's slots of
// shared memory meanwhile, 16 bytes at a time (no barrier, no registers), and read the indices of the one after it.
// Bound: the issue slots (63% in use, 12 instructions a value) and the three barriers a tile.  32768 x 4096 in 16 groups
// through an index: 62 us, 3.3 TB/s (64 values a thread without the walk 134, bulk copies of the rows 71, eight bytes a
// copy 66); 3001 x 2048 5.4 us.
namespace br {
constexpr int THREADS = 256, TILE = 128;
}
template <int FMT, bool E4>
__global__ void __launch_bounds__(br::THREADS, 4) block_recode_kernel(const BlockRecodeArgs a) {
    using namespace br;
    __shared__ __align__(16) uint8_t code[TILE * TILE];
    __shared__ __align__(16) uint2 in[8][THREADS];
    __shared__ __align__(16) float part[8][TILE];
    __shared__ __align__(16) float scale[TILE];
    __shared__ __align__(16) float fac[2][TILE];  // the rows' factors, of every other tile
    __shared__ Walk walk;
    extern __shared__ __align__(16) uint8_t dyn[];
    const GroupTable table = group_table(dyn, a.n_groups);  // only with offsets
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rr = tid >> 4, cc = tid & 15;
    const uint32_t cols = (uint32_t)a.cols, src_rows = (uint32_t)a.src_rows;
    pdl_wait();
    pdl_trigger();
    if (a.offsets) build_group_table(table, a.offsets, a.n_groups, a.rows);
    if (tid == 0) walk_start(walk, table, a.offsets, a.n_groups, a.rows, a.tiles, a.across);
    __syncthreads();
    int32_t src;  // lane i of each 16: the source of row 8rr + i of the tile whose codes come next, -1: zeros
    const auto look = [&](const Step &s) {
        src = -1;
        if ((lane & 15) < 8 && 8 * rr + (lane & 7) < s.n) {
            src = (int32_t)s.r0 + 8 * rr + (lane & 7);
            if (a.index) src = __ldg(a.index + src);
        }
    };
    const auto fetch = [&](const Step &s, int slot) {
        if (src >= 0 && (uint32_t)src >= src_rows) src = -1;
        if ((lane & 15) < 8)
            copy_async<4>(&fac[slot][8 * rr + (lane & 7)], a.s + (src >= 0 ? wide_mul(s.col, src_rows) + (uint32_t)src : 0), src >= 0);
        // rows and columns that are not there: none is copied, and the address stays on the tensor
        const uint32_t c = s.col * TILE + 8 * (cc & 14);
        const uint8_t *q = a.q + min(c, cols - 16);
        const int32_t least = c < cols ? 0 : 0x7fffffff;
        const int half = 4 * (lane & 1);  // of two neighbours one copies the first four rows for both, one the others
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int32_t r = __shfl_sync(0xffffffffu, src, (lane & 16) + half + i);
            copy_async<16, true>(&in[half + i][tid & ~1], q + wide_mul(max(r, 0), cols), r >= least);
        }
    };
    look(walk.step[0]);
    fetch(walk.step[0], 0);
    look(walk.step[1]);
    for (int cur = 0, slot = 0; walk.step[cur].n; slot ^= 1) {
        const int next = cur == 2 ? 0 : cur + 1, after = next == 2 ? 0 : next + 1, n = walk.step[cur].n;
        const bool busy = 16 * warp < n;  // the warp has rows
        copy_wait_all();
        __syncwarp();  // a row's factor is another lane's copy
        uint2 u[8];
#pragma unroll
        for (int i = 0; i < 8; i++) u[i] = in[i][tid];
        __syncwarp();  // before a neighbour copies over them
        if (walk.step[next].n) fetch(walk.step[next], slot ^ 1);
        const float *f = &fac[slot][8 * rr];
        float m[8];
#pragma unroll
        for (int j = 0; j < 8; j++) m[j] = 0.0f;
        if (busy) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 k = *reinterpret_cast<const float2 *>(f + i);
#pragma unroll
                for (int p = 0; p < 4; p++) {
                    float2 x = pair_of<E4>(u[i], p, k.x), y = pair_of<E4>(u[i + 1], p, k.y);
                    // an infinity turns into NaN, which does not count
                    x = __ffma2_rn(x, f2(0.0f), x), y = __ffma2_rn(y, f2(0.0f), y);
                    m[2 * p] = max3(m[2 * p], x.x, y.x), m[2 * p + 1] = max3(m[2 * p + 1], x.y, y.y);
                }
            }
            const bool up = lane & 16;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float send = up ? m[j] : m[j + 4], keep = up ? m[j + 4] : m[j];
                m[j] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 16));
            }
        }
        *reinterpret_cast<float4 *>(&part[warp][8 * cc + (lane & 16 ? 4 : 0)]) = make_float4(m[0], m[1], m[2], m[3]);
        __syncthreads();
        if (tid < TILE) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; w += 2) t = max3(t, part[w][tid], part[w + 1][tid]);
            const float2 sc = block_scale_fast<FMT>(t);
            scale[tid] = sc.x;
            const uint32_t c = walk.step[cur].col * TILE + tid;
            if (c < cols) a.col_s[wide_mul(walk.step[cur].tile, cols) + c] = sc.y;
        } else if (tid == TILE) {
            walk_on(walk, table, a.offsets, a.rows, a.across, next, after);
        }
        __syncthreads();
        look(walk.step[after]);
        uint8_t *at = code + 8 * cc * TILE + ((rr ^ cc) << 3);
        if (busy) {
#pragma unroll
            for (int p = 0; p < 4; p++) {  // columns 8cc + 2p and the next, four rows at a time
                const float2 sc = *reinterpret_cast<const float2 *>(&scale[8 * cc + 2 * p]);
                uint32_t w[2][2];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float4 k = *reinterpret_cast<const float4 *>(f + 4 * h);
                    float2 y[4];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        asm volatile("" : "+r"(u[4 * h + i].x), "+r"(u[4 * h + i].y)::"memory");  // decoded again, not kept
                        const float2 x = pair_of<E4>(u[4 * h + i], p, i == 0 ? k.x : i == 1 ? k.y : i == 2 ? k.z : k.w);
                        y[i] = __fmul2_rn(x, sc);
                    }
                    w[0][h] = codes4<FMT>(y[0].x, y[1].x, y[2].x, y[3].x), w[1][h] = codes4<FMT>(y[0].y, y[1].y, y[2].y, y[3].y);
                }
                *reinterpret_cast<uint2 *>(at + 2 * p * TILE) = make_uint2(w[0][0], w[0][1]);
                *reinterpret_cast<uint2 *>(at + (2 * p + 1) * TILE) = make_uint2(w[1][0], w[1][1]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) *reinterpret_cast<uint2 *>(at + j * TILE) = make_uint2(0u, 0u);
        }
        __syncthreads();
        const int ch = tid & 7;
        const uint32_t first = walk.step[cur].col * TILE, ld = (uint32_t)a.col_ld, left = min((uint32_t)TILE, cols - first);
        uint8_t *to = a.col_q + wide_mul(first + (tid >> 3), ld) + walk.step[cur].tile * TILE + 16 * ch;
        const uint8_t *from = code + (tid >> 3) * TILE;
#pragma unroll
        for (int k = 0; k < 4; k++) {  // two pieces of 8 bytes, each where the XOR put it
            const uint32_t c = (tid >> 3) + 32 * k, g = c >> 3;
            const uint2 x = *reinterpret_cast<const uint2 *>(from + 32 * k * TILE + (((2 * ch) ^ g) << 3));
            const uint2 y = *reinterpret_cast<const uint2 *>(from + 32 * k * TILE + (((2 * ch + 1) ^ g) << 3));
            if (c < left) *reinterpret_cast<uint4 *>(to) = make_uint4(x.x, x.y, y.x, y.y);
            to += wide_mul(32, ld);
        }
        cur = next;
    }
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
    const bool split = gated && cols % 128 != 0;
    a.jobs = (uint32_t)((cols + 127) / 128 + (split && h_q ? (a.wide + 127) / 128 : 0));
    const int64_t ctas = (rows + ba::ACT_ROWS - 1) / ba::ACT_ROWS * a.jobs;
    FP8DL_TRY(check_tiles(ctas, rows, cols));
    int sms = 0;
    FP8DL_TRY(current_device(nullptr, &sms));
    const int64_t resident = (int64_t)sms * ba::ACT_CTAS;
    if (rows == 0) return FP8DL_OK;
    const bool pdl = short_call_bytes((double)rows * a.wide * ((h_dtype == FP8DL_BF16 ? 2.0 : 4.0) + (h_q ? 1.0 : 0.0)) + (double)rows * cols);
    const bool keep = h_q && !split;
    auto *kernel = &block_act_kernel<FP8DL_BF16, FP8DL_E4M3, false, false, false>;
#define FP8DL_ACT_KEEP(X, F, G, S) (keep ? block_act_kernel<X, F, G, S, true> : block_act_kernel<X, F, G, S, false>)
#define FP8DL_ACT(X, F)                                                                                           \
    kernel = gated ? (act_silu(act) ? FP8DL_ACT_KEEP(X, F, true, true) : FP8DL_ACT_KEEP(X, F, true, false))         \
                   : (act_silu(act) ? FP8DL_ACT_KEEP(X, F, false, true) : FP8DL_ACT_KEEP(X, F, false, false))
    if (h_dtype == FP8DL_BF16 && out_dtype == FP8DL_E4M3) FP8DL_ACT(FP8DL_BF16, FP8DL_E4M3);
    else if (h_dtype == FP8DL_BF16) FP8DL_ACT(FP8DL_BF16, FP8DL_E5M2);
    else if (out_dtype == FP8DL_E4M3) FP8DL_ACT(FP8DL_F32, FP8DL_E4M3);
    else FP8DL_ACT(FP8DL_F32, FP8DL_E5M2);
#undef FP8DL_ACT
#undef FP8DL_ACT_KEEP
    (void)launch_kernel(kernel, dim3((unsigned)(ctas < resident ? ctas : resident)), dim3(ba::ACT_THREADS), 0, (cudaStream_t)stream, 0, pdl, a);
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
    int dev = 0, sms = 0;
    FP8DL_TRY(current_device(&dev, &sms));
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
    FP8DL_TRY(launch(a, tiles, dev, sms, st, pdl));
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
    a.q = src_rows ? q : col_q, a.s = src_rows ? s : col_s;  // without source rows nothing is read
    a.src_rows = src_rows;
    a.rows = rows;
    a.cols = cols;
    a.index = index, a.offsets = offsets;
    a.n_groups = n_groups;
    a.col_q = col_q, a.col_s = col_s;
    a.col_ld = fp8_block_padded_rows(rows, n_groups);
    a.across = (uint32_t)((cols + 127) / 128);
    a.tiles = (uint32_t)(a.col_ld / 128);
    const int64_t most = a.col_ld / 128 * a.across;
    FP8DL_TRY(check_tiles(most, rows, cols));
    int dev = 0, sms = 0;
    FP8DL_TRY(current_device(&dev, &sms));
    if (rows == 0) return FP8DL_OK;
    const bool pdl = short_call_bytes(2.0 * (double)rows * (double)cols), e4 = q_fp8 == FP8DL_E4M3;
    auto *kernel = out_dtype == FP8DL_E4M3 ? (e4 ? block_recode_kernel<FP8DL_E4M3, true> : block_recode_kernel<FP8DL_E4M3, false>)
                                           : (e4 ? block_recode_kernel<FP8DL_E5M2, true> : block_recode_kernel<FP8DL_E5M2, false>);
    static std::atomic<uint64_t> done[4];  // past 48 KB with the groups' table
    FP8DL_TRY(allow_smem(kernel, group_table_bytes(kMaxGroups), dev, done[2 * (out_dtype == FP8DL_E4M3) + e4], "fp8_block_recode"));
    (void)launch_kernel(kernel, dim3((unsigned)(most < 4 * sms ? most : 4 * sms)), dim3(br::THREADS), group_table_bytes(n_groups),
                        (cudaStream_t)stream, 0, pdl, a);
    note_launch();
    return check_launch("fp8_block_recode");
}
