/*
 * fp8dl.h — C ABI of the GB300 (sm_103a) FP8 delayed-scaling linear layer.
 *
 * The method (per-tensor FP8 training with delayed scaling, as run by
 * Transformer Engine's te.Linear under a DelayedScaling recipe) is described
 * in "FP8 低精度训练：Transformer Engine 简析" (m.haoling.cc), §三 "FP8技术分析":
 *   - §三.1 "宏观实现框架": one scale per tensor, symmetric linear quantisation;
 *     delayed scaling takes the max of an amax history window and sets
 *     scale = (FP8_MAX / amax) / 2^margin; recipe parameters margin, interval,
 *     fp8_format (forward E4M3, backward E5M2 in HYBRID), amax_history_len.
 *   - §三.3 "FP8框架TE计算流程": inputs and weights are cast to FP8 with the
 *     stored scale, the cast writes its amax into the history, fp8_gemm
 *     computes; at autocast exit the amaxes update history and scale.
 *   - §三.4 "Tensor Core如何进行FP8训练": the GEMM returns a high-precision
 *     result; every dimension is a multiple of 16.
 * MXFP8 (block-scaled FP8) is named by the Transformer Engine README
 * ("亮点": MXFP8 on Blackwell); the pages do not define it.  This library reads
 * it as E4M3 data with one E8M0 (power-of-two) scale per 32 consecutive
 * elements along the reduction axis.
 *
 * Conventions shared by every call
 *   Memory      All pointers are DEVICE pointers owned by the caller, unless a
 *               parameter says "host".  The library allocates no device memory;
 *               where a call needs scratch space the caller passes it in
 *               (see fp8_cast_workspace_size).
 *   Layout      Matrices are row-major and densely packed.  FP8 data are one
 *               byte per element (E4M3 or E5M2 codes).  bf16 is IEEE bfloat16.
 *   GEMMs       Every GEMM is "TN": D[M,N] = A[M,K] * B[N,K]^T, both operands
 *               row-major with K contiguous.  The linear layer uses it three
 *               times: forward Y = X W^T (A = X, B = W), dgrad dX = dY W
 *               (A = dY, B = W^T, the transposed copy of W's cast), wgrad
 *               dW = dY^T X (A = dY^T, B = X^T, the transposed copies).
 *   Shapes      Every dimension must be a positive multiple of 16 (32 for the
 *               MXFP8 calls); otherwise FP8DL_ERR_SHAPE.  Pointers must be
 *               16-byte aligned (FP8DL_ERR_ALIGN).
 *   Streams     Every call is asynchronous on `stream` (NULL = the legacy
 *               default stream) and never synchronises with the host.
 *               Scales are read from device memory, so a training step never
 *               waits for the host.
 *   Errors      Argument checks run on the host before any launch and return a
 *               status; nothing throws across the ABI and no kernel traps.
 *               fp8dl_last_error() returns the calling thread's last message.
 *               GEMM pipelines bound every wait; if a wait runs out the kernel
 *               stops, writes FP8DL_ERR_TIMEOUT into *dev_status (when given)
 *               and returns, leaving D undefined.
 *   Device      The library is built for sm_103a only (GB300).  Calls on any
 *               other device return FP8DL_ERR_UNSUPPORTED_DEVICE.
 */
#ifndef FP8DL_H
#define FP8DL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same handle as cudaStream_t. */
typedef struct CUstream_st *fp8dl_stream_t;

typedef enum {
    FP8DL_OK = 0,
    FP8DL_ERR_INVALID_ARG = 1,        /* null pointer, unknown enum, bad recipe   */
    FP8DL_ERR_SHAPE = 2,              /* dimension not a positive multiple of 16  */
    FP8DL_ERR_ALIGN = 3,              /* pointer not 16-byte aligned              */
    FP8DL_ERR_UNSUPPORTED_DEVICE = 4, /* current device is not sm_103             */
    FP8DL_ERR_CUDA = 5,               /* a CUDA runtime/driver call failed        */
    FP8DL_ERR_TIMEOUT = 6,            /* written to *dev_status by a kernel only  */
    FP8DL_ERR_WORKSPACE = 7           /* workspace missing or too small           */
} fp8dl_status;

/* FP8 element formats.  E4M3: bias 7, max 448, no infinity, S.1111.111 = NaN.
 * E5M2: bias 15, max 57344, S.11111.00 = infinity, other S.11111.xx = NaN. */
typedef enum { FP8DL_E4M3 = 0, FP8DL_E5M2 = 1 } fp8dl_fp8_dtype;

/* High-precision element types. */
typedef enum { FP8DL_F32 = 0, FP8DL_BF16 = 1 } fp8dl_hp_dtype;

/* Recipe format: E4M3 everywhere, or HYBRID (E4M3 forward, E5M2 gradients). */
typedef enum { FP8DL_FORMAT_E4M3 = 0, FP8DL_FORMAT_HYBRID = 1 } fp8dl_format;

/* Delayed-scaling recipe (§三.1 "宏观实现框架" lists margin, interval,
 * fp8_format and amax_history_len; "max" is the window algorithm of the
 * Transformer Engine tutorial's HYBRID recipe).  Host struct. */
typedef struct {
    int32_t margin;            /* scale = (FP8_MAX/amax) / 2^margin, 0 <= margin <= 126 */
    int32_t interval;          /* recompute the scale when step % interval == 0, >= 1   */
    int32_t fp8_format;        /* fp8dl_format; informs which slots use E5M2            */
    int32_t amax_history_len;  /* L >= 1, window length of the amax history            */
    int32_t amax_compute_algo; /* 0 = max over the window (the only algorithm)         */
} fp8dl_recipe;

/* ----------------------------------------------------------------------------
 * Scaling state.  One "slot" per scaled tensor (e.g. input, weight and
 * grad_output of each GEMM).  The state of n slots is one caller-allocated
 * device block of fp8dl_scaling_state_bytes(L, n) bytes; slot i starts at
 * byte i * fp8dl_slot_stride(L) and holds
 *     float   scale       offset 0   multiplier used by the next casts
 *     float   scale_inv   offset 4   1/scale, read by the GEMM epilogue
 *     float   amax        offset 8   amax recorded since the last update;
 *                                    casts max their |x| into it atomically
 *     int32   hist_pos    offset 12  next write position in the history ring
 *     int32   fp8_dtype   offset 16  fp8dl_fp8_dtype of the slot (FP8_MAX)
 *     int32   reserved[3]
 *     float   hist[L]     offset 32  amax history ring
 * The block is plain data: saving and restoring it (with the caller's step
 * counter) resumes training bit-identically.
 * ------------------------------------------------------------------------- */
size_t fp8dl_slot_stride(int32_t amax_history_len);
size_t fp8dl_scaling_state_bytes(int32_t amax_history_len, int32_t n_slots);

/* Initialise n_slots slots: scale = scale_inv = 1, amax = 0, hist = 0,
 * hist_pos = 0, fp8_dtype = slot_fp8_dtype[i] (HOST array of n_slots). */
fp8dl_status fp8_scaling_state_init(const fp8dl_recipe *recipe, int32_t n_slots,
                                    const int32_t *slot_fp8_dtype, void *state,
                                    fp8dl_stream_t stream);

/* Delayed scale update of every slot (§三.1 "宏观实现框架", §三.3: at autocast
 * exit the recorded amaxes update the history and the scale).  Per slot:
 *   hist[hist_pos] = amax; hist_pos = (hist_pos + 1) % L; amax = 0;
 *   if (step % interval == 0):
 *       a = max(hist[0..L))
 *       if a > 0 and finite: s = fl32(FP8_MAX / a) / 2^margin
 *           if s > 0 and finite: scale = s, scale_inv = fl32(1 / s)
 *   (otherwise scale and scale_inv keep their values).
 * `step` is the caller's step counter.  One launch for all slots. */
fp8dl_status fp8_update_scale(const fp8dl_recipe *recipe, int32_t n_slots, void *state,
                              int64_t step, fp8dl_stream_t stream);

/* First step: fill every history entry with the slot's recorded amax (from
 * an amax-only cast pass), clear amax, set hist_pos = 0 and derive the scale
 * as above, so the first real cast already uses a data-derived scale. */
fp8dl_status fp8_seed_amax_history(const fp8dl_recipe *recipe, int32_t n_slots, void *state,
                                   fp8dl_stream_t stream);

/* ----------------------------------------------------------------------------
 * Fused cast + amax (+ transpose) (+ bias gradient) (§三.1 / §三.3: the cast
 * to FP8 uses the stored scale and records the tensor's amax).
 *   x        [rows x cols], x_dtype (FP8DL_F32 or FP8DL_BF16)
 *   scale    device float (a slot's scale)
 *   out      [rows x cols] FP8 codes, out[i,j] = enc(fl32(x[i,j] * scale)), or NULL
 *   out_t    [cols x rows] FP8 codes, out_t[j,i] = out[i,j], or NULL
 *   amax     device float, atomically max-ed with max |x| (pre-scale), or NULL
 *   scale_inv_out  device float receiving fl32(1 / *scale), the factor that
 *            decodes these codes, or NULL.  Codes kept past the next scale
 *            update (a weight cast once and reused over micro-batches, §三.3:
 *            the cast is skipped while a cached FP8 copy exists) carry their
 *            own decode factor this way, since the update rewrites the slot's
 *            scale_inv.  Written by a one-thread kernel after the cast.
 *   dbias    [cols] fp32 column sums of x (the bias gradient when x is
 *            grad_output), or NULL; overwritten, not accumulated
 *   workspace/workspace_bytes  scratch of fp8_cast_workspace_size(rows, cols)
 *            bytes, needed only when dbias != NULL
 * Encoding: round to nearest even, saturating to +-FP8_MAX (including
 * infinities); NaN gives a NaN code.  With out, out_t and dbias all NULL the
 * call is an amax-only pass. */
size_t fp8_cast_workspace_size(int64_t rows, int64_t cols);

fp8dl_status fp8_cast_amax_transpose(const void *x, int32_t x_dtype, int64_t rows, int64_t cols,
                                     int32_t out_dtype, const float *scale, uint8_t *out,
                                     uint8_t *out_t, float *amax, float *scale_inv_out, float *dbias,
                                     void *workspace, size_t workspace_bytes, fp8dl_stream_t stream);

/* Grouped cast: the casts of up to 8 tensors (say the two weights of a
 * LayerNormMLP, or the weights of several layers) in one launch, so that the
 * small tensors share one grid instead of each paying a launch, a ramp-up
 * and a tail.  Per tensor the results are exactly those of
 * fp8_cast_amax_transpose without dbias (§三.1 / §三.3: the cast with the
 * stored scale records the tensor's amax).
 *   items  HOST array of n items (1 <= n <= 8), each with its own x
 *          [rows x cols], scale, outputs and amax, as in
 *          fp8_cast_amax_transpose; all share x_dtype and out_dtype.
 *   Argument errors of any item are reported before any launch. */
typedef struct {
    const void *x;          /* [rows x cols] of the call's x_dtype */
    int64_t rows, cols;     /* positive multiples of 16 */
    const float *scale;     /* device float */
    uint8_t *out;           /* [rows x cols] codes, or NULL */
    uint8_t *out_t;         /* [cols x rows] codes, or NULL */
    float *amax;            /* device float, max-ed with max |x|, or NULL */
    float *scale_inv_out;   /* device float receiving fl32(1 / *scale), or NULL */
} fp8dl_cast_item;

fp8dl_status fp8_cast_amax_transpose_multi(int32_t n, const fp8dl_cast_item *items, int32_t x_dtype,
                                           int32_t out_dtype, fp8dl_stream_t stream);

/* The same cast for callers that cannot allocate device memory.  The paper
 * has no counterpart to this call: it exists for callers that only hand the
 * library their input and output buffers (a plugin or custom-op interface
 * whose fixed signature has no workspace argument, or a process whose device
 * memory belongs to another allocator that does not let it call cudaMalloc),
 * so they can neither pass the bias-gradient workspace nor allocate one.
 *   Arguments, layouts and results are those of fp8_cast_amax_transpose,
 *   without workspace/workspace_bytes.
 *   Scratch: the dbias workspace is a 4 MiB array in the library's static
 *   device memory (every GPU that loads the library holds it until the
 *   process exits).  Calls with dbias != NULL need
 *   fp8_cast_workspace_size(rows, cols) <= 4 MiB, i.e.
 *   ceil(rows/128) * cols * 4 <= 4194304; larger ones return
 *   FP8DL_ERR_WORKSPACE before any launch.  The call allocates nothing
 *   (no cudaMalloc, cudaFree or allocating library routine).
 *   First call per device: looks up the array's device address with
 *   cudaGetSymbolAddress (that device current) and caches it; make that first
 *   call before any stream capture.
 *   Sharing: all calls on a device share the one array, which keeps the last
 *   call's contents; each call writes every scratch entry it reads, so no
 *   clearing is needed.  A call enqueues its two launches (partials, then
 *   their reduction) under a library lock, so calls from several host
 *   threads on one stream run one after another on the GPU.  Calls whose
 *   work overlaps on the GPU (different streams not ordered by events) race
 *   on the array and give wrong dbias: put them on one stream. */
fp8dl_status fp8_cast_amax_transpose_noalloc(const void *x, int32_t x_dtype, int64_t rows, int64_t cols,
                                             int32_t out_dtype, const float *scale, uint8_t *out,
                                             uint8_t *out_t, float *amax, float *dbias,
                                             fp8dl_stream_t stream);

/* ----------------------------------------------------------------------------
 * FP8 GEMM with dequantising epilogue (§三.3 fp8_gemm; §三.4 high-precision
 * output, dims multiple of 16):
 *   D[m,n] = round_d( acc[m,n] * fl32(a_scale_inv * b_scale_inv) + bias[n] )
 *   (the product and the bias add are one fp32 fused multiply-add)
 *   acc[m,n] = sum_k A[m,k] * B[n,k] on the tcgen05 tensor cores, fp32 accumulate.
 *     A GEMM with K > 8192 and at least two waves of tiles sums the k-blocks of
 *     every other tile of a CTA (pair) last to first (less DRAM traffic); the
 *     order is fixed by the shape and the GPU's SM count, so repeated calls give
 *     the same bits.
 *   A [M x K] codes of a_dtype, B [N x K] codes of b_dtype (E4M3/E5M2 mixed ok)
 *   a_scale_inv, b_scale_inv   device floats (the operands' slots' scale_inv)
 *   bias       [N] of bias_dtype, or NULL
 *   D          [M x N] of d_dtype (FP8DL_BF16 or FP8DL_F32)
 *   dev_status device int or NULL; set to FP8DL_ERR_TIMEOUT if a pipeline wait
 *              runs out (never reset to 0 by the library). */
fp8dl_status fp8_gemm(const uint8_t *A, int32_t a_dtype, const uint8_t *B, int32_t b_dtype,
                      int64_t M, int64_t N, int64_t K, const float *a_scale_inv,
                      const float *b_scale_inv, const void *bias, int32_t bias_dtype, void *D,
                      int32_t d_dtype, int32_t *dev_status, fp8dl_stream_t stream);

/* FP8 GEMM whose epilogue also applies GELU and the FP8 cast of the result
 * (the fc1 GEMM of a LayerNormMLP).  Delayed scaling knows the cast's scale
 * before the GEMM runs ("FP8 低精度训练：Transformer Engine 简析" §三.1: with the
 * scale known in advance the computation stays in one kernel), so the GELU
 * output never makes an HBM round trip:
 *   H[m,n] = bf16( acc[m,n] * fl32(a_scale_inv * b_scale_inv) + bias[n] )   (as fp8_gemm)
 *   G = bf16( GELU(H) )  (erf form; see fp8_gelu_cast)
 *   q = enc(fl32(G * q_scale)) [M x N], q_t = q^T [N x M], *q_amax max-ed with max |G|
 *   g [M x N] bf16 receives G, or NULL.
 * H is bf16.  Results are identical to fp8_gemm followed by fp8_gelu_cast. */
fp8dl_status fp8_gemm_gelu_cast(const uint8_t *A, int32_t a_dtype, const uint8_t *B, int32_t b_dtype,
                                int64_t M, int64_t N, int64_t K, const float *a_scale_inv,
                                const float *b_scale_inv, const void *bias, int32_t bias_dtype, void *H,
                                int32_t q_dtype, const float *q_scale, uint8_t *q, uint8_t *q_t,
                                float *q_amax, void *g, int32_t *dev_status, fp8dl_stream_t stream);

/* FP8 GEMM whose epilogue applies dGELU and the FP8 cast of the result (the
 * fc2 dgrad GEMM of a LayerNormMLP feeding the fc1 backward), with the fc1
 * bias gradient.  As for fp8_gemm_gelu_cast, the delayed scale of the output
 * is known before the GEMM, so dg never makes an HBM round trip:
 *   dg[m,n] = bf16( acc[m,n] * fl32(a_scale_inv * b_scale_inv) )   (no bias)
 *   dh = bf16( dg * GELU'(h) )  (erf form; see fp8_dgelu_cast), h [M x N] bf16
 *   q = enc(fl32(dh * q_scale)) [M x N], q_t = q^T [N x M], *q_amax max-ed with max |dh|
 *   dbias[n] = sum over m of dh[m,n] (fp32, a fixed order), or NULL
 *   dg and dh [M x N] bf16 receive those tensors, or NULL.
 * workspace: fp8_gemm_dgelu_workspace_size(M, N) bytes (16-byte aligned),
 * needed only when dbias != NULL.  Codes, amax, dg and dh are identical to
 * fp8_gemm followed by fp8_dgelu_cast; dbias agrees within its summation
 * bound (the order of the sum differs).  Needs CTA-pair clusters
 * (FP8DL_ERR_UNSUPPORTED_DEVICE otherwise). */
size_t fp8_gemm_dgelu_workspace_size(int64_t M, int64_t N);

fp8dl_status fp8_gemm_dgelu_cast(const uint8_t *A, int32_t a_dtype, const uint8_t *B, int32_t b_dtype,
                                 int64_t M, int64_t N, int64_t K, const float *a_scale_inv,
                                 const float *b_scale_inv, const void *h, void *dg, int32_t q_dtype,
                                 const float *q_scale, uint8_t *q, uint8_t *q_t, float *q_amax,
                                 float *dbias, void *workspace, size_t workspace_bytes, void *dh,
                                 int32_t *dev_status, fp8dl_stream_t stream);

/* ----------------------------------------------------------------------------
 * MXFP8 quantisation (block-scaled FP8, named by the Transformer Engine
 * README).  x [rows x cols] (bf16 or fp32).  Blocks are 32 consecutive
 * elements; per block: e = the smallest integer with amax_b * 2^-e <= 448,
 * clamped to [-127, 127] (amax_b = 0 gives e = 0); scale byte = e + 127 (E8M0);
 * data = enc_e4m3(fl32(x * 2^-e)).
 *   row_q [rows x cols]: blocks along each row, or NULL
 *   row_s  scales of row_q in the tiled layout below (R = rows, NB = cols/32)
 *   col_q [cols x rows]: blocks along each column, stored transposed (row j
 *         of col_q is column j of x), or NULL
 *   col_s  scales of col_q in the tiled layout (R = cols, NB = rows/32)
 * rows and cols must be multiples of 32.
 *
 * Tiled scale layout (the order the tensor cores read block scales in).  For
 * a matrix of R rows with NB blocks per row, S[r][b] is the scale byte of
 * block b of row r.  Rows are grouped by 128 and blocks by 4; each
 * (row group g, block group h) is one 512-byte tile at byte offset
 * (g * ceil(NB/4) + h) * 512, and inside the tile
 *     byte (r % 32) * 16 + ((r % 128) / 32) * 4 + (b % 4)  holds  S[r][b].
 * Total size: mxfp8_scale_bytes(R, 32*NB).  Entries for rows >= R or blocks
 * >= NB (padding) are written as 127 (2^0).
 *
 * dbias [cols] fp32 receives the column sums of x (the bias gradient when x
 * is grad_output; the te.Linear example has bias=True), in the same pass over
 * x, or NULL; overwritten, not accumulated.  The sum runs in a fixed order,
 * so repeated calls give the same bits.  workspace/workspace_bytes: scratch
 * of fp8_cast_workspace_size(rows, cols) bytes (16-byte aligned), needed
 * only when dbias != NULL (FP8DL_ERR_WORKSPACE otherwise). */
size_t mxfp8_scale_bytes(int64_t rows, int64_t cols);

fp8dl_status mxfp8_quantize(const void *x, int32_t x_dtype, int64_t rows, int64_t cols,
                            uint8_t *row_q, uint8_t *row_s, uint8_t *col_q, uint8_t *col_s,
                            float *dbias, void *workspace, size_t workspace_bytes,
                            fp8dl_stream_t stream);

/* MXFP8 GEMM: D[m,n] = round_d( sum_b 2^(ea[m,b]+eb[n,b]) * sum_{k in b} A[m,k]*B[n,k]
 *                               + bias[n] )
 * A [M x K] E4M3 with scales A_s (tiled layout, R = M, NB = K/32);
 * B [N x K] E4M3 with scales B_s (tiled layout, R = N, NB = K/32), as produced
 * by mxfp8_quantize (row_q/row_s of X and W for the forward GEMM; col_q/col_s
 * for the operands of the gradient GEMMs).  M, N, K multiples of 32.
 * bias, D, dev_status and the order of the k-blocks as for fp8_gemm. */
fp8dl_status mxfp8_gemm(const uint8_t *A, const uint8_t *A_s, const uint8_t *B, const uint8_t *B_s,
                        int64_t M, int64_t N, int64_t K, const void *bias, int32_t bias_dtype,
                        void *D, int32_t d_dtype, int32_t *dev_status, fp8dl_stream_t stream);

/* ----------------------------------------------------------------------------
 * Block-scaled FP8: one fp32 scale per 128 values, for a linear layer and for
 * the linear layers of experts (ragged groups of tokens, one weight each).
 * The scale of a block is the just-in-time form of the per-tensor scale
 * FP8_MAX / amax of "FP8 低精度训练：Transformer Engine 简析" §三.1, taken over
 *   1 x 128 blocks of activations and gradients, along the reduction axis of
 *           the product that reads them, and
 *   128 x 128 blocks of weights (one scale serves both of their copies).
 * Per block:  amax = the largest finite |x|;
 *             scale = fl32(FP8_MAX / max(amax, 2^-100)), or 1 if amax = 0;
 *             q = enc(fl32(x * scale)); the stored factor is fl32(1 / scale).
 * Encoding as for the cast (infinities saturate, NaN gives a NaN code).  The
 * last block of a row or column may be short.
 *
 * Scale layouts are block-major: s[b][r] holds the factor of block b of row r,
 * with rows contiguous (a warp of 32 rows reads 128 consecutive bytes).
 *
 * Token dimensions may have any length, also 0 (nothing is written, except
 * sums over no tokens, which are zeros; the tensors may then be NULL).
 * Feature dimensions are positive multiples of 16, those of D below 2^29.
 *
 * Groups: offsets is a DEVICE array of n_groups + 1 non-decreasing int32 with
 * offsets[0] >= 0 and offsets[n_groups] <= rows; group g owns rows
 * offsets[g] .. offsets[g+1]-1, possibly none; 1 <= n_groups <= 1024.  Rows
 * outside every group are neither read nor written.  The host does not see
 * the values: the kernels clamp them to the tensor, so wrong offsets give
 * wrong results but no access out of bounds.  For the same reason a grouped
 * product is laid out for all rows of its tensor: one that is much longer than
 * its groups costs time. */

/* Columns of the transposed codes of fp8_block_quantize: every group is padded
 * to a multiple of 128, at most floor128(rows + 127 * min(n_groups, rows)) in
 * all; for n_groups <= 1 the rows rounded up to a multiple of 128. */
int64_t fp8_block_padded_rows(int64_t rows, int32_t n_groups);

/* Quantise activations or gradients x [rows x cols] (bf16 or fp32) into either
 * or both of
 *   row_q [rows x cols], row_s [ceil(cols/128) x rows]: blocks along each row,
 *         the A operand of the forward and dgrad products;
 *   col_q [cols x T], col_s [T/128 x cols], T = fp8_block_padded_rows(rows,
 *         n_groups): blocks along each column, transposed, the operands of the
 *         wgrad product.  Group g's rows take the next ceil128(length) columns;
 *         its padding columns are zero codes.  Columns beyond the last group's
 *         are not written.
 * offsets/n_groups: NULL and 0 for the whole matrix.
 * dbias [cols] fp32 receives the column sums of x (fixed order), or NULL; only
 * without offsets; workspace of fp8_cast_workspace_size(rows, cols) bytes. */
fp8dl_status fp8_block_quantize(const void *x, int32_t x_dtype, int64_t rows, int64_t cols,
                                const int32_t *offsets, int32_t n_groups, int32_t out_dtype,
                                uint8_t *row_q, float *row_s, uint8_t *col_q, float *col_s,
                                float *dbias, void *workspace, size_t workspace_bytes,
                                fp8dl_stream_t stream);

/* Quantise n_mats weights w [n_mats x rows x cols] (bf16 or fp32) in 128 x 128
 * blocks into either or both of
 *   q   [n_mats x rows x cols], s   [n_mats x ceil(cols/128) x ceil(rows/128)]
 *   q_t [n_mats x cols x rows], s_t [n_mats x ceil(rows/128) x ceil(cols/128)]
 * q/s is the B operand of the forward product, q_t/s_t that of dgrad; q_t is
 * q transposed, code by code.  1 <= n_mats <= 65535. */
fp8dl_status fp8_block_quantize_weight(const void *w, int32_t w_dtype, int32_t n_mats, int64_t rows,
                                       int64_t cols, int32_t out_dtype, uint8_t *q, float *s, uint8_t *q_t,
                                       float *s_t, fp8dl_stream_t stream);

/* Block-scaled FP8 GEMM:
 *   D[m,n] = round_d( sum_b fl32(a_s[b][m] * b_s[b][n / b_rows]) * sum_{k in block b} A[m,k] * B[n,k]
 *                     + bias[n] )
 * Each block's 128 products are summed on the tcgen05 tensor cores in fp32;
 * the sum over blocks is an fp32 fused multiply-add per block, in ascending
 * order of b within each of the up to six contiguous parts that K may be
 * split into for a tile of D; the parts are added in order.
 * Repeated calls give the same bits.
 *   A [M x K] codes of a_dtype, a_s [ceil(K/128) x M]
 *   B [N x K] codes of b_dtype, b_s [ceil(K/128) x ceil(N/b_rows)],
 *     b_rows = 128 (a weight) or 1 (an activation or gradient)
 *   bias [N] of bias_dtype, or NULL; D [M x N] of d_dtype; dev_status as for
 *   fp8_gemm.  M >= 0; N and K positive multiples of 16. */
fp8dl_status fp8_block_gemm(const uint8_t *A, int32_t a_dtype, const float *a_s, const uint8_t *B,
                            int32_t b_dtype, const float *b_s, int32_t b_rows, int64_t M, int64_t N,
                            int64_t K, const void *bias, int32_t bias_dtype, void *D, int32_t d_dtype,
                            int32_t *dev_status, fp8dl_stream_t stream);

/* What fp8_block_gemm (n_groups 0) or fp8_block_gemm_grouped (b_rows 128) runs
 * a product as on the current device; launches nothing.  *tile_rows rows of A
 * are a tile's: 16, 32 or 64 where they are few, else 256; *whole tiles are
 * computed alone and *shared tiles by *shares CTAs (256 rows: CTA pairs; 1 if no
 * tile is shared), each with a part of K.  Groups: the most tiles there can be, whatever the
 * offsets.  M >= 1. */
fp8dl_status fp8_block_gemm_plan(int32_t b_rows, int32_t n_groups, int64_t M, int64_t N, int64_t K,
                                 int32_t *tile_rows, int32_t *shares, int64_t *whole, int64_t *shared);

/* The products of ragged groups of rows with their group's weight (the expert
 * layers' forward product with q/s of the weights, dgrad with q_t/s_t):
 *   D[m,:] = A[m,:] * B[g]^T for the rows m of group g, summed as above
 *   A [M x K], a_s [ceil(K/128) x M]; B [n_groups x N x K],
 *   b_s [n_groups x ceil(K/128) x ceil(N/128)]; D [M x N]. */
fp8dl_status fp8_block_gemm_grouped(const uint8_t *A, int32_t a_dtype, const float *a_s, const uint8_t *B,
                                    int32_t b_dtype, const float *b_s, const int32_t *offsets,
                                    int32_t n_groups, int64_t M, int64_t N, int64_t K, void *D,
                                    int32_t d_dtype, int32_t *dev_status, fp8dl_stream_t stream);

/* The weight gradients of the groups (a ragged reduction over their tokens):
 *   D[g,m,n] = sum over group g's token blocks b of
 *              fl32(a_s[b][m] * b_s[b][n]) * sum_{t in block b} A[m,t] * B[n,t]
 *   A [M x T] with a_s [T/128 x M] and B [N x T] with b_s [T/128 x N]: col_q
 *   and col_s of fp8_block_quantize with the same offsets (A of grad_output,
 *   B of the input), T its padded length, a multiple of 128 (0 if there are no
 *   rows); D [n_groups x M x N]; a group without rows gets zeros.  M >= 1;
 *   N a positive multiple of 16. */
fp8dl_status fp8_block_gemm_grouped_wgrad(const uint8_t *A, int32_t a_dtype, const float *a_s, const uint8_t *B,
                                          int32_t b_dtype, const float *b_s, const int32_t *offsets,
                                          int32_t n_groups, int64_t M, int64_t N, int64_t T, void *D,
                                          int32_t d_dtype, int32_t *dev_status, fp8dl_stream_t stream);

/* ----------------------------------------------------------------------------
 * Expert routing: which experts each token goes to, with which weight and into
 * which row of the grouped products above, and how evenly the experts are used.
 *
 * Token counts may be 0; n_experts is in [1, 1024], any number; k in
 * [1, min(n_experts, 32)]; tokens * k < 2^31.  Logits are bf16 or fp32, all
 * arithmetic is fp32, sums run in a fixed order: repeated calls give the same
 * bits. */

/* Route `tokens` tokens, logits l [tokens x n_experts]:
 *   p[t,e]   = exp(l[t,e] - max l[t,:]) / sum_e exp(..)         (softmax)
 *   expert   [tokens x k] int32: the experts of the k largest logits, largest
 *            first, equal ones by the lower expert
 *   weight   [tokens x k] fp32: p of those experts, with `normalize` divided
 *            by their sum over the token's k
 *   offsets  [n_experts + 1] int32: the first row of each expert's group, as the
 *            grouped calls read them; counts [n_experts] int32: their lengths, or NULL
 *   position [tokens x k] int32: the row of the token's copy for that expert;
 *            an expert's rows are in the order of their tokens
 *   token    [tokens * k] int32: the token of each row.  Entries behind the
 *            last row (offsets[n_experts]) keep their values.
 * A logit of -infinity or NaN is never chosen.  A token with fewer than k
 * others, or with valid[t] = 0 (padding; valid [tokens] bytes, or NULL), has
 * expert and position -1 and weight 0 in the places that are left.  A NaN
 * or +infinity among the logits of a valid token makes its weights NaN, and the
 * loss (as softmax does).
 * Balance loss (both or neither of slope and loss NULL), over the N tokens that
 * have an expert and C = offsets[n_experts] choices:
 *   slope [n_experts] fp32 = n_experts * counts[e] / (C * N)    (0 if N = 0)
 *   loss  [1] fp32 = sum_e slope[e] * sum_t p[t,e]
 * i.e. n_experts * sum_e (share of choices) * (mean probability): 1 when both
 * are even.  slope is the gradient of loss by each p[t,e] of those tokens
 * (counts do not carry a gradient).
 * workspace: moe_route_workspace_size(tokens, n_experts) bytes, 16-byte aligned. */
size_t moe_route_workspace_size(int64_t tokens, int32_t n_experts);

fp8dl_status moe_route(const void *logits, int32_t dtype, int64_t tokens, int32_t n_experts, int32_t k,
                       const uint8_t *valid, int32_t normalize, int32_t *expert, float *weight,
                       int32_t *position, int32_t *token, int32_t *offsets, int32_t *counts, float *slope,
                       float *loss, void *workspace, size_t workspace_bytes, fp8dl_stream_t stream);

/* Gradient of moe_route's weights and loss by the logits:
 *   dp[t,e] = dloss * slope[e]
 *             + (e chosen at j: dweight[t,j], with `normalize`
 *                (dweight[t,j] - sum_i dweight[t,i] * weight[t,i]) / (sum of the chosen p))
 *   dlogits[t,e] = p[t,e] * (dp[t,e] - sum_e p[t,e] * dp[t,e])        (of `dtype`)
 * expert, weight and slope as moe_route wrote them; dweight [tokens x k] fp32 or
 * NULL (zeros); dloss a device float, or NULL (0; slope may then be NULL).  The row
 * of a token without experts is zeros. */
fp8dl_status moe_route_bwd(const void *logits, int32_t dtype, int64_t tokens, int32_t n_experts, int32_t k,
                           int32_t normalize, const int32_t *expert, const float *weight,
                           const float *dweight, const float *slope, const float *dloss, void *dlogits,
                           fp8dl_stream_t stream);

/* Quantise tokens x [tokens x cols] (bf16 or fp32) in blocks of 128 along each row,
 * once, and put the codes and factors of token t into row position[t,j] of every
 * j: row_q [rows x cols], row_s [ceil(cols/128) x rows], the A operand of
 * the experts' product.  q [tokens x cols] and s [ceil(cols/128) x tokens] receive
 * them in token order too (the checkpoint that fp8_block_recode reads), or NULL.
 * A position outside [0, rows) is skipped; rows without a token keep their
 * values; a row that two positions name holds one of the two tokens or a mixture.
 * 1 <= k <= 32; cols a positive multiple of 16. */
fp8dl_status fp8_block_dispatch(const void *x, int32_t x_dtype, int64_t tokens, int64_t cols, int32_t out_dtype,
                                const int32_t *position, int32_t k, int64_t rows, uint8_t *row_q,
                                float *row_s, uint8_t *q, float *s, fp8dl_stream_t stream);

/* The experts' results back in token order:
 *   out[t,:] = round( sum_j weight[t,j] * y[position[t,j],:] )
 * (fp32, j ascending; fused multiply-adds), over the positions inside [0, rows);
 * zeros for a token without any.  y [rows x cols] and out [tokens x cols] of
 * `dtype` (bf16 or fp32); weight NULL: 1 (the gradient of fp8_block_dispatch's
 * input).  1 <= k <= 32; cols a positive multiple of 16. */
fp8dl_status moe_combine(const void *y, int32_t dtype, int64_t rows, int64_t cols, const int32_t *position,
                         const float *weight, int64_t tokens, int32_t k, void *out, fp8dl_stream_t stream);

/* Gradients of moe_combine, dout [tokens x cols]:
 *   dy[position[t,j],:] = round( weight[t,j] * dout[t,:] )        (of `dtype`)
 *   dweight[t,j] = sum_c dout[t,c] * y[position[t,j],c]           (fp32, a fixed order)
 * dweight is 0 where the position is outside [0, rows); rows of dy without a
 * token keep their values, a row that two positions name holds either's or a
 * mixture.  dy and dweight may each be NULL (y too without
 * dweight, weight too without dy). */
fp8dl_status moe_combine_bwd(const void *dout, const void *y, int32_t dtype, int64_t rows, int64_t cols,
                             const int32_t *position, const float *weight, int64_t tokens, int32_t k,
                             void *dy, float *dweight, fp8dl_stream_t stream);

/* ----------------------------------------------------------------------------
 * Activations kept in 8 bits.  Between two block-scaled products the forward
 * pass quantises the activation's result straight from fp32 and keeps its argument
 * h as row-wise codes (half the bytes of bf16); the backward pass decodes those,
 * and computes from them both the gradient's codes and the activation's transposed
 * codes, which therefore need not be kept.
 *   act        FP8DL_ACT_GELU, FP8DL_ACT_SILU: g = act(h), h [rows x cols]
 *              FP8DL_ACT_GEGLU, FP8DL_ACT_SWIGLU: g = act(a) * u, h = [a | u]
 *              [rows x 2 cols], GELU or SiLU
 *   GELU(a) = a * Phi(a) (erf form), SiLU(a) = a / (1 + exp(-a)), in fp32, relative
 *   errors at most (1.25 a^2 + 23) * 2^-24 (a >= 0: 23) and (1.25 |a| + 9) * 2^-24;
 *   results below 2^-126 keep what bits subnormal numbers have, but for SiLU of
 *   a < -87.3, which is 0.
 * Groups, rows of any number, factors' layouts and the rule of a block's scale as
 * above: offsets/n_groups NULL and 0 for the whole matrix, rows outside the
 * groups are neither read nor written. */
typedef enum {
    FP8DL_ACT_GELU = 0,
    FP8DL_ACT_SILU = 1,
    FP8DL_ACT_GEGLU = 2,
    FP8DL_ACT_SWIGLU = 3
} fp8dl_activation;

/* Forward: g_q [rows x cols], g_s [ceil(cols/128) x rows] codes of g along the rows;
 * h_q, h_s (or both NULL) exactly what fp8_block_quantize gives for h along the
 * rows: h_q [rows x W], h_s [ceil(W/128) x rows], W = cols or 2 cols.  h of
 * h_dtype, both codes of out_dtype. */
fp8dl_status fp8_block_act(const void *h, int32_t h_dtype, int32_t act, int64_t rows, int64_t cols,
                           const int32_t *offsets, int32_t n_groups, int32_t out_dtype, uint8_t *g_q,
                           float *g_s, uint8_t *h_q, float *h_s, fp8dl_stream_t stream);

/* Backward, h = fl32(code * factor) of h_q, h_s (codes of h_fp8):
 *   dh = dg * act'(h), or [dg * u * act'(a) | dg * act(a)];  dg [rows x cols] of dg_dtype
 *   dh_q/dh_s    [rows x W], [ceil(W/128) x rows]: codes of dh along the rows
 *   dh_qt/dh_st  [W x T], [T/128 x W]: transposed, T = fp8_block_padded_rows(rows, n_groups)
 *   g_qt/g_st    [cols x T], [T/128 x cols]: transposed codes (of h_fp8) of
 *                g = act(h) or act(a) * u
 *   dbias        [W] fp32 column sums of dh (fixed order; not with offsets);
 *                workspace of fp8_cast_workspace_size(rows, W) bytes
 * any of them NULL (codes and factors in pairs).  dh's codes are of out_dtype.  Nothing
 * is rounded between the checkpoint's values and the codes but fp32.  Transposed codes
 * and padding as fp8_block_quantize writes them. */
fp8dl_status fp8_block_dact(const void *dg, int32_t dg_dtype, int32_t act, int64_t rows, int64_t cols,
                            const uint8_t *h_q, int32_t h_fp8, const float *h_s, const int32_t *offsets,
                            int32_t n_groups, int32_t out_dtype, uint8_t *dh_q, float *dh_s, uint8_t *dh_qt,
                            float *dh_st, uint8_t *g_qt, float *g_st, float *dbias,
                            void *workspace, size_t workspace_bytes, fp8dl_stream_t stream);

/* Transposed codes from row-wise ones: the values fl32(code * factor) of
 * q [src_rows x cols], s [ceil(cols/128) x src_rows] (codes of q_fp8) quantised
 * in blocks of 128 along the rows into col_q [cols x T], col_s [T/128 x cols] as
 * fp8_block_quantize does.  index [rows] int32: row r is row index[r] of q, zeros
 * if that is outside [0, src_rows); NULL: r itself (rows <= src_rows). */
fp8dl_status fp8_block_recode(const uint8_t *q, int32_t q_fp8, const float *s, int64_t src_rows, int64_t rows,
                              int64_t cols, const int32_t *index, const int32_t *offsets, int32_t n_groups,
                              int32_t out_dtype, uint8_t *col_q, float *col_s, fp8dl_stream_t stream);

/* ----------------------------------------------------------------------------
 * LayerNormMLP pieces.  The Transformer Engine tutorial builds its blocks
 * from te.LayerNormMLP (LayerNorm -> fc1 -> GELU -> fc2), mirrored in plain
 * PyTorch by nn.LayerNorm and nn.GELU (erf form).  Under delayed scaling the
 * scale of each activation's FP8 cast is known before the activation runs
 * ("FP8 低精度训练：Transformer Engine 简析" §三.1), so each activation is fused
 * with the cast of its output (cast semantics as fp8_cast_amax_transpose).
 * All high-precision tensors here are bf16; mu and rsigma are fp32.
 */

/* LayerNorm forward + cast, per row of x [rows x cols] (cols <= 8192):
 *   mu = mean(x), var = mean((x - mu)^2) (biased), rsigma = 1/sqrt(var + eps)
 *   y = bf16((x - mu) * rsigma * gamma + beta)       (fp32 arithmetic)
 *   out = enc(fl32(y * scale)), out_t = out^T, amax max-ed with max |y|
 * gamma, beta [cols] bf16; mu, rsigma [rows] fp32 (for the backward);
 * y [rows x cols] bf16 or NULL; out/out_t/amax nullable as for the cast. */
fp8dl_status fp8_layernorm_cast(const void *x, int64_t rows, int64_t cols, const void *gamma,
                                const void *beta, float eps, int32_t out_dtype, const float *scale,
                                uint8_t *out, uint8_t *out_t, float *amax, float *mu, float *rsigma,
                                void *y, fp8dl_stream_t stream);

/* GELU + cast: g = bf16(0.5 * h * (1 + erf(h / sqrt2))) in fp32 arithmetic, then the
 * cast of g (out, out_t, amax of g).  h [rows x cols] bf16 (the fc1 output);
 * g [rows x cols] bf16 or NULL. */
fp8dl_status fp8_gelu_cast(const void *h, int64_t rows, int64_t cols, int32_t out_dtype,
                           const float *scale, uint8_t *out, uint8_t *out_t, float *amax, void *g,
                           fp8dl_stream_t stream);

/* dGELU + cast: dh = bf16(dg * (0.5 * (1 + erf(h/sqrt2)) + h * exp(-h^2/2) / sqrt(2 pi))),
 * then the cast of dh (E5M2 in HYBRID) with amax, transposed copy and the
 * bias gradient dbias = column sums of dh (workspace as for the cast).
 * dg, h [rows x cols] bf16; dh [rows x cols] bf16 or NULL. */
fp8dl_status fp8_dgelu_cast(const void *dg, const void *h, int64_t rows, int64_t cols, int32_t out_dtype,
                            const float *scale, uint8_t *out, uint8_t *out_t, float *amax, float *dbias,
                            void *workspace, size_t workspace_bytes, void *dh, fp8dl_stream_t stream);

/* LayerNorm backward from the forward's mu and rsigma:
 *   xhat = (x - mu) * rsigma, g = dy * gamma
 *   dx = bf16(rsigma * (g - mean(g) - xhat * mean(g * xhat)))
 *   dgamma = sum_rows dy * xhat, dbeta = sum_rows dy   (fp32 [cols], overwritten)
 * dy, x [rows x cols] bf16, gamma [cols] bf16; workspace of
 * fp8_layernorm_bwd_workspace_size(rows, cols) bytes. */
size_t fp8_layernorm_bwd_workspace_size(int64_t rows, int64_t cols);

fp8dl_status fp8_layernorm_bwd(const void *dy, const void *x, const void *gamma, const float *mu,
                               const float *rsigma, int64_t rows, int64_t cols, void *dx, float *dgamma,
                               float *dbeta, void *workspace, size_t workspace_bytes,
                               fp8dl_stream_t stream);

/* ----------------------------------------------------------------------------
 * Library state. */
/* 1 if `device` is an sm_103 GPU this library can run on, else 0. */
int32_t fp8dl_device_supported(int32_t device);
/* Last error message of the calling thread ("" if none). */
const char *fp8dl_last_error(void);
/* Self-test of failure detection without a GPU fault.  One thread waits,
 * through the same bounded wait the GEMM pipelines use, on a shared-memory
 * barrier phase; if arrive_first is 0 nothing ever completes it, the wait
 * gives up after budget_cycles SM clock cycles (<= 2^32), writes
 * FP8DL_ERR_TIMEOUT into *dev_status and the kernel returns; with
 * arrive_first = 1 the phase completes and *dev_status is set to FP8DL_OK.
 * The CUDA context stays usable either way. */
fp8dl_status fp8dl_wait_selftest(int64_t budget_cycles, int32_t arrive_first, int32_t *dev_status,
                                 fp8dl_stream_t stream);
/* Clock probe (measurement): n_ctas CTAs each write, to out[3 * i .. 3 * i + 2]
 * (device memory, 16-byte aligned, 3 * n_ctas uint64), the id of the SM CTA i
 * ran on, that SM's cycle counter (clock64) and the global nanosecond timer
 * (%globaltimer), read back to back.  Two probes on a stream around some work
 * give each SM's mean clock over it: (cycles_2 - cycles_1) / (ns_2 - ns_1) GHz
 * for an SM seen in both.  One launch; no other effect. */
fp8dl_status fp8dl_clock_probe(uint64_t *out, int32_t n_ctas, fp8dl_stream_t stream);
/* Library version, major*10000 + minor*100 + patch. */
int32_t fp8dl_version(void);
/* Number of kernels this library has enqueued in this process, over all threads
 * and devices (launches that failed are not counted).  A CUDA graph replay
 * launches its captured kernels without calling the library, so it does not
 * count: count one eager step to know what a replayed step launches. */
uint64_t fp8dl_kernel_launches(void);

/* ----------------------------------------------------------------------------
 * Environment switches (testing and diagnosis).  They choose which kernel, tile
 * order or grid runs.  The GEMM switches leave every output bit unchanged,
 * except in a GEMM with K > 8192 and two or more waves of tiles, where they
 * can change which tiles sum K last to first (within the GEMM's error bound;
 * the one-CTA kernel always sums first to last).  The LayerNorm ones can
 * change the rounding of the row statistics and of dgamma / dbeta, within the
 * tolerances the tests state.
 *   FP8DL_DEBUG=1               print every launch and error message to stderr
 *                               (read once per process)
 *   FP8DL_GEMM_VARIANT=1sm|2sm  force the one-CTA or the CTA-pair FP8 GEMM
 *   FP8DL_GEMM_RASTER=m|n       group the GEMM tiles along rows (m) or columns (n)
 *   FP8DL_GEMM_GROUP=g          tiles per group (g > 0)
 *   FP8DL_GEMM_TILE_N=256|128   tile width of the plain pair GEMM (by default 128
 *                               only for a short GEMM with under two waves of
 *                               256-column tiles)
 *   FP8DL_GEMM_SNAKE=0          every GEMM tile sums K first to last
 *   FP8DL_LN_VARIANT=tiles      LayerNorm by the two-pass tile kernels
 *   FP8DL_LN_CLUSTERS=n         cap on the clusters of the LayerNorm cluster kernels
 *   FP8DL_PDL=0                 launch without programmatic dependent launch: every
 *                               kernel then starts only after the previous kernel of
 *                               its stream has finished (read once per process)
 * All but FP8DL_DEBUG and FP8DL_PDL are read at each call.
 *
 * Launch order.  The kernels of a short call (under 64 MB moved or 64 GFLOP)
 * are launched with the programmatic stream serialization attribute: such a
 * kernel may be scheduled while the previous kernel of the stream is still
 * running, does only its own set-up (shared-memory barriers, tensor-memory
 * allocation, descriptor prefetch), and waits for that kernel to complete
 * before its first access to global memory.  Every kernel makes that wait, so
 * stream order and results are those of ordinary launches. */

#ifdef __cplusplus
}
#endif
#endif /* FP8DL_H */
