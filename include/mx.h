/*
 * mx.h -- C ABI of the MXFP4 (OCP Microscaling) training hot path for AMD
 * MI355X (gfx950): block quantizer, MXFP4 GEMMs, quantized linear layer and
 * the post-step weight de-oscillation pass.
 *
 * The operations follow these pages:
 *  [TJ]   "Oscillation-Reduced MXFP4 Training for Vision Transformers"
 *         (rebuttal, Question 2: Y = Q_D(X) Q_D(W^T), the STE weight gradient,
 *         1x32 / 32x1 group shapes and the double quantization Q_S(Q_D(X))).
 *  [ALTO] "ALTO MXFP4 training -- Weight de-oscillation -- What does it mean?"
 *         (Jargon: MXFP4, E2M1, Bin, RHT, Stochastic rounding; the ratio
 *         paragraph: window of 200 steps, d_w, d_Q, threshold 4.0, snap to
 *         the current bin centre, post-step hook).
 *  [OAS]  "Unveiling the Potential of Quantization with MXFP4" (abstract:
 *         power-of-two block scale).
 *  [MRG]  "Microscaling FP4 Quantization: MR-GPTQ ..." (section "FP4
 *         Quantization with Micro-Rotated GPTQ Algorithm": block-wise Hadamard).
 * Conventions the pages leave open follow the OCP MX v1.0 specification
 * (E2M1 values {0, .5, 1, 1.5, 2, 3, 4, 6}; shared exponent
 * floor(log2 amax) - 2 stored as an E8M0 byte with bias 127; values above 6
 * saturate to 6).
 *
 * Data layout
 *  - A "packed MXFP4 matrix" with B-element blocks along its last axis is two
 *    dense row-major arrays: codes [outer][inner/2] (element 2j in the low
 *    nibble of byte j, bit 3 = sign, bits 0-2 = index of the magnitude) and
 *    scales [outer][inner/32] (E8M0: value 2^(byte-127), 0xFF = NaN).
 *  - MX_ROW quantizes 1x32 blocks along the columns of a [rows, cols] input:
 *    codes [rows][cols/2], scales [rows][cols/32].
 *  - MX_COL quantizes 32x1 blocks along the rows and stores the result
 *    transposed: codes [cols][rows/2], scales [cols][rows/32].  So every GEMM
 *    operand is contiguous along its contraction axis.
 *  - Stochastic rounding rounds an element up iff floor(t * 2^22) + r22 >= 2^22,
 *    with t in [0, 1) the relative distance to the lower neighbour.  The
 *    elements 2i and 2i+1 of a block share output idx+1 of SplitMix64 started
 *    from `seed` (Steele, Lea & Flood, OOPSLA 2014), idx the logical row-major
 *    index of element 2i in the input: element 2i takes bits 42..63 as r22,
 *    element 2i+1 bits 9..30.  The result does not depend on tiling or launch
 *    shape.
 *
 * Ownership and execution
 *  - Every pointer argument is a DEVICE pointer owned by the caller, except
 *    `offs` of the grouped calls (host; mx_gemv_grouped takes device offsets).  The library never allocates, frees or
 *    synchronizes; it keeps no state between calls, so every entry point is
 *    reentrant.  Work is enqueued on `stream` (a hipStream_t; NULL = default
 *    stream) and the call returns before it runs.
 *  - Input and output buffers must not overlap unless stated.  A workspace is in use
 *    until the call's work has run: calls that share one must be ordered (one stream,
 *    or captured graphs that are never replayed at the same time).
 *
 * Errors
 *  - Every entry point returns an mx_status.  Arguments are validated before
 *    any launch; on a validation error nothing is written and nothing is
 *    enqueued.  MX_ERR_HIP reports a failed launch (the stream may then hold
 *    earlier work of the same call).
 *  - Base pointers of device arrays must be 16-byte aligned (MX_ERR_ALIGN).
 */
#ifndef MX355_MX_H
#define MX355_MX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MX_OK = 0,
  MX_ERR_NULL = 1,      /* a required pointer is NULL */
  MX_ERR_SHAPE = 2,     /* a size is negative, a block axis is not a multiple of 32, ... */
  MX_ERR_ALIGN = 3,     /* a device pointer is not 16-byte aligned */
  MX_ERR_ENUM = 4,      /* dtype / axis / rounding / flag out of range */
  MX_ERR_WORKSPACE = 5, /* workspace NULL or smaller than required */
  MX_ERR_HIP = 6        /* the HIP runtime rejected a launch */
} mx_status;

enum { MX_F32 = 0, MX_BF16 = 1 };   /* element types of unquantized tensors */
enum { MX_ROW = 0, MX_COL = 1 };    /* 1x32 blocks along cols / 32x1 blocks along rows */
enum { MX_RNE = 0, MX_SR = 1 };     /* Q_D: nearest, ties to even / Q_S: stochastic */
enum { MX_I32 = 0, MX_I64 = 1 };    /* types of expert ids */
enum { MX_SILU = 0, MX_GELU = 1 };  /* activations of mx_glu: g / (1 + e^-g), g Phi(g) */

/* Largest number of groups mx_gemm_grouped accepts. */
#define MX_MAX_GROUPS 128

/* Human-readable name of a status code (static string). */
const char* mx_status_string(int status);

/* ------------------------------------------------------------------ quantizer
 * mx_quantize: MXFP4-quantize a [rows, cols] row-major tensor x (dtype MX_F32
 * or MX_BF16) -- [ALTO] Jargon "MXFP4", "E2M1", "Bin", "Stochastic rounding";
 * [TJ] Question 2 for the two group shapes.
 *  For each block of 32 values v (after the optional rotation):
 *    e = clamp(floor(log2 max|v|) - 2, -127, 127) (e = -127 for an all-zero
 *    block), scale byte = e + 127; a_i = |v_i| 2^-e; the magnitude is the
 *    nearest of {0,.5,1,1.5,2,3,4,6} with ties to the even code (MX_RNE) or
 *    one of the two neighbours chosen by stochastic rounding (MX_SR); a_i > 6
 *    gives 6; the sign bit is the sign bit of v_i (so -0 codes as 0x8).
 *    A block holding NaN or Inf gets scale byte 0xFF and zero codes.
 *  axis MX_ROW: cols % 32 == 0; writes codes [rows][cols/2], scales [rows][cols/32].
 *  axis MX_COL: rows % 32 == 0 and cols % 8 == 0; writes codes [cols][rows/2],
 *       scales [cols][rows/32] (transposed).
 *  hadamard != 0: each block is first rotated, v = H32 (s . x), H32 the
 *    unnormalised Sylvester Hadamard matrix (H H^T = 32 I) and s_j = -1 where
 *    bit j of sign_mask is set -- [ALTO] Jargon "Randomized Hadamard transform",
 *    [MRG] block-wise Hadamard.  Computed in float32 with butterfly stages
 *    h = 1, 2, 4, 8, 16.
 *  seed is used only by MX_SR.  rows or cols == 0 is a no-op.
 */
int mx_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int axis, int round,
                uint64_t seed, int hadamard, uint32_t sign_mask,
                uint8_t* codes, uint8_t* scales, void* stream);

/* mx_quantize_ld: mx_quantize with the output's scale rows scale_ld bytes apart
 * (scale row r starts at scales + r * scale_ld; scale_ld >= the blocks per
 * output row, cols/32 for MX_ROW, rows/32 for MX_COL, else MX_ERR_SHAPE).  The
 * bytes of a scale row past its blocks are not written.  Codes are packed as
 * for mx_quantize.  Scale rows padded to a multiple of 16 bytes let the GEMMs
 * load the scales of four K-steps of a row at once (mx_gemm_ld,
 * mx_gemm_grouped_ld). */
int mx_quantize_ld(const void* x, int dtype, int64_t rows, int64_t cols, int axis, int round,
                   uint64_t seed, int hadamard, uint32_t sign_mask,
                   uint8_t* codes, uint8_t* scales, int64_t scale_ld, void* stream);

/* mx_quantize_dual: one read of a [rows, cols] tensor, two quantizations:
 * a MX_ROW one (codes_row [rows][cols/2], scales_row [rows][cols/32], seed
 * seed_row) and a MX_COL one (codes_col [cols][rows/2], scales_col
 * [cols][rows/32], seed seed_col), both with rounding `round`.  Equal,
 * bit for bit, to two mx_quantize calls.  This is the gradient dY of the
 * backward pass, which both backward GEMMs consume in different group
 * shapes ([TJ] Question 2 (2)).  rows % 32 == 0, cols % 32 == 0. */
int mx_quantize_dual(const void* x, int dtype, int64_t rows, int64_t cols, int round,
                     uint64_t seed_row, uint64_t seed_col,
                     uint8_t* codes_row, uint8_t* scales_row,
                     uint8_t* codes_col, uint8_t* scales_col, void* stream);

/* mx_quantize_pair: two MX_ROW quantizations in one launch -- the forward
 * layer's two operands Q_D(X) and Q_D(W) ([TJ] Question 2 (1): both 1x32 along
 * the contraction axis).  x0 [rows0, cols] and x1 [rows1, cols] (same dtype,
 * rounding, rotation and sign_mask) are quantized exactly as two mx_quantize
 * calls with axis MX_ROW and seeds seed0 / seed1 would (each tensor's
 * stochastic-rounding index starts at 0), writing codes0 [rows0][cols/2],
 * scales0 [rows0][cols/32] and codes1 / scales1 likewise.  cols % 32 == 0; a
 * tensor with 0 rows is skipped (its pointers may then be NULL). */
int mx_quantize_pair(const void* x0, int64_t rows0, const void* x1, int64_t rows1, int64_t cols,
                     int dtype, int round, uint64_t seed0, uint64_t seed1, int hadamard,
                     uint32_t sign_mask, uint8_t* codes0, uint8_t* scales0,
                     uint8_t* codes1, uint8_t* scales1, void* stream);

/* mx_quantize_dual_rht: mx_quantize_dual with the random-sign block Hadamard
 * ([ALTO] Jargon "Randomized Hadamard transform"; the "MXFP4 + RHT +
 * stochastic rounding" rows of its steps table) on both outputs: each row
 * block and each column block is rotated, y = H32 (s . x) with s from
 * sign_mask (bit j set: element j of the block negated), before it is
 * quantized -- equal, bit for bit, to two mx_quantize calls with hadamard = 1.
 * Arguments otherwise as mx_quantize_dual. */
int mx_quantize_dual_rht(const void* x, int dtype, int64_t rows, int64_t cols, int round,
                         uint64_t seed_row, uint64_t seed_col, uint32_t sign_mask,
                         uint8_t* codes_row, uint8_t* scales_row,
                         uint8_t* codes_col, uint8_t* scales_col, void* stream);

/* mx_requantize: double quantization Q(Q_D(X)) -- [TJ] Question 2 (2), the
 * double-quantized operand Q_S^(6)(Q_D^(1)(X)).  Input: a packed MX_ROW matrix
 * of logical shape [rows, cols] (codes_in [rows][cols/2], scales_in
 * [rows][cols/32]).  Its exact values are quantized again with 32x1 blocks
 * (MX_COL, output transposed: codes_out [cols][rows/2], scales_out
 * [cols][rows/32]) with rounding `round` and `seed`; the stochastic-rounding
 * index is the logical row-major index in [rows, cols].  Equal to
 * mx_quantize(dequantized input, MX_COL, ...).  rows % 32 == 0, cols % 32 == 0. */
int mx_requantize(const uint8_t* codes_in, const uint8_t* scales_in, int64_t rows, int64_t cols,
                  int round, uint64_t seed, uint8_t* codes_out, uint8_t* scales_out, void* stream);

/* mx_requantize_pair: two double quantizations in one launch -- the backward
 * layer's Q_S^(4)(Q_D(W)) and Q_S^(6)(Q_D(X)) ([TJ] Question 2 (2)).  The
 * packed MX_ROW inputs [rows0, cols] and [rows1, cols] are requantized exactly
 * as two mx_requantize calls with seeds seed0 / seed1 would, outputs transposed
 * (codes_out0 [cols][rows0/2], scales_out0 [cols][rows0/32], and likewise for
 * input 1).  rows0, rows1, cols multiples of 32; an input with 0 rows is skipped
 * (its pointers may then be NULL). */
int mx_requantize_pair(const uint8_t* codes_in0, const uint8_t* scales_in0, int64_t rows0,
                       const uint8_t* codes_in1, const uint8_t* scales_in1, int64_t rows1,
                       int64_t cols, int round, uint64_t seed0, uint64_t seed1,
                       uint8_t* codes_out0, uint8_t* scales_out0,
                       uint8_t* codes_out1, uint8_t* scales_out1, void* stream);

/* mx_requantize_rht: double quantization of an operand kept in the rotated
 * domain (the rotated layer's saved Q_D(H X), rotated along cols with
 * sign_mask): the input's row blocks are decoded and rotated back exactly as
 * mx_dequantize with hadamard = 1 does it (float32), then each 32x1 column
 * block is rotated with the same signs and quantized (output transposed, as
 * mx_requantize; the stochastic-rounding index is the logical row-major index
 * of the rotated position).  Equal to mx_quantize(mx_dequantize(in, MX_ROW,
 * hadamard = 1), MX_COL, hadamard = 1).  rows % 32 == 0, cols % 32 == 0. */
int mx_requantize_rht(const uint8_t* codes_in, const uint8_t* scales_in, int64_t rows,
                      int64_t cols, int round, uint64_t seed, uint32_t sign_mask,
                      uint8_t* codes_out, uint8_t* scales_out, void* stream);

/* mx_dequantize: exact values of a packed matrix -- [ALTO] Jargon "MXFP4" (each
 * block of 32 values shares one power-of-two scale, and an element's value is
 * its 4-bit E2M1 number times that scale) and "E2M1"; it is the deq(.) inside
 * every product of [TJ] Question 2 and the bin value q(w) of the
 * de-oscillation pass.  Input: a packed matrix of logical shape [rows, cols]
 * quantized along `axis` (the inverse layout of mx_quantize), written row-major
 * [rows, cols] as float32 or bf16 (out_dtype).  value = sign * E2M1[code & 7]
 * * 2^(byte - 127) (exact in both types), byte 0xFF gives NaN.  hadamard != 0
 * undoes the rotation: x = s . (H32 y) 2^-5 per block in float32 (bf16 output
 * then rounds to nearest even).  rows (MX_COL) or cols (MX_ROW) % 32 == 0;
 * rows or cols == 0 is a no-op.  Errors as for mx_quantize. */
int mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                  int axis, int hadamard, uint32_t sign_mask, void* out, int out_dtype,
                  void* stream);

/* ------------------------------------------------------------------ GEMM
 * mx_gemm: C[m][n] = alpha * sum_k deq(A)[m][k] * deq(B)[n][k]  -- the MXFP4
 * matrix product of [TJ] Question 2 (1), (1x32) x (32x1) groups.
 *  A: packed MX_ROW [M, K] (a_codes [M][K/2], a_scales [M][K/32]);
 *  B: packed MX_ROW [N, K] (b_codes [N][K/2], b_scales [N][K/32]);
 *  C: float32 row-major, leading dimension ldc >= N (ldc % 4 == 0), overwritten.
 *  K % 32 == 0; M, N >= 0 (M or N == 0: no-op; K == 0: C = 0); M, N <= 2^31 and
 *  K < 2^31, else MX_ERR_SHAPE (the same bounds hold for every GEMM call below).
 *  Products of FP4 values and E8M0 scales are exact; sums are float32 in an
 *  unspecified order (error <= ~K/64 * 2^-24 * sum |a b|). */
int mx_gemm(const uint8_t* a_codes, const uint8_t* a_scales,
            const uint8_t* b_codes, const uint8_t* b_scales,
            int64_t M, int64_t N, int64_t K, float alpha, float* c, int64_t ldc, void* stream);

/* mx_gemm_grouped: per-group products for a mixture-of-experts layer ([ALTO]
 * news paragraph: the MoE model trained in MXFP4).  offs is a HOST array of
 * groups+1 non-decreasing row offsets with offs[0] == 0; rows
 * offs[g] .. offs[g+1]-1 of A and C use B_g, the g-th [N, K] matrix of b
 * (b_codes + g*N*K/2, b_scales + g*N*K/32).  C is [offs[groups]][N], ldc = N.
 * 1 <= groups <= MX_MAX_GROUPS, K % 32 == 0, N % 4 == 0. */
int mx_gemm_grouped(const uint8_t* a_codes, const uint8_t* a_scales,
                    const uint8_t* b_codes, const uint8_t* b_scales,
                    const int64_t* offs, int64_t groups, int64_t N, int64_t K, float alpha,
                    float* c, void* stream);

/* mx_gemm_ld / mx_gemm_grouped_ld: mx_gemm / mx_gemm_grouped with the scale
 * rows of A and of B a_scale_ld and b_scale_ld bytes apart (each >= K/32, else
 * MX_ERR_SHAPE; the bytes past K/32 in a row are never used as data); for the
 * grouped form, B_g's scales start at b_scales + g*N*b_scale_ld.  Codes are
 * packed as for mx_gemm.  Same results, bit for bit, as the packed calls on the
 * same values; pitches that are multiples of 16 (with 16-byte aligned scale
 * arrays) take the fastest scale loads whatever K is. */
int mx_gemm_ld(const uint8_t* a_codes, const uint8_t* a_scales, int64_t a_scale_ld,
               const uint8_t* b_codes, const uint8_t* b_scales, int64_t b_scale_ld,
               int64_t M, int64_t N, int64_t K, float alpha, float* c, int64_t ldc,
               void* stream);
int mx_gemm_grouped_ld(const uint8_t* a_codes, const uint8_t* a_scales, int64_t a_scale_ld,
                       const uint8_t* b_codes, const uint8_t* b_scales, int64_t b_scale_ld,
                       const int64_t* offs, int64_t groups, int64_t N, int64_t K, float alpha,
                       float* c, void* stream);

/* ------------------------------------------------------------------ token segments
 * The 32x1 quantizers of a grouped (mixture-of-experts) layer run per token
 * segment: segment g is rows offs[g] .. offs[g+1]-1 (offs: HOST array of
 * groups+1 non-decreasing offsets, offs[0] == 0, offs[groups] == rows, 1 <=
 * groups <= MX_MAX_GROUPS).  Blocks start at the segment's first row; the
 * segment's tail is zero-padded to a multiple of 128 rows, so the transposed
 * outputs have a padded row axis of P = mx_segments_padded_rows(offs, groups)
 * positions, segment g's starting at the sum of the padded lengths before it.
 * Padding blocks hold code 0 and scale byte 0.  The stochastic-rounding index
 * of a real element is its row-major index in [rows, cols]. */
int64_t mx_segments_padded_rows(const int64_t* offs, int64_t groups);

/* mx_quantize_segments: 32x1 blocks of x [rows, cols] (`dtype`) per segment:
 * codes [cols][P/2], scales [cols][P/32].  cols % 8 == 0. */
int mx_quantize_segments(const void* x, int dtype, int64_t rows, int64_t cols,
                         const int64_t* offs, int64_t groups, int round, uint64_t seed,
                         uint8_t* codes, uint8_t* scales, void* stream);

/* mx_requantize_segments: mx_requantize per segment -- the exact values of a
 * packed MX_ROW [rows, cols] matrix quantized with 32x1 blocks per segment:
 * codes_out [cols][P/2], scales_out [cols][P/32].  cols % 32 == 0. */
int mx_requantize_segments(const uint8_t* codes_in, const uint8_t* scales_in, int64_t rows,
                           int64_t cols, const int64_t* offs, int64_t groups, int round,
                           uint64_t seed, uint8_t* codes_out, uint8_t* scales_out, void* stream);

/* ------------------------------------------------------------------ linear layer
 * mx_linear_fwd: forward of the quantized linear layer, Y = Q_D(X) Q_D(W)^T
 * ([TJ] Question 2 (1)); X [M, K], W [N, K] (nn.Linear layout), both `dtype`;
 * Q_D is MX_ROW + MX_RNE along K.  Writes y [M][N] float32 and the packed
 * operands kept for the backward pass: xq_codes [M][K/2], xq_scales [M][K/32],
 * wq_codes [N][K/2], wq_scales [N][K/32].  M, N, K multiples of 32 and below 2^31,
 * N % 4 == 0 (else MX_ERR_SHAPE, before any launch).  M or N == 0: no-op;
 * K == 0: Y = 0 and nothing else is read or written (x, w and the packed
 * operands may then be NULL). */
int mx_linear_fwd(const void* x, const void* w, int dtype, int64_t M, int64_t N, int64_t K,
                  float* y, uint8_t* xq_codes, uint8_t* xq_scales,
                  uint8_t* wq_codes, uint8_t* wq_scales, void* stream);

/* Bytes of device workspace mx_linear_bwd needs for these sizes. */
size_t mx_linear_bwd_workspace_size(int64_t M, int64_t N, int64_t K);

/* mx_linear_bwd: backward of the quantized linear layer with straight-through
 * gradients ([TJ] Question 2 (1) and (2)):
 *   dX = Q_S^(3)(dY) . Q_S^(4)(Q_D(W))       contraction over N
 *   dW = Q_S^(5)(dY)^T . Q_S^(6)(Q_D(X))     contraction over M
 * Q^(3): dY 1x32 along N; Q^(5): dY 32x1 along M; Q^(4), Q^(6): double
 * quantization of the saved forward operands with 32x1 blocks along N and M.
 * Stochastic rounding; quantizer q uses seed + q.  dy [M][N] (`dtype`);
 * the saved operands are mx_linear_fwd's outputs; writes dx [M][K] and
 * dw [N][K] float32.  workspace: device buffer of at least
 * mx_linear_bwd_workspace_size(M, N, K) bytes, 16-byte aligned.
 * M, N, K multiples of 32 and below 2^31, K % 4 == 0.  K == 0: no-op.  M == 0 or
 * N == 0 (an empty contraction for one of the products): dx = 0 and dw = 0 are
 * written and nothing else is read (only dx, when M > 0, and dw, when N > 0,
 * are required). */
int mx_linear_bwd(const void* dy, int dtype, int64_t M, int64_t N, int64_t K,
                  const uint8_t* xq_codes, const uint8_t* xq_scales,
                  const uint8_t* wq_codes, const uint8_t* wq_scales,
                  uint64_t seed, float* dx, float* dw,
                  void* workspace, size_t workspace_bytes, void* stream);

/* mx_linear_bwd_noalloc: mx_linear_bwd for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): no workspace argument and no allocation of any kind; the
 * workspace is a file-scope device array of mx_linear_bwd_noalloc_max_workspace()
 * bytes (64 MiB) that each GPU the library runs on holds from library load until
 * the process ends.  Layers whose workspace (mx_linear_bwd_workspace_size) is
 * larger are rejected with MX_ERR_WORKSPACE before anything is enqueued (the
 * DeiT-S MLP layers need 36-43 MiB; the Llama-3-8B up-projection needs 166 MiB
 * and must use mx_linear_bwd).  Every call on one GPU shares that GPU's array,
 * so calls that may overlap on one GPU (on different streams, or from different
 * threads without ordering) race and give wrong results; calls on one stream are
 * ordered and safe.  Nothing in the array needs to start at zero.  The first call
 * on a device looks up the array's device address (MX_ERR_HIP if the runtime
 * cannot give it).  Arguments, results and other errors as mx_linear_bwd, bit
 * for bit. */
int mx_linear_bwd_noalloc(const void* dy, int dtype, int64_t M, int64_t N, int64_t K,
                          const uint8_t* xq_codes, const uint8_t* xq_scales,
                          const uint8_t* wq_codes, const uint8_t* wq_scales,
                          uint64_t seed, float* dx, float* dw, void* stream);
size_t mx_linear_bwd_noalloc_max_workspace(void);

/* mx_linear_fwd_rht / mx_linear_bwd_rht: the same layer with the random-sign
 * block Hadamard on every product ([ALTO] Jargon "Randomized Hadamard
 * transform", the "MXFP4 + RHT + stochastic rounding" rows of its steps
 * table): both operands of a product are rotated along that product's
 * contraction axis with the same signs (sign_mask), and since H H^T = 32 I the
 * product is scaled by alpha = 2^-5 (exact):
 *   Y  = 2^-5 Q_D(H_K X) Q_D(H_K W)^T
 *   dX = 2^-5 Q_S^(3)(H_N dY) . Q_S^(4)(H_N W~)      W~ = H_K^-1 deq(Q_D(H_K W))
 *   dW = 2^-5 Q_S^(5)(H_M dY)^T . Q_S^(6)(H_M X~)    X~ = H_K^-1 deq(Q_D(H_K X))
 * The saved operands (xq, wq) are in the K-rotated domain; the backward takes
 * them back before its own rotations (mx_requantize_rht).  Arguments, layouts,
 * seeds (seed + q), workspace (mx_linear_bwd_workspace_size) and errors as
 * mx_linear_fwd / mx_linear_bwd. */
int mx_linear_fwd_rht(const void* x, const void* w, int dtype, int64_t M, int64_t N, int64_t K,
                      uint32_t sign_mask, float* y, uint8_t* xq_codes, uint8_t* xq_scales,
                      uint8_t* wq_codes, uint8_t* wq_scales, void* stream);
int mx_linear_bwd_rht(const void* dy, int dtype, int64_t M, int64_t N, int64_t K,
                      const uint8_t* xq_codes, const uint8_t* xq_scales,
                      const uint8_t* wq_codes, const uint8_t* wq_scales,
                      uint64_t seed, uint32_t sign_mask, float* dx, float* dw,
                      void* workspace, size_t workspace_bytes, void* stream);

/* mx_grouped_linear_bwd: backward of a grouped (mixture-of-experts) linear
 * layer whose forward is mx_gemm_grouped(Q_D(X), Q_D(W)) ([ALTO] news
 * paragraph: the MoE model trained in MXFP4; the group shapes and double
 * quantization of [TJ] Question 2, per expert):
 *   dX[rows of e] = Q_S^(3)(dY)[rows of e] . Q_S^(4)(Q_D(W_e))  contraction over N
 *   dW_e          = Q_S^(5)(dY_e)^T . Q_S^(6)(Q_D(X_e))        contraction over e's tokens
 * Q^(3): 1x32 along N; Q^(4): 32x1 along N of each expert's [N, K] weight (the
 * index is that of the stacked [groups*N, K] weight); Q^(5), Q^(6): 32x1 along
 * the tokens of each expert (token segments, zero-padded tails).  Stochastic
 * rounding, quantizer q uses seed + q.  dy [R][N] (`dtype`, R = offs[groups]);
 * xq: Q_D(X) [R][K/2] + [R][K/32]; wq: the stacked Q_D(W) [groups*N][K/2] +
 * [groups*N][K/32].  Writes dx [R][K] and dw [groups][N][K] float32 (an expert
 * without tokens gets dW_e = 0).  N, K multiples of 32 and below 2^31, and the
 * workspace's token axis (each expert's tokens padded to a multiple of 512) below
 * 2^31 (else MX_ERR_SHAPE).  workspace: at least
 * mx_grouped_linear_bwd_workspace_size(offs, groups, N, K) bytes, 16-byte
 * aligned. */
size_t mx_grouped_linear_bwd_workspace_size(const int64_t* offs, int64_t groups, int64_t N,
                                            int64_t K);
int mx_grouped_linear_bwd(const void* dy, int dtype, const int64_t* offs, int64_t groups,
                          int64_t N, int64_t K, const uint8_t* xq_codes, const uint8_t* xq_scales,
                          const uint8_t* wq_codes, const uint8_t* wq_scales, uint64_t seed,
                          float* dx, float* dw, void* workspace, size_t workspace_bytes,
                          void* stream);

/* ------------------------------------------------------------------ few rows
 * mx_gemv: y[m][n] = alpha * sum_k x[m][k] * deq(W)[n][k] -- unquantized rows x
 * (x_dtype MX_F32 or MX_BF16, rows ldx >= K elements apart) times a packed MX_ROW
 * weight [N, K] (w_codes [N][K/2]; scale rows w_scale_ld >= K/32 bytes apart, as
 * mx_quantize_ld writes them): the product of a layer whose weights stay packed
 * while a few tokens are decoded.  y (y_dtype) has rows ldy >= N elements apart.
 * Any M, N >= 0 below 2^31 (M or N == 0: no-op), K % 32 == 0, K and w_scale_ld
 * below 2^26 (K == 0: y = 0, x and the weights may be NULL).  The weights are read
 * once per 16 rows of a bf16 x and per 4 of a float32 x.  x is used to its full
 * precision (a float32 x down to bits of 2^-133): products are exact, sums are float32
 * in a fixed order, and one rounding to nearest even gives a bf16 y.  A weight block
 * with scale byte 0xFF makes its sums NaN; sums over values past the float32 range
 * (scale bytes 253 and 254, which no quantizer writes) are not finite.  workspace: at
 * least mx_gemv_workspace_size bytes (the partial sums of a long contraction, up to
 * 256 MiB; 0: may be NULL), 16-byte aligned. */
size_t mx_gemv_workspace_size(int x_dtype, int64_t M, int64_t N, int64_t K);
int mx_gemv(const void* x, int x_dtype, int64_t ldx, const uint8_t* w_codes,
            const uint8_t* w_scales, int64_t w_scale_ld, int64_t M, int64_t N, int64_t K,
            float alpha, void* y, int y_dtype, int64_t ldy, void* workspace,
            size_t workspace_bytes, void* stream);

/* mx_gemv_grouped: mx_gemv per expert, without the host: offs is a DEVICE array of
 * groups+1 non-decreasing row offsets (mx_moe_plan's), offs[0] == 0.  Rows
 * offs[g] .. offs[g+1]-1 of y use W_g, the g-th [N, K] matrix (w_codes + g*N*K/2,
 * w_scales + g*N*w_scale_ld).  Row r takes row src[r] / top_k of x [x_rows, K]
 * (src: mx_moe_plan's slots, so that is the row's token), or row r where src is
 * NULL.  rows bounds offs[groups] and is the number of rows y and src have room
 * for; rows of y from offs[groups] on, and rows whose source is outside x, are left
 * as they were.  1 <= groups <= MX_MAX_GROUPS, top_k >= 1; N, K, alpha, strides
 * and types as mx_gemv. */
int mx_gemv_grouped(const void* x, int x_dtype, int64_t ldx, int64_t x_rows, const int32_t* src,
                    int64_t top_k, const uint8_t* w_codes, const uint8_t* w_scales,
                    int64_t w_scale_ld, const int64_t* offs, int64_t groups, int64_t rows,
                    int64_t N, int64_t K, float alpha, void* y, int y_dtype, int64_t ldy,
                    void* stream);

/* ------------------------------------------------------------------ 8-bit matrices
 * For layers that four bits are too coarse for, and for what is kept for a backward pass.
 * An 8-bit matrix of logical shape [rows, cols] is codes [rows][ld] (OCP E4M3: sign, four
 * exponent bits of bias 7, three mantissa bits, largest value 448) and scales
 * [rows][scale_ld] (E8M0), one byte per 128 columns; the last block of a row may be
 * shorter.  ld >= cols rounded up to a multiple of 16, ld % 16 == 0, ld <= 2^23; the bytes
 * from cols up to that multiple are 0.  scale_ld >= 4 ceil(cols / 512), scale_ld % 4 == 0,
 * scale_ld <= 2^23; the quantizers fill the last dword of a row with 0.  Any rows and cols.
 * A block's scale is the smallest 2^e, e >= -127, with max|v| <= 448 2^e (e = -127 for a
 * block of zeros); an element's code is the E4M3 value nearest to v 2^-e, ties to even, with
 * v's sign.  A block holding NaN or Inf gets scale byte 0xFF and zero codes.  Blocks are
 *   1x128 along the columns (MX_ROW: activations, gradients),
 *   128x1 along the rows, stored transposed as a [cols, rows] matrix (MX_COL), or
 *   128x128 (tile: weights; each row of a tile holds the tile's byte), so that a product and
 *   its transpose see the same values.
 * The rules for NULL, empty sizes, alignment and errors are those of the calls above.
 *
 * mx_quantize8: x [rows][cols] (`dtype`, rows ldx >= cols elements apart) along `axis`. */
int mx_quantize8(const void* x, int dtype, int64_t ldx, int64_t rows, int64_t cols, int axis,
                 uint8_t* codes, int64_t ld, uint8_t* scales, int64_t scale_ld, void* stream);

/* mx_quantize8_dual: both layouts from one read of x: codes / scales [rows, cols] and
 * codes_t / scales_t [cols, rows].  tile == 0: 1x128 and 128x1 blocks, equal bit for bit to
 * two mx_quantize8 calls (a gradient that both backward products take).  tile == 1: 128x128
 * blocks, the same values in both layouts (a weight); codes_t and scales_t may then both be
 * NULL (a weight that is not trained). */
int mx_quantize8_dual(const void* x, int dtype, int64_t ldx, int64_t rows, int64_t cols, int tile,
                      uint8_t* codes, int64_t ld, uint8_t* scales, int64_t scale_ld,
                      uint8_t* codes_t, int64_t ld_t, uint8_t* scales_t, int64_t scale_ld_t,
                      void* stream);

/* mx_requantize8: double quantization: the values of an 8-bit matrix [rows, cols] quantized
 * with 128x1 blocks, transposed -- equal to mx_quantize8(MX_COL) of its float32 values
 * (values past the float32 range, which a block of float32 values near it can round to,
 * count as infinite). */
int mx_requantize8(const uint8_t* codes, int64_t ld, const uint8_t* scales, int64_t scale_ld,
                   int64_t rows, int64_t cols, uint8_t* codes_t, int64_t ld_t, uint8_t* scales_t,
                   int64_t scale_ld_t, void* stream);

/* mx_dequantize8: float32 values (exact; rounded to nearest even for a bf16 out) of an 8-bit
 * matrix, out rows ldo >= cols elements apart; a block with scale byte 0xFF is NaN. */
int mx_dequantize8(const uint8_t* codes, int64_t ld, const uint8_t* scales, int64_t scale_ld,
                   int64_t rows, int64_t cols, void* out, int out_dtype, int64_t ldo, void* stream);

/* mx_gemm8: C[m][n] = alpha * sum_k deq(A)[m][k] * deq(B)[n][k] of two 8-bit matrices
 * A [M, K] and B [N, K]; C (c_dtype) has rows ldc >= N elements apart.  Any M, N < 2^31,
 * K <= 2^23 (M or N == 0: no-op; K == 0: C = 0, the operands may be NULL).  Sums are float32
 * in a fixed order, one rounding to nearest even gives a bf16 C.  For a float32 C the products
 * are exact too (of values used down to bits of 2^-133).  A bf16 C takes the 8-bit matrix
 * instructions, at twice the rate: they add the products of eight neighbouring k with 13
 * bits below the largest of them (2e-5 of C's norm for normal operands).  Scale byte 0xFF makes its
 * row's or column's sums NaN.  Up to 64 rows of A the weights B are read once.  workspace: at
 * least mx_gemm8_workspace_size bytes (the partial sums of sliced contractions; 0: may be
 * NULL), 16-byte aligned. */
size_t mx_gemm8_workspace_size(int64_t M, int64_t N, int64_t K);
int mx_gemm8(const uint8_t* a_codes, int64_t lda, const uint8_t* a_scales, int64_t a_scale_ld,
             const uint8_t* b_codes, int64_t ldb, const uint8_t* b_scales, int64_t b_scale_ld,
             int64_t M, int64_t N, int64_t K, float alpha, void* c, int c_dtype, int64_t ldc,
             void* workspace, size_t workspace_bytes, void* stream);

/* mx_linear8_fwd / mx_linear8_bwd: the linear layer on 8-bit matrices,
 *   Y = Q(X) Q(W)^T;  dX = Q(dY) Q(W);  dW = Q^T(dY) Q^T(Q(X))^T (straight-through)
 * with Q(X), Q(dY) in 1x128 blocks along the contraction, Q(W) in 128x128 tiles, and Q^T the
 * 128x1 blocks along the rows.  X [M, K], W [N, K], Y, dY [M, N]; each with a type and rows
 * ld* elements apart of its own; dw is float32.  A bf16 y or dx takes the 8-bit matrix
 * instructions, a float32 one exact products, as mx_gemm8's C.  The forward writes y and what the backward
 * takes: the 8-bit checkpoint of X (xq_codes [M][K16], xq_scales [M][4 ceil(K/512)]; K16: K
 * rounded up to a multiple of 16), and the weight in both layouts (wq_codes [N][K16],
 * wq_scales [N][4 ceil(K/512)], wt_codes [K][N16], wt_scales [K][4 ceil(N/512)]).  wt_codes
 * and wt_scales NULL: no backward is to come.  w NULL: wq holds the quantized weight already
 * (several forwards with the same weight; wt is not touched).  Any M, N, K <= 2^23.  Forward:
 * M or N == 0 writes no y; K == 0: y = 0.  Backward: K == 0 is a no-op; M or N == 0 gives dx = 0
 * and dw = 0 and reads nothing.  workspace as mx_linear_bwd's, of at least the bytes that the
 * _workspace_size call gives (0: may be NULL). */
size_t mx_linear8_fwd_workspace_size(int64_t M, int64_t N, int64_t K);
int mx_linear8_fwd(const void* x, int x_dtype, int64_t ldx, const void* w, int w_dtype, int64_t ldw,
                   int64_t M, int64_t N, int64_t K, void* y, int y_dtype, int64_t ldy,
                   uint8_t* xq_codes, uint8_t* xq_scales, uint8_t* wq_codes, uint8_t* wq_scales,
                   uint8_t* wt_codes, uint8_t* wt_scales, void* workspace, size_t workspace_bytes,
                   void* stream);
size_t mx_linear8_bwd_workspace_size(int64_t M, int64_t N, int64_t K);
int mx_linear8_bwd(const void* dy, int dy_dtype, int64_t lddy, int64_t M, int64_t N, int64_t K,
                   const uint8_t* xq_codes, const uint8_t* xq_scales, const uint8_t* wt_codes,
                   const uint8_t* wt_scales, void* dx, int dx_dtype, int64_t lddx, float* dw,
                   int64_t lddw, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ gated activation
 * h = act(g) u of rows z = (g, u): z [rows][2 cols], rows ldz >= 2 cols elements apart, g the
 * first half of a row, u the second; act MX_SILU or MX_GELU (Phi the normal distribution);
 * float32 arithmetic, one rounding to h's type.  It stands between an MLP's up and down
 * products.  live: DEVICE counter of the rows in use (mx_moe_plan's offs + experts, 8-byte
 * aligned), or NULL for all; outputs of rows from *live on are left as they were.
 * kept_codes / kept_scales (both NULL: nothing is kept): the checkpoint for the backward
 * pass, the 8-bit matrix of [2 rows, cols] whose rows 2r and 2r+1 are g and u of row r --
 * what mx_quantize8 (MX_ROW) writes for z seen as [2 rows][cols].  Any rows < 2^30, cols <=
 * 2^23; rows or cols == 0: no-op.
 *
 * mx_glu: h [rows][cols] (h_dtype, rows ldh elements apart).
 * mx_glu_quantize: h as the packed MXFP4 operand of the next product instead, the codes and
 *   scales of mx_quantize_ld (MX_ROW, MX_RNE, no rotation) of float32 h; cols % 32 == 0.
 * mx_glu_quantize8: h as an 8-bit matrix, mx_quantize8 (MX_ROW) of float32 h.
 * mx_glu_bwd: dz = (dh u act'(g), dh act(g)), g and u the values that the checkpoint holds,
 *   one rounding to dz's type. */
int mx_glu(const void* z, int z_dtype, int64_t ldz, const int64_t* live, int64_t rows, int64_t cols,
           int act, void* h, int h_dtype, int64_t ldh, uint8_t* kept_codes, int64_t kept_ld,
           uint8_t* kept_scales, int64_t kept_scale_ld, void* stream);
int mx_glu_quantize(const void* z, int z_dtype, int64_t ldz, const int64_t* live, int64_t rows,
                    int64_t cols, int act, uint8_t* codes, uint8_t* scales, int64_t scale_ld,
                    uint8_t* kept_codes, int64_t kept_ld, uint8_t* kept_scales,
                    int64_t kept_scale_ld, void* stream);
int mx_glu_quantize8(const void* z, int z_dtype, int64_t ldz, const int64_t* live, int64_t rows,
                     int64_t cols, int act, uint8_t* codes, int64_t ld, uint8_t* scales,
                     int64_t scale_ld, uint8_t* kept_codes, int64_t kept_ld, uint8_t* kept_scales,
                     int64_t kept_scale_ld, void* stream);
int mx_glu_bwd(const void* dh, int dh_dtype, int64_t lddh, const uint8_t* kept_codes, int64_t kept_ld,
               const uint8_t* kept_scales, int64_t kept_scale_ld, const int64_t* live, int64_t rows,
               int64_t cols, int act, void* dz, int dz_dtype, int64_t lddz, void* stream);

/* ------------------------------------------------------------------ router
 * mx_moe_route: the choices of a mixture-of-experts layer's router.  logits [tokens][experts]
 * (`dtype`, rows ld >= experts elements apart), s their softmax over the experts.  A token takes
 * part if mask [tokens] is NULL or not 0 there and some logit of it is not -Inf; n such tokens.
 *   ids [tokens][top_k]     the experts of the largest logits, in falling order, of equal ones
 *                           the lowest first; -1 (a slot left out, as mx_moe_plan takes it)
 *                           where only -Inf or NaN is left, and for a token that takes no part
 *   weights [tokens][top_k] float32: s of the choice, divided by the choices' sum where
 *                           renormalize is 1; 0 for a slot left out
 *   counts [experts + 1]    slots of each expert; n
 *   sums [experts]          float32: sum of s over the tokens that take part
 *   loss [1]                float32: the balance loss E sum_e f_e P_e, f_e = counts_e / (n
 *                           top_k), P_e = sums_e / n; 0 if n is 0
 * NaN or +Inf among a token's logits makes its weights, the sums and the loss NaN.  The order of
 * the sums is fixed.  1 <= experts <= MX_MAX_GROUPS, 1 <= top_k <= min(experts, 16), tokens *
 * top_k < 2^31.  workspace: at least mx_moe_route_workspace_size bytes (0: may be NULL).
 *
 * mx_moe_route_bwd: dlogits (`dtype`, rows ldd elements apart) from dweights [tokens][top_k]
 * (mx_moe_combine_bwd's) and dloss [1] (each float32 or NULL for 0), with the forward's ids
 * and counts; the choices and counts are constants of the gradient.  counts may be summed over
 * several devices' batches first (the loss is then that of all of them).  0 for a token that
 * takes no part; dweights of a slot left out are not used. */
size_t mx_moe_route_workspace_size(int64_t tokens, int64_t experts, int64_t top_k);
int mx_moe_route(const void* logits, int dtype, int64_t ld, const uint8_t* mask, int64_t tokens,
                 int64_t experts, int64_t top_k, int renormalize, int32_t* ids, float* weights,
                 int32_t* counts, float* sums, float* loss, void* workspace,
                 size_t workspace_bytes, void* stream);
int mx_moe_route_bwd(const void* logits, int dtype, int64_t ld, const uint8_t* mask, int64_t tokens,
                     int64_t experts, int64_t top_k, int renormalize, const int32_t* ids,
                     const int32_t* counts, const float* dweights, const float* dloss,
                     void* dlogits, int64_t ldd, void* stream);

/* ------------------------------------------------------------------ expert routing
 * Rows of a mixture-of-experts layer ([ALTO] news paragraph: the MoE model trained
 * in MXFP4) between token order and the expert order of the grouped products.  Slot
 * s = token * top_k + j is a token's j-th choice.  top_k >= 1, and tokens * top_k and
 * rows are below 2^31.
 *
 * mx_moe_plan: slots sorted by expert, stably (rows of an expert in slot order).
 * ids [tokens][top_k] (id_type MX_I32 or MX_I64); an id outside 0 .. experts-1
 * leaves its slot out (padding tokens).  Writes offs [experts+1] (offs[e] = slots of
 * the experts before e; offs[experts] = sorted rows R), src [tokens*top_k] (slot of
 * row r; -1 from row R on) and pos [tokens][top_k] (row of a slot; -1 for one left
 * out).  1 <= experts <= MX_MAX_GROUPS.  workspace: at least
 * mx_moe_plan_workspace_size bytes (0: may be NULL), 16-byte aligned.  tokens == 0
 * writes offs = 0 (ids, src, pos may be NULL).  The grouped products that take host
 * offsets need offs copied to the host. */
size_t mx_moe_plan_workspace_size(int64_t tokens, int64_t top_k, int64_t experts);
int mx_moe_plan(const void* ids, int id_type, int64_t tokens, int64_t top_k, int64_t experts,
                int64_t* offs, int32_t* src, int32_t* pos, void* workspace,
                size_t workspace_bytes, void* stream);

/* The row calls take pos as mx_moe_plan writes it: entries in 0 .. rows-1, each at
 * most once; an entry outside that range leaves its slot out.  Rows of an expert-
 * ordered output that no slot maps to are left as they were.  Row strides (ld*, in
 * elements) are at least cols.  weights: float32 [tokens][top_k], or NULL for 1; the
 * weight of a slot left out is not used.
 *
 * mx_moe_dispatch: out[pos[t][j]] = weights[t][j] * x[t] for every slot; x [tokens]
 * [cols] and out [rows][cols] are `dtype`.  Without weights an exact copy (the
 * gather in front of a grouped product), with weights the gradient of
 * mx_moe_combine alone.  One read of x. */
int mx_moe_dispatch(const void* x, int dtype, int64_t ldx, const int32_t* pos,
                    const float* weights, int64_t tokens, int64_t top_k, int64_t rows,
                    int64_t cols, void* out, int64_t ldo, void* stream);

/* mx_moe_dispatch_quantize: Q_D of mx_moe_dispatch's copy, the grouped forward's
 * operand, without the copy: codes [rows][cols/2] and scales (rows scale_ld >=
 * cols/32 bytes apart) equal, bit for bit, those of mx_quantize_ld (MX_ROW, MX_RNE,
 * no rotation) on the gathered rows.  cols % 32 == 0. */
int mx_moe_dispatch_quantize(const void* x, int dtype, int64_t ldx, const int32_t* pos,
                             int64_t tokens, int64_t top_k, int64_t rows, int64_t cols,
                             uint8_t* codes, uint8_t* scales, int64_t scale_ld, void* stream);

/* mx_moe_combine: y[t] = sum_j weights[t][j] * z[pos[t][j]] over the token's slots in
 * order, float32 sums of rounded products, one rounding to y's type; 0 for a token
 * without slots.  z [rows][cols] (z_dtype), y [tokens][cols] (y_dtype).  Without
 * weights it is the gradient of mx_moe_dispatch (straight through the quantizer for
 * mx_moe_dispatch_quantize). */
int mx_moe_combine(const void* z, int z_dtype, int64_t ldz, int64_t rows, const int32_t* pos,
                   const float* weights, int64_t tokens, int64_t top_k, int64_t cols, void* y,
                   int y_dtype, int64_t ldy, void* stream);

/* mx_moe_combine_bwd: gradients of mx_moe_combine, given dy [tokens][cols] (dy_dtype)
 * and the forward's z, pos and weights:
 *   dz[pos[t][j]] = weights[t][j] * dy[t]                      (dy_dtype)
 *   dweights[t][j] = sum_c dy[t][c] * z[pos[t][j]][c]  (float32; 0 for a slot left out)
 * in one pass over dy and z.  The order of the sums is fixed. */
int mx_moe_combine_bwd(const void* dy, int dy_dtype, int64_t lddy, const void* z, int z_dtype,
                       int64_t ldz, int64_t rows, const int32_t* pos, const float* weights,
                       int64_t tokens, int64_t top_k, int64_t cols, void* dz, int64_t lddz,
                       float* dweights, void* stream);

/* ------------------------------------------------------------------ de-oscillation
 * Weight de-oscillation as a post-optimizer-step pass ([ALTO] "How does ALTO
 * detect and fix oscillating weights?" and the ratio paragraph).  w is the
 * float32 master weight [rows, cols]; its bin value q(w) is the forward weight
 * quantizer's output deq(Q_D(w)) with 1x32 RNE blocks along cols.  The state is
 * three caller-owned float32 arrays of the same shape: w_prev (snapshot),
 * d_w (master-weight path length) and d_q (quantized path length).
 *
 * mx_deosc_init: w_prev = w, d_w = d_q = 0. */
int mx_deosc_init(const float* w, int64_t rows, int64_t cols,
                  float* w_prev, float* d_w, float* d_q, void* stream);

/* mx_deosc_step: call once after every optimizer step, in float32:
 *   d_w += |w - w_prev|;  d_q += |q(w) - q(w_prev)|;  w_prev = w.
 * If end_of_window != 0 (every P-th call, P = 200 on the page): flag =
 * d_q > threshold * d_w (threshold 4.0 on the page); flagged elements are
 * snapped, w = q(w); then w_prev = w and d_w = d_q = 0; flags (uint8 [rows][cols],
 * required then, else ignored) receives 1 for flagged elements, 0 otherwise.
 * cols % 32 == 0.  w is updated in place. */
int mx_deosc_step(float* w, int64_t rows, int64_t cols, float* w_prev, float* d_w, float* d_q,
                  int end_of_window, float threshold, uint8_t* flags, void* stream);

/* mx_deosc_step_quantize: mx_deosc_step, and in the same pass the next forward's
 * weight operand Q_D(w) of the updated w (1x32 blocks along cols, nearest
 * rounding), written to wq_codes [rows][cols/2] and wq_scales [rows][cols/32]
 * (caller-owned device memory; wq_codes 16-byte aligned) -- bit-identical to
 * mx_quantize(w, MX_F32, rows, cols, MX_ROW, MX_RNE, ...) after the step.  The
 * ALTO page runs the hook and the forward's weight quantization separately;
 * snapping to the bin value keeps every code and scale, so one pass gives both.
 * Arguments and errors otherwise as mx_deosc_step. */
int mx_deosc_step_quantize(float* w, int64_t rows, int64_t cols, float* w_prev, float* d_w,
                           float* d_q, int end_of_window, float threshold, uint8_t* flags,
                           uint8_t* wq_codes, uint8_t* wq_scales, void* stream);

/* mx_qema_step: Q-EMA post-step update ("Oscillation-Reduced MXFP4 Training for
 * Vision Transformers", rebuttal: Question 4 -- one EMA copy per linear weight;
 * the overhead answer -- it is updated with the parameters and it is what the
 * forward quantizes; the hyperparameter answer -- beta 0.998 by default).  In
 * float32, in this order:  ema = (beta * ema) + ((1 - beta) * w), 1 - beta
 * rounded to float32 first; then wq_codes / wq_scales = Q_D(ema) (1x32 blocks
 * along cols, nearest rounding), the next forward's weight operand.
 * w [rows][cols] float32 (read), ema [rows][cols] float32 (updated in place;
 * the caller starts it as a copy of w).  cols % 32 == 0; w, ema, wq_codes
 * 16-byte aligned device memory owned by the caller. */
int mx_qema_step(const float* w, float* ema, int64_t rows, int64_t cols, float beta,
                 uint8_t* wq_codes, uint8_t* wq_scales, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MX355_MX_H */
