/*
 * qgemm_w8a8.h -- C ABI of the 8-bit operators of a decoder layer's feed-forward half on MI355X
 * (gfx950): the residual's addition with the RMS norm, which can hand its result on in 8 bits, and
 * products of 8-bit activations with 8-bit weights, alone or as a gated pair.
 *
 * Conventions are those of qgemm.h: status codes, qgemm_last_error, caller-owned buffers, calls
 * that validate on the host, enqueue on `stream` and return, no allocation, no exception.
 *
 * Values in 8 bits are OCP e4m3 codes with one fp32 scale per block, value = code * scale:
 *   activations  codes [tokens][K], scales [K / 128][tokens]: a block is 128 consecutive values of a token;
 *   weights      codes [rows][K], scales [ceil(rows / 128)][K / 128]: a block is 128 x 128.
 * An activation block x is held with
 *   scale = max(max |x|, 2^-100) / 448,  code = RNE_e4m3(x / scale)
 * in fp32 (the quotient within 2 ulp); a block with a value that is not finite gets a NaN scale and NaN codes.
 */
#ifndef QGEMM_W8A8_H
#define QGEMM_W8A8_H

#include "qgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * qgemm_add_norm_t -- `tokens` rows of `dim` values.
 *   tokens in [0, 2^24] (more threads than one launch holds, from 2^22 rows on: UNSUPPORTED); dim a multiple of 8
 *   in [8, 32768]; dtype F16 or BF16: the type of x, residual,
 *   weight and sum_out; out_dtype the same type, or FP8_E4M3 (dim then a multiple of 128);
 *   norm: 1 = RMS norm, 0 = none (y is the sum itself).  eps >= 0 (finite), used with norm.
 */
typedef struct qgemm_add_norm {
  int64_t tokens;
  int32_t dim, dtype, out_dtype, norm;
  float eps;
  int32_t reserved;                 /* 0 */
} qgemm_add_norm_t;

/*
 * qgemm_add_norm -- enqueue, for every row,
 *   s = x + residual,   y[d] = s[d] / sqrt(mean(s^2) + eps) * weight[d]
 * in fp32; y is made from the sum before it is rounded.
 *   x, residual, sum_out  16-bit [tokens][dim] with token strides of their own (elements, a multiple of 8, at
 *             least dim).  residual may be NULL (s = x); sum_out, which receives s, may be NULL, and may be x or
 *             residual themselves (same pointer and stride), otherwise must not overlap them.
 *   weight    dim 16-bit values, or NULL (ones); ignored for norm = 0.
 *   y         [tokens][dim] contiguous, of out_dtype; overlaps no other argument.
 *   y_scales  fp32 [dim / 128][tokens] for FP8_E4M3, otherwise NULL.
 * Pointers are 16-byte aligned (y_scales: 4).  |s| up to 2^56 is covered: beyond it the sum of squares overflows.  So is any
 * eps, but with eps below 2^-126 a row whose root mean square is below 2^-56: its squares underflow.  With eps = 0 a row
 * of zeros is NaN, as 0 / 0 is.
 */
qgemm_status_t qgemm_add_norm(const qgemm_add_norm_t* problem, const void* x, int64_t x_stride, const void* residual,
                              int64_t residual_stride, const void* weight, void* sum_out, int64_t sum_stride, void* y,
                              float* y_scales, void* stream);

#define QGEMM_GATE_NONE 0
#define QGEMM_GATE_SILU 1           /* act(g) = g / (1 + exp(-g))  (either act: 0 where it lies below 2^-119)  */
#define QGEMM_GATE_GELU_TANH 2      /* act(g) = g / 2 (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3)))              */

/* kernel_hint values (testing and tuning; 0 is the right choice for applications) */
#define QGEMM_W8A8_AUTO 0
#define QGEMM_W8A8_ROWS 1           /* the weights stream past a few tokens: M <= 64             */
#define QGEMM_W8A8_TILES 2          /* tiles of tokens x weight rows, any M                      */

/* sums values: how products enter their sums (qgemm_w8a8_run) */
#define QGEMM_W8A8_SUMS_AUTO 0      /* as fine as the outputs show in ordinary data              */
#define QGEMM_W8A8_SUMS_WHOLE 1     /* every product whole, whatever the outputs and the kernel  */

/*
 * qgemm_w8a8_t -- out [M][N] from activations A [M][K] and weights W.
 *   M in [0, 2^24]; N a multiple of 16 in [16, 2^24]; K a multiple of 128 in [128, 2^22] (more workgroups than one
 *   launch holds: UNSUPPORTED);
 *   gate QGEMM_GATE_*: without a gate W is [N][K]; with one it is [2 N][K], the N rows of the gate's projection
 *   and then the N rows of the other, and w_scales is [2 ceil(N / 128)][K / 128] likewise (each has row blocks of
 *   its own, the last one short where N is no multiple of 128);
 *   out_dtype F16, BF16 or F32, or with a gate FP8_E4M3 (N then a multiple of 128): the activations of the next product;
 *   kernel_hint QGEMM_W8A8_*; split_hint 0 = automatic, else the workgroups (1 to 32) that share the K axis of
 *   one tile, in the kernel and with the tile that are taken without it; tile_hint 0 = automatic, else the tokens of a tile of the tiles kernel (64, 128 or 256);
 *   sums QGEMM_W8A8_SUMS_* (other values are reserved).
 *   The launch depends on the descriptor only.
 */
typedef struct qgemm_w8a8 {
  int64_t M, N, K;
  int32_t out_dtype, gate, kernel_hint, split_hint, tile_hint, sums;
} qgemm_w8a8_t;

/*
 * qgemm_w8a8_quantize -- offline, host memory only: fp32 weights w [rows][K] (rows = N, or 2 N with a gate) to
 * codes uint8 [rows][K] and scales fp32 (shapes above), scale = absmax / 448 in fp32 and
 * code = RNE_e4m3(clamp(w / scale, +-448)), the division in double; an all-zero block gets scale 0 and codes 0.
 * A weight that is not finite is refused.  M is ignored.  Codes and scales of other origin are as good: the
 * device reads both as they are.
 */
qgemm_status_t qgemm_w8a8_quantize(const qgemm_w8a8_t* problem, const float* w, uint8_t* codes, float* scales);

/* qgemm_w8a8_workspace_bytes -- device workspace of qgemm_w8a8_run (0 when none): zero-filled once by the caller,
 * then reusable by later calls in stream order.  One workspace of the largest size asked for serves all the descriptors it
 * was asked for; calls that overlap in time need different ones.  The size does not grow with M (11008 x 4096 gated to
 * e4m3: 1.9 MB for 16 tokens, 11.8 for 40, 0 for 200, 50.9 for 4096, 0 for 8192): a program that runs several M asks for each. */
qgemm_status_t qgemm_w8a8_workspace_bytes(const qgemm_w8a8_t* problem, size_t* bytes);

/*
 * qgemm_w8a8_run -- enqueue
 *   p_r[m] = sum_b a_scale[b][m] w_scale[r / 128][b] (sum_{k in block b} a[m][k] w[r][k])
 *   out[m][n] = p_n[m],  or act(p_n[m]) p_{N + n}[m] with a gate,
 * the sums in fp32, one rounding to out_dtype.  With F32 and FP8_E4M3 outputs, in the rows kernel and with sums =
 * QGEMM_W8A8_SUMS_WHOLE every product enters its sum whole.  Otherwise, with F16 and BF16 outputs, the tiles kernel (without a
 * hint from 17 tokens on, always above 64) adds the products of eight consecutive k first, cut off at 2^-13 of the largest
 * one's power of two: an error of at most 7 * 2^-13 times the sum of the groups' largest products (of normally distributed
 * values 1.4e-5 of an output's standard deviation).  Whole sums take the tiles kernel up to twice as long; ask for them where
 * large products may cancel, or where one token and a prompt must agree beyond the cut.
 *   A, W        e4m3 codes, contiguous, 16-byte aligned;  a_scales, w_scales fp32, contiguous, 4-byte aligned.  The two scales of
 *               a block sum are multiplied first: their product is covered from 2^-126 to 2^127, and 0.
 *   out         [M][N] of out_dtype, contiguous, 16-byte aligned;  out_scales fp32 [N / 128][M] for FP8_E4M3,
 *               otherwise NULL.
 *   workspace   see qgemm_w8a8_workspace_bytes; 256-byte aligned; may be NULL when 0 bytes are needed.
 * out, out_scales and the needed part of workspace overlap each other and the inputs nowhere (refused: INVALID_ARGUMENT).
 * M = 0 enqueues nothing.  Results are bitwise deterministic.
 */
qgemm_status_t qgemm_w8a8_run(const qgemm_w8a8_t* problem, const void* A, const float* a_scales, const void* W,
                              const float* w_scales, void* out, float* out_scales, void* workspace,
                              size_t workspace_bytes, void* stream);

/* qgemm_w8a8_describe -- as qgemm_plan_describe: one line naming the launch. */
qgemm_status_t qgemm_w8a8_describe(const qgemm_w8a8_t* problem, char* buf, size_t len);

#ifdef __cplusplus
}
#endif

#endif /* QGEMM_W8A8_H */
