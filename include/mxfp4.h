/*
 * mxfp4.h — C ABI of the MXFP4 linear layer and its mixture-of-experts form
 * for AMD Instinct MI355X (gfx950); built as libmxfp4.so.
 *
 * MXFP4 is the 4-bit floating point format of the OCP Microscaling Formats
 * specification v1.0 (sections 5 and 6.3): blocks of 32 consecutive columns
 * share one power-of-two scale, each element is an e2m1 code.
 *     code    sign (bit 3), exponent (bits 2-1, bias 1), mantissa (bit 0):
 *             magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6
 *     scale   one byte e8m0 per block: 2^(byte - 127); 255 is NaN
 *     value   2^(scale byte - 127) * code
 * Layout of a matrix of `rows` rows and K columns (dense, row-major):
 *     codes [rows, K/2] bytes: column 2i in the low nibble of byte i of the
 *           row, column 2i + 1 in the high nibble
 *     scales[rows, K/32] bytes
 *
 * Conventions shared by every entry point (those of w4a16.h, whose status
 * codes are used):
 *   - Every tensor pointer is a DEVICE pointer into memory the caller owns;
 *     the library allocates nothing and keeps no state between calls.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Work is enqueued
 *     asynchronously; nothing synchronizes.  Every call can be captured into
 *     a graph (no memset or memcpy node is recorded).
 *   - Arguments are validated on the host before anything is enqueued; a
 *     non-zero status means nothing was enqueued.
 *   - dtype: MXFP4_FP16, MXFP4_BF16 or MXFP4_FP32 where listed.
 *   - Sizes: 0 <= rows, M, N, T, R <= 2^24, 0 <= K <= 2^24, K % 32 == 0
 *     (else W4A16_ERR_SHAPE).  A call whose output has no element enqueues
 *     nothing (its pointers may then be NULL).  K == 0 makes every output of
 *     a product 0 (inputs without elements may be NULL).
 *   - Row strides count elements, at least K (else W4A16_ERR_INVALID_ARG).
 *   - Alignment: X, its row stride in bytes, codes and the Y of
 *     mxfp4_dequantize 16; other tensors their element size (else
 *     W4A16_ERR_MISALIGNED).
 *   - Outputs must not overlap inputs or each other (W4A16_ERR_INVALID_ARG).
 *   - Infinities and NaN are legal in every floating point input.
 *   - The current HIP device must be gfx950 (W4A16_ERR_DEVICE).
 */
#ifndef MXFP4_H
#define MXFP4_H

#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MXFP4_BLOCK 32

enum { MXFP4_FP16 = 0, MXFP4_BF16 = 1, MXFP4_FP32 = 2 };
/* Added to the dtype of mxfp4_grouped_linear or moe_combine: the experts' rows
 * (Y) are fp32, so that a token's sum over them is rounded once, at its end. */
#define MXFP4_FP32_ROWS 16

/* Quantize X [rows, K] (fp16, bf16 or fp32, rows `x_stride` elements apart).
 * Per block of 32 columns:
 *     a = max |x|;  E = clamp(floor(log2 a) - 2, -127, 127), 0 where a == 0
 *     code = x / 2^E rounded to the nearest e2m1 value, ties to the even
 *            mantissa, saturated at +-6 (the sign of a zero is kept)
 *     scale byte = E + 127
 * A block that holds an infinity or a NaN gets the scale 255 and codes 0, so
 * that it dequantizes to NaN and every product that meets it is NaN.
 * Bit-exact: exactly one correct output exists for every input. */
int mxfp4_quantize(const void* X, int dtype, int64_t rows, int64_t K, int64_t x_stride,
                   uint8_t* codes, uint8_t* scales, void* stream);

/* The values of MXFP4 codes and scales as Y [rows, K] (dense; fp16, bf16 or
 * fp32), each rounded once to nearest even (exact wherever dtype holds it). */
int mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                     void* Y, int dtype, void* stream);

/* Weight-only linear layer: Y[m,n] = sum_k X[m,k] * W[n,k].
 *   X  in : fp16 or bf16 [M, K], rows x_stride elements apart
 *   W  in : MXFP4 codes [N, K/2] and scales [N, K/32], dequantized in registers
 *   Y  out: [M, N] of X's dtype, dense
 * Accuracy: weights enter exactly, products are summed in fp32, y is rounded
 * once (RNE): |y - y_exact| <= (K/8 + 64) 2^-24 sum_k |x_k w_k| + u |y_exact| + t,
 * u = 2^-8 (bf16) or 2^-11 (fp16), t half the dtype's smallest subnormal.
 *   workspace  NULL with 0 bytes, or DEVICE memory, 16-byte aligned, of at
 *              least mxfp4_linear_workspace_bytes(M, N, K) bytes (0 for most
 *              shapes) for fp32 partial sums of K slices: few rows over a long
 *              K then run on more compute units.  No initial contents needed;
 *              in use until the call's work on the stream has finished.  With
 *              NULL the sums are not split. */
size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);
int mxfp4_linear(const void* X, int dtype, int64_t M, int64_t x_stride, const uint8_t* codes,
                 const uint8_t* scales, int64_t N, int64_t K, void* Y, void* workspace,
                 size_t workspace_bytes, void* stream);

/* Product of two MXFP4 matrices: Y[m,n] = sum_k A[m,k] * B[n,k], on the
 * block-scaled matrix instructions (fp32 sums; dtype fp16, bf16 or fp32,
 * rounded once).  A: [M, K], B: [N, K].  Accuracy as mxfp4_linear, u = 2^-24
 * for fp32.  workspace as for mxfp4_linear, with its own size. */
size_t mxfp4_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K);
int mxfp4_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M,
                 const uint8_t* b_codes, const uint8_t* b_scales, int64_t N, int64_t K,
                 void* Y, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* ---- Mixture of experts.  T tokens, E experts (1 <= E <= MOE_MAX_EXPERTS),
 * k choices per token (1 <= k <= min(E, MOE_MAX_CHOICES)). */
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_CHOICES 32

/* Top-k routing of logits [T, E] (fp16, bf16 or fp32, rows `stride` elements
 * apart, element-aligned):
 *   ids     out: int32 [T, k], the k largest logits in falling order, ties to
 *                the lowest expert; a NaN counts as larger than every number
 *   weights out: fp32 [T, k]: exp(l - max) over its sum, taken over the chosen
 *                (renormalize != 0) or over all E experts (0)
 * An expert whose logit is -infinity is never chosen: a slot left over has id
 * -1 and weight 0 (a row of -infinities, e.g. a padding token, chooses none).
 * A row with a NaN, or with +infinity, has NaN weights in its used slots. */
int moe_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t stride, int64_t k,
              int renormalize, int32_t* ids, float* weights, void* stream);

/* Orders the R = T k choices by expert (stable: by token and slot within an
 * expert).  An id outside [0, E) is no choice.
 *   offsets   out: int32 [E + 1]: expert e owns the rows offsets[e] up to
 *                  offsets[e + 1]
 *   tokens    out: int32 [R]: the token of each row; -1 in the rows from
 *                  offsets[E] on
 *   positions out: int32 [T, k]: the row of each choice, -1 for no choice
 *   workspace DEVICE, 4-byte aligned, at least moe_plan_workspace_bytes(T, k, E)
 *             bytes (0 for small R; then it may be NULL); no initial contents
 *             needed, in use until the call's work on the stream has finished.
 * T k <= 2^24. */
size_t moe_plan_workspace_bytes(int64_t T, int64_t k, int64_t E);
int moe_plan(const int32_t* ids, int64_t T, int64_t k, int64_t E, int32_t* offsets,
             int32_t* tokens, int32_t* positions, void* workspace, size_t workspace_bytes,
             void* stream);

/* Product by expert over ragged row groups, each with its expert's weights:
 *     for offsets[e] <= r < offsets[e+1]:
 *         h[n] = sum_k X[s, k] * W[e][n, k],  s = tokens ? tokens[r] : r
 *         Y[r, n] = h[n]                                  (swiglu == 0)
 *         Y[r, n] = h[n] / (1 + exp(-h[n])) * h[N/2 + n]  (swiglu != 0, n < N/2)
 *   X       in : fp16 or bf16 [x_rows, K], rows x_stride elements apart
 *   tokens  in : int32 [R] or NULL (then x_rows >= R); an index outside
 *                [0, x_rows) reads a row of zeros
 *   codes, scales in: MXFP4 [E, N, K/2], [E, N, K/32]
 *   offsets in : int32 [E + 1], rising; whatever they hold, an entry counts as at
 *                least 0 and those before it, at most R (a falling pair is an
 *                empty expert), and every row of Y is written once
 *   Y       out: [R, N] ([R, N/2] with swiglu, N even) of X's dtype, dense;
 *                rows of no expert (before offsets[0], from offsets[E] on) are 0
 *   dtype   X's; with MXFP4_FP32_ROWS added Y is fp32 (not with swiglu:
 *           W4A16_ERR_INVALID_ARG)
 * Accuracy per h as mxfp4_linear before its rounding; Y is rounded once. */
int mxfp4_grouped_linear(const void* X, int dtype, int64_t x_rows, int64_t x_stride,
                         const int32_t* tokens, int64_t R, const uint8_t* codes,
                         const uint8_t* scales, const int32_t* offsets, int64_t E, int64_t N,
                         int64_t K, int swiglu, void* Y, void* stream);

/* Weighted sum of each token's rows: out[t, n] = sum_j weights[t, j] *
 * Y[positions[t, j], n] in fp32, j rising, rounded once; a position outside
 * [0, R) adds nothing.  Y: fp16 or bf16 [R, N], out: [T, N] of that dtype; with
 * MXFP4_FP32_ROWS added to the dtype Y is fp32 (16-bit rows take half the traffic,
 * and their own roundings make the error of out 1.4 times as large). */
int moe_combine(const void* Y, int dtype, int64_t R, int64_t N, const int32_t* positions,
                const float* weights, int64_t T, int64_t k, void* out, void* stream);

/* Static description of a status code (never NULL). */
const char* mxfp4_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
