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
 *     mxfp4_dequantize 16, dX 16; other tensors their element size (else
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

/* ---- Products with an epilogue, and the backward pass of the layers above.
 * Weights stay what they are (codes): gradients go to activations, biases and
 * the router. */

/* The activation of an epilogue, z in fp32:
 *   NONE z;  RELU z where z is not below 0;  SILU z / (1 + exp(-z));
 *   GELU z erfc(-z / sqrt 2) / 2;
 *   GELU_TANH z / (1 + exp(-2u)), u = sqrt(2 / pi) (z + 0.044715 z^3), which is
 *             z (1 + tanh u) / 2;
 *   SWIGLU of a gate and an up value: gate / (1 + exp(-gate)) * up; N is even,
 *          columns n < N/2 are gates, n + N/2 their up values.
 * An infinite z follows the formula (SILU and GELU of -infinity are NaN); its
 * slope is the limit, 0 or 1. */
enum {
    MXFP4_ACT_NONE = 0,
    MXFP4_ACT_RELU = 1,
    MXFP4_ACT_SILU = 2,
    MXFP4_ACT_GELU = 3,
    MXFP4_ACT_GELU_TANH = 4,
    MXFP4_ACT_SWIGLU = 5
};

/* mxfp4_linear with an epilogue, F = N columns of Y (N/2 with SWIGLU):
 *     z[m,n] = sum_k X[m,k] * W[n,k] + bias[n]
 *     Y[m,f] = activation(z)[m,f] + residual[m,f]
 *   bias     in : [N] of X's dtype, or NULL
 *   residual in : [M, F] of X's dtype, rows r_stride elements apart, or NULL
 *   Y        out: [M, F] of X's dtype, dense
 *   Z        out: [M, N] of X's dtype, dense: z, for the backward pass; or NULL
 * Sums, z and the activation are fp32; Y and Z are rounded once each.
 * workspace as for mxfp4_linear, with its own size, which is that of any activation. */
size_t mxfp4_linear_act_workspace_bytes(int64_t M, int64_t N, int64_t K);
int mxfp4_linear_act(const void* X, int dtype, int64_t M, int64_t x_stride, const uint8_t* codes,
                     const uint8_t* scales, int64_t N, int64_t K, const void* bias,
                     int activation, const void* residual, int64_t r_stride, void* Y, void* Z,
                     void* workspace, size_t workspace_bytes, void* stream);

/* mxfp4_grouped_linear with the epilogue, each expert with its bias [E, N] (or
 * NULL).  Y: [R, F]; fp32 with MXFP4_FP32_ROWS (here with SWIGLU too); Z [R, N]
 * of X's dtype or NULL.  Rows of no expert are 0 in both (no bias). */
int mxfp4_grouped_linear_act(const void* X, int dtype, int64_t x_rows, int64_t x_stride,
                             const int32_t* tokens, int64_t R, const uint8_t* codes,
                             const uint8_t* scales, const int32_t* offsets, int64_t E, int64_t N,
                             int64_t K, const void* bias, int activation, void* Y, void* Z,
                             void* stream);

/* Gradient through an activation, and the bias's:
 *     dZ[r,n] = dY * activation'(Z), with SWIGLU
 *               dgate = dY * up * silu'(gate), dup = dY * silu(gate)
 *     dbias[e,n] = sum of dZ[r,n] over the expert's rows, before their rounding
 *   dY      in : fp16 or bf16 [R, F], rows y_stride elements apart
 *   Z       in : [R, N] of that dtype, rows z_stride elements apart
 *   offsets in : int32 [E + 1] as for mxfp4_grouped_linear, or NULL with E = 0:
 *                one bias, of all rows.  Rows of no expert are in no sum.
 *   dZ      out: [R, N] of that dtype, dense, every row
 *   dbias   out: fp32 [E, N] ([1, N] without offsets), or NULL
 *   workspace  DEVICE, 4-byte aligned, at least
 *              mxfp4_activation_grad_workspace_bytes(R, N, E) bytes (may be NULL
 *              where that is 0, or without dbias); no initial contents needed, in
 *              use until the call's work on the stream has finished.
 * RELU's slope at 0 is 0.  R = 0 makes dbias 0. */
size_t mxfp4_activation_grad_workspace_bytes(int64_t R, int64_t N, int64_t E);
int mxfp4_activation_grad(const void* dY, int dtype, int64_t R, int64_t y_stride, const void* Z,
                          int64_t z_stride, int64_t N, int activation, const int32_t* offsets,
                          int64_t E, void* dZ, float* dbias, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Gradient through the weight-only product: dX[m,k] = sum_n dY[m,n] * W[n,k].
 *   dY in : fp16 or bf16 [M, N], rows y_stride elements apart (any N, element
 *           alignment; more than 16 rows are read fastest where N is a multiple of 8
 *           and rows start on 16 bytes; 3001 of them take three to four times as long
 *           elsewhere)
 *   W  in : MXFP4 codes [N, K/2] and scales [N, K/32]
 *   dX out: [M, K] of dY's dtype, dense, 16-byte aligned
 * Accuracy as mxfp4_linear, with N terms: |dX - exact| <= (N/8 + 64) 2^-24
 * sum_n |dY w| + u |exact| + t.  workspace as for mxfp4_linear, with its own size. */
size_t mxfp4_linear_grad_workspace_bytes(int64_t M, int64_t N, int64_t K);
int mxfp4_linear_grad(const void* dY, int dtype, int64_t M, int64_t y_stride,
                      const uint8_t* codes, const uint8_t* scales, int64_t N, int64_t K, void* dX,
                      void* workspace, size_t workspace_bytes, void* stream);

/* The same by expert: dX[r,k] = sum_n dY[r,n] * W[e][n,k] for offsets[e] <= r <
 * offsets[e+1] (offsets as for mxfp4_grouped_linear; rows of no expert are 0).
 * dX: [R, K] of dY's dtype, fp32 with MXFP4_FP32_ROWS added to it; 16-byte
 * aligned.  The gradient of a gathered input is moe_combine of these rows with
 * weights of 1. */
int mxfp4_grouped_linear_grad(const void* dY, int dtype, int64_t R, int64_t y_stride,
                              const uint8_t* codes, const uint8_t* scales, const int32_t* offsets,
                              int64_t E, int64_t N, int64_t K, void* dX, void* stream);

/* Balance loss of a routing and the choices of each expert.  P = softmax of a
 * token's logits over all experts (an expert at -infinity has 0), c_e the ids
 * equal to e (ids outside [0, E) are no choice), C their sum, T' the tokens with
 * a logit above -infinity:
 *     loss = E * sum_e (c_e / C) * (sum_t P[t,e] / T')       (1 when balanced)
 *   logits in : fp16, bf16 or fp32 [T, E], rows `stride` elements apart
 *   ids    in : int32 [T, k], 1 <= k <= MOE_MAX_CHOICES
 *   loss   out: fp32, one value (0 where C or T' is 0)
 *   counts out: int32 [E + 1]: c_e, and T' in counts[E]
 *   workspace DEVICE, 4-byte aligned, at least moe_balance_workspace_bytes(T, E, k)
 *             bytes (may be NULL where that is 0); no initial contents needed, in use
 *             until the call's work on the stream has finished.
 * A logit of NaN or +infinity makes the loss NaN (and its token counts in T').
 * T k <= 2^29. */
size_t moe_balance_workspace_bytes(int64_t T, int64_t E, int64_t k);
int moe_balance(const void* logits, int dtype, int64_t T, int64_t E, int64_t stride,
                const int32_t* ids, int64_t k, float* loss, int32_t* counts, void* workspace,
                size_t workspace_bytes, void* stream);

/* Gradient of the routing weights and of the balance loss with respect to the
 * logits, the choices and counts being constants:
 *     dlogits[t,e] = sum_j dweights[t,j] * d weights[t,j] / d logits[t,e]
 *                    + *dloss * d loss / d logits[t,e]
 *   dweights in : fp32 [T, k], the gradient of moe_route's weights, or NULL (no
 *                 such part; ids may then be NULL).  renormalize as in moe_route.
 *                 Choices outside [0, E), or of an expert at -infinity, have none.
 *   counts   in : int32 [E + 1] of moe_balance (over more tokens than these T
 *                 where a loss spans several batches), or NULL (no such part)
 *   dloss    in : fp32, one value, with counts
 *   dlogits  out: [T, E] of the logits' dtype, dense.  0 for an expert at
 *                 -infinity, where the row has no NaN and no +infinity.
 * With renormalize and without counts a row's gradients depend on the logits of its
 * chosen experts alone: a NaN or +infinity among these makes the chosen experts'
 * gradients NaN, one elsewhere changes nothing.  In every other case a NaN or
 * +infinity makes all of the row's gradients NaN. */
int moe_route_grad(const void* logits, int dtype, int64_t T, int64_t E, int64_t stride,
                   const int32_t* ids, int64_t k, const float* dweights, int renormalize,
                   const int32_t* counts, const float* dloss, void* dlogits, void* stream);

/* Gradient of moe_combine: for r = positions[t,j],
 *     dY[r,n] = weights[t,j] * dout[t,n]
 *     dweights[t,j] = sum_n dout[t,n] * Y[r,n]     (fp32; 0 for no choice)
 *   dout   in : fp16 or bf16 [T, N];  Y in: [R, N] of that dtype, or fp32 with
 *               MXFP4_FP32_ROWS added to the dtype
 *   tokens in : int32 [R], positions int32 [T, k], of one moe_plan;  weights fp32
 *   dY     out: [R, N] of dout's dtype; a row that no choice of its token names
 *               is 0 (choices of one token that name one row add their weights). */
int moe_combine_grad(const void* dout, int dtype, int64_t T, int64_t N, const void* Y, int64_t R,
                     const int32_t* tokens, const int32_t* positions, const float* weights,
                     int64_t k, void* dY, float* dweights, void* stream);

/* Static description of a status code (never NULL). */
const char* mxfp4_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
