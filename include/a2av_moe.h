/*
 * a2av_moe.h -- C ABI of the operators that stand around the variable-count
 * exchange in an expert-parallel layer on one MI355X (gfx950): the top-k
 * router that makes the exchange's gather lists and counts, the products of
 * the received rows with their experts' weights, the weighted return of the
 * rows to their tokens, and the microscaled 4-bit format for rows and weights.
 *
 * Conventions, all entry points:
 *   - Pointers are device addresses unless said otherwise; the work runs on
 *     the device current at the call and on `stream` (a hipStream_t, NULL =
 *     default stream).  A call enqueues kernel launches only (no copies, no
 *     memsets, no allocation, no synchronization), so it may be captured into
 *     a HIP graph; every replay reads the buffers' contents at replay time.
 *   - Host checks run before anything is enqueued, in this order: NULLPTR (a
 *     required pointer is NULL; a pointer to an operand without bytes may be
 *     NULL) -> UNSUPPORTED_DTYPE -> INVALID_ARGS (sizes, strides, alignment,
 *     an output that shares a byte with another operand; rows of one may lie
 *     between another's, as columns of one buffer do).  A failed launch is
 *     A2AV_ERR_HIP.
 *   - `status` is a device int32 that may be NULL.  The device writes it only
 *     when a check on device data fails (the codes of a2av.h), so it is a
 *     latch that the caller clears; the call itself has returned A2AV_OK.
 *   - Strides are in elements from one row to the next, below 2^31; rows are
 *     contiguous.
 *   - Sums, softmax statistics and gradients of weights are held in FP32; a
 *     result is rounded once, to nearest even, to its type.  No result depends
 *     on the order in which workgroups run.
 */
#ifndef A2AV_MOE_H
#define A2AV_MOE_H

#include <stdint.h>

#include "a2av.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- the router
 *
 * For every token t the k largest of its E logits, in falling order, equal
 * ones by their lower number.  A logit of -inf is not chosen; a token with
 * fewer than k other logits has empty slots.  With p = softmax(logits[t]):
 *   experts[t][j]  the j-th expert, -1 for an empty slot
 *   weights[t][j]  p of that expert, with renormalize != 0 divided by the sum
 *                  over the token's chosen ones; 0 for an empty slot, and where
 *                  exp(l - largest l) lies below 2^-126
 *   counts[e]      tokens that chose e
 *   order[r]       the token of row r when the slots stand in expert order,
 *                  within an expert by token: the gather list that the
 *                  products below take (and that a2av_run_indexed takes as
 *                  its index); -1 past the rows in use
 *   place[t][j]    the row of slot j, -1 for an empty one
 * A NaN logit ranks above every number (the lowest numbered first) and makes
 * the token's weights NaN, as softmax does; so does +inf.
 * Limits: tokens * k <= 2^30, E in 1..1024, k in 1..min(E, 16).
 */

/* Bytes of workspace that a2av_moe_route needs for these sizes (0 when it
 * needs none).  Pure host function; `bytes` is a host pointer. */
int a2av_moe_route_workspace(int64_t tokens, int32_t E, int32_t k, int64_t *bytes);

/*   logits     [tokens, E] of dtype FP32, FP16 or BF16, row stride
 *              logits_stride >= E
 *   experts    int32 [tokens, k]      weights  float [tokens, k]
 *   counts     int32 [E]              order    int32 [tokens * k]
 *   place      int32 [tokens, k]
 *   workspace  workspace_bytes >= a2av_moe_route_workspace, 16-byte aligned;
 *              its contents are scratch, of use to this call only */
int a2av_moe_route(const void *logits, int64_t logits_stride, int64_t tokens, int32_t E, int32_t k,
                   int32_t renormalize, int32_t dtype, int32_t *experts, float *weights,
                   int32_t *counts, int32_t *order, int32_t *place, void *workspace,
                   int64_t workspace_bytes, void *stream);

/* The gradient of the weights with respect to the logits:
 *   dlogits[t][e] = q_e * (g_e - sum_j weights[t][j] * dweights[t][j])
 * with g_e = dweights of the slot that chose e (0 if none; a token's slots
 * choose different experts, as the router's do) and q = softmax of
 * the logits, or with renormalize != 0 the weights themselves (0 where not
 * chosen).  Empty slots' dweights are not read into the sum; logits of -inf
 * get 0.  dlogits [tokens, E] has the logits' dtype and is contiguous.  An
 * expert outside [-1, E) counts as an empty slot. */
int a2av_moe_route_backward(const void *logits, int64_t logits_stride, int64_t tokens, int32_t E,
                            int32_t k, int32_t renormalize, int32_t dtype, const int32_t *experts,
                            const float *weights, const float *dweights, void *dlogits,
                            void *stream);

/* ------------------------------------------------- products grouped by expert
 *
 * `rows` rows stand in expert order: the first counts[0] belong to expert 0,
 * the next counts[1] to expert 1, and so on; rows past the counts' sum are
 * neither read nor written.  index, when not NULL, names for each of them the
 * row of x that it is (the router's order); x has x_rows rows.
 *   gmm     y [r][:] = W[e(r)] x[index[r]]           W [E, N, K], contiguous
 *   gmm_dx  dx[r][:] = W[e(r)]^T dy[r]
 *   gmm_dw  dW[e]    = sum over the rows r of e of dy[r] x[index[r]]^T
 * dtype FP16 or BF16 for every operand; dw_dtype is dtype or FP32.  An expert
 * without rows gets dW = 0.
 * Device checks: a negative count, or counts that sum to more than `rows` ->
 * INVALID_ARGS, nothing written (a forward product or gmm_dx of 0 rows enqueues
 * nothing and looks at no counts); an index in use outside [0, x_rows) ->
 * INVALID_ARGS, and that row counts as a row of zeros: its y is 0, or NaN where
 * W holds a NaN or an infinity (in dW, where dy does).
 * Limits: rows, x_rows, N, K <= 2^30, E in 1..4096.
 */
int a2av_moe_gmm(const void *x, int64_t x_stride, int64_t x_rows, const void *w,
                 const int32_t *counts, const int32_t *index, void *y, int64_t y_stride,
                 int64_t rows, int32_t E, int64_t N, int64_t K, int32_t dtype, int32_t *status,
                 void *stream);
int a2av_moe_gmm_dx(const void *dy, int64_t dy_stride, const void *w, const int32_t *counts,
                    void *dx, int64_t dx_stride, int64_t rows, int32_t E, int64_t N, int64_t K,
                    int32_t dtype, int32_t *status, void *stream);
int a2av_moe_gmm_dw(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride,
                    int64_t x_rows, const int32_t *counts, const int32_t *index, void *dw,
                    int64_t rows, int32_t E, int64_t N, int64_t K, int32_t dtype, int32_t dw_dtype,
                    int32_t *status, void *stream);

/* ------------------------------------------------------- the weighted return
 *
 *   combine   out[t] = sum_j weights[t][j] * y[place[t][j]]
 *   backward  dy[place[t][j]] = weights[t][j] * dout[t]
 *             dweights[t][j]  = <dout[t], y[place[t][j]]>
 * A slot with place -1 is left out (its dweights are 0); a token without
 * slots gets zeros.  weights NULL: every weight is 1 (the gradient of a
 * gather), and dweights may then be NULL.  y [y_rows, width], out and dout
 * [tokens, width] of dtype FP32, FP16 or BF16; weights float [tokens, k].
 * Rows of dy that no slot names are not written; a row may be named by one
 * slot only (two leave one of the two values).  Device check: a place outside
 * [-1, y_rows) -> INVALID_ARGS, and the slot counts as empty.
 * Limits: tokens, y_rows, width <= 2^30, k in 1..64.
 */
int a2av_moe_combine(const void *y, int64_t y_stride, int64_t y_rows, const int32_t *place,
                     const float *weights, void *out, int64_t out_stride, int64_t tokens,
                     int32_t k, int64_t width, int32_t dtype, int32_t *status, void *stream);
int a2av_moe_combine_backward(const void *dout, int64_t dout_stride, const void *y,
                              int64_t y_stride, int64_t y_rows, const int32_t *place,
                              const float *weights, void *dy, int64_t dy_stride, float *dweights,
                              int64_t tokens, int32_t k, int64_t width, int32_t dtype,
                              int32_t *status, void *stream);

/* -------------------------------------------------- microscaled 4-bit values
 *
 * A row of `cols` values is B = ceil(cols / 32) blocks of 32 (the last one
 * filled up with zeros): B scale bytes and 16 * B code bytes, both contiguous.
 * Scale byte s stands for 2^(s - 127), 255 for NaN.  A code is sign, two
 * exponent bits and one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6 and their
 * negatives; value 2i of a block is the low nibble of byte i, value 2i + 1 the
 * high one.
 * quantize: s = floor(log2(largest magnitude)) - 2 + 127, at least 0 (a block
 * of zeros has s = 0); codes are value / 2^(s - 127) rounded to nearest, ties
 * to even, magnitudes past 6 to 6; a zero keeps its sign.  A block with a NaN
 * or an infinity has s = 255 and codes 0.
 * dequantize: code * 2^(s - 127) rounded to dtype (past its range: infinity).
 * x FP32, FP16 or BF16.  Limits: rows, cols <= 2^30; codes 16-byte aligned.
 */
int a2av_moe_mx4_quantize(const void *x, int64_t x_stride, int64_t rows, int64_t cols,
                          int32_t dtype, uint8_t *codes, uint8_t *scales, void *stream);
int a2av_moe_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                            int32_t dtype, void *x, int64_t x_stride, void *stream);

/* gmm on the 4-bit values: x_codes [x_rows, 16 * B], x_scales [x_rows, B] and
 * w_codes [E, N, 16 * B], w_scales [E, N, B] with B = ceil(K / 32); codes past
 * a row's K values must be zero on one side at least (quantize writes them
 * so).  y is FP16, BF16 or FP32; counts, index, status, limits and device
 * checks as in gmm.  Codes 16-byte aligned. */
int a2av_moe_gmm_mx4(const uint8_t *x_codes, const uint8_t *x_scales, int64_t x_rows,
                     const uint8_t *w_codes, const uint8_t *w_scales, const int32_t *counts,
                     const int32_t *index, void *y, int64_t y_stride, int64_t rows, int32_t E,
                     int64_t N, int64_t K, int32_t y_dtype, int32_t *status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* A2AV_MOE_H */
