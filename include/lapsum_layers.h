/*
 * lapsum_layers.h -- C ABI of the operators around a routed layer: the norm in
 * front of it and the loss behind it, each with its gradients.
 *
 *   norm   y = (x - mean) / sqrt(var + eps) * weight + bias, row by row
 *   loss   softmax cross entropy of x W^T + b with one target a row, without
 *          the logits ever being kept
 *
 * The conventions are those of lapsum_experts.h: device pointers, rows
 * contiguous, outputs that alias nothing, all work ordered on `stream`,
 * nothing allocated, waited for or kept, scratch memory the caller's (16-byte
 * aligned, free again when the call's work on the stream is done), argument
 * errors returned before anything is launched, the same results every run.
 * Calls may be captured into a graph.
 */
#ifndef LAPSUM_LAYERS_H_
#define LAPSUM_LAYERS_H_

#include "lapsum_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Layer norm of rows.
 *   x, y         : dtype[rows, width].
 *   weight, bias : wtype[width], each may be NULL (1 and 0); wtype is dtype or
 *                  LAPSUM_F32.
 *   mean, rstd   : fp32[rows], what the VJP wants of the forward pass; each
 *                  may be NULL.
 * 0 <= rows <= LAPSUM_MAX_PAIRS, 1 <= width < 2^31, eps >= 0.  Statistics are
 * fp32, the variance from values about the mean; one past fp32's range is
 * infinite, and y is the bias.
 */
lapsum_status_t lapsum_layer_norm(const void* x, const void* weight, const void* bias, lapsum_dtype_t dtype,
                                  lapsum_dtype_t wtype, int64_t rows, int64_t width, float eps, void* y, float* mean,
                                  float* rstd, lapsum_stream_t stream);

/* dx: dtype[rows, width]; dweight, dbias: wtype[width], summed over the rows in
 * fp32; each may be NULL.  weight as in the forward call.  scratch:
 * lapsum_layer_norm_vjp_scratch_bytes(...) bytes, may be NULL when neither
 * dweight nor dbias is wanted. */
size_t lapsum_layer_norm_vjp_scratch_bytes(lapsum_dtype_t dtype, int64_t rows, int64_t width);
lapsum_status_t lapsum_layer_norm_vjp(const void* x, const void* weight, const float* mean, const float* rstd,
                                      const void* dy, lapsum_dtype_t dtype, lapsum_dtype_t wtype, int64_t rows,
                                      int64_t width, void* dx, void* dweight, void* dbias, void* scratch,
                                      lapsum_stream_t stream);

/* How the rows' losses leave: one each, their sum, or their sum over the number
 * of rows with a target (over 1 when there is none). */
typedef enum { LAPSUM_REDUCE_NONE = 0, LAPSUM_REDUCE_SUM = 1, LAPSUM_REDUCE_MEAN = 2 } lapsum_reduction_t;

#define LAPSUM_MAX_LOSS_SIDE 0x1000000 /* rows, vocabulary and width, at most */

/*
 * Softmax cross entropy of z = x W^T + bias: loss[t] = log sum_v e^z[t, v] -
 * z[t, target[t]].
 *   x      : dtype[rows, width].   weight: dtype[vocab, width].
 *   bias   : dtype[vocab] or NULL; -inf takes an entry out of the vocabulary.
 *   target : int64[rows]; a row whose target is outside [0, vocab) is ignored:
 *            its loss is 0, it has no gradient and a mean does not count it.
 *   loss   : fp32[rows], or fp32[1] with a reduction.
 *   lse    : fp32[rows], the logarithms, for the VJP; may be NULL.
 * A logit of +inf or NaN, or a row of nothing but -inf, makes its row's loss
 * NaN or infinite.  rows >= 0, vocab >= 1, width >= 0, each at most
 * LAPSUM_MAX_LOSS_SIDE.
 */
size_t lapsum_linear_cross_entropy_scratch_bytes(lapsum_dtype_t dtype, int64_t rows, int64_t vocab, int64_t width);
lapsum_status_t lapsum_linear_cross_entropy(const void* x, const void* weight, const void* bias,
                                            const int64_t* target, lapsum_dtype_t dtype, int64_t rows, int64_t vocab,
                                            int64_t width, lapsum_reduction_t reduction, float* loss, float* lse,
                                            void* scratch, lapsum_stream_t stream);

/*
 * With d = (e^(z - lse) - onehot) times the gradient of a row's loss: dx = d W,
 * dweight = d^T x, dbias = the sum of d over the rows.  For dx and dweight d is
 * rounded to dtype once, over the largest gradient of a row's loss, which
 * multiplies the fp32 sums again; dbias is summed before that rounding.
 *   lse   : the forward's.
 *   dloss : fp32, the gradient of what the forward returned: [rows], or [1]
 *           with a reduction.  A row that is ignored or whose gradient is 0
 *           has a dx of 0 and adds nothing to dweight and dbias, whatever it
 *           and its logits hold (infinities and NaN too).
 *   dx, dweight, dbias: dtype, shaped as x, weight, bias; each may be NULL.
 */
size_t lapsum_linear_cross_entropy_vjp_scratch_bytes(lapsum_dtype_t dtype, int64_t rows, int64_t vocab,
                                                     int64_t width);
lapsum_status_t lapsum_linear_cross_entropy_vjp(const void* x, const void* weight, const void* bias,
                                                const int64_t* target, const float* lse, const float* dloss,
                                                lapsum_dtype_t dtype, int64_t rows, int64_t vocab, int64_t width,
                                                lapsum_reduction_t reduction, void* dx, void* dweight, void* dbias,
                                                void* scratch, lapsum_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LAPSUM_LAYERS_H_ */
