/*
 * sinkhorn_head.h -- the output end of a model, from its last hidden states to
 * what the losses of sinkhorn_losses.h take of a frozen model: old and
 * reference log-probabilities, a teacher's top tokens.
 *
 * The norm with the residual's addition, in the stream's type (with its
 * gradient) or in 8 bits; the product of 8-bit activations and weights, which
 * makes the logits; and the scores of a row of logits: log-probability,
 * entropy and top alternatives, with the gradient of the first two.
 *
 * Conventions (those of sinkhorn.h, and)
 *   - Matrices are rows of values side by side, `ld...` elements from one row to
 *     the next (at least a row's length; what lies between rows is neither read
 *     nor written, but for the 8-bit product's inputs, see there), at any
 *     address that suits their type.  `dtype` is SK_F32 or SK_BF16.
 *   - 0 <= T <= 2^24 rows.  With T == 0 the pointers of row arrays may be NULL.
 *   - Outputs and the workspace share no memory with one another or with inputs,
 *     but where an entry point says that an output may be an input itself: the
 *     same address and row distance.  Any other overlap is refused, and so are
 *     matrices of different row distances (in bytes) that lie between one another's rows.
 *   - Precision.  Sums of squares and of products within a row of the norm are
 *     fp64, the factor and the products with it fp32.  A row's exponentials and
 *     the sums of a thread over them are fp32; the joins of those, logarithms
 *     and log-probabilities are fp64 and rounded once.  A gradient value is an
 *     fp32 exponential times fp32 coefficients: off, relative, by a few 2^-24 and
 *     by 3 2^-24 of its distance s (M - z) from the row's maximum M, then rounded.
 *   - Same inputs at the same addresses modulo 128 bytes, same bits: no result
 *     depends on an order of atomics.
 *   - Every call enqueues kernels only and returns without waiting; it can be
 *     captured in a graph.  Calls that overlap need workspaces of their own,
 *     and a captured call's workspace has to outlive its graph.
 */
#ifndef SINKHORN_HEAD_H
#define SINKHORN_HEAD_H

#include <stddef.h>
#include <stdint.h>

#include "sinkhorn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Operation ids for sinkhorn_head_workspace_bytes(). */
enum {
    SK_OP_RMS_NORM_BACKWARD = 0,
    SK_OP_INT8_LINEAR = 1,
    SK_OP_TOKEN_SCORES = 2,
    SK_OP_TOKEN_SCORES_BACKWARD = 3
};

/*
 * Workspace bytes of an operation (0 if the arguments are out of range): T rows
 * of V values (d of the norm, N of the product) and k = the product's K, the
 * scores' number of alternatives, else 0.  No initialisation needed; contents
 * undefined after a call.
 */
size_t sinkhorn_head_workspace_bytes(int op, int T, int V, int k, int dtype);

/*
 * Root-mean-square norm of T rows of d values (1 <= d <= 32768), with the
 * addition of the residual stream before it:
 *     h = x + residual, rounded to the type (h = x if residual is NULL),
 *     y = h weight / sqrt(sum h^2 / d + eps)          (weight NULL: 1).
 * y is the norm of h as it is stored, so that the backward pass, which has h
 * alone, is its gradient.  h may be NULL (not written); without a residual it
 * is a copy of x.  eps in [1e-30, 1e30].
 * y or h may be x or the residual themselves (not both the same one).  Sums of
 * squares are fp64; the factor, its product with h and that with the weight are fp32,
 * and y is rounded to the type behind them.  (Of rows whose root mean square is beyond
 * 2^126 the factor lies below fp32's normal range: another 2^-22 of y, and of
 * the parts of the gradient.)
 */
int sinkhorn_rms_norm(const void *x, int dtype, int64_t ldx, const void *residual, int64_t ldr,
                      const void *weight, int T, int d, double eps, void *y, int64_t ldy,
                      void *h, int64_t ldh, void *stream);

/*
 * The same with y in 8 bits and a scale for each row: with p = h weight and
 * a = max |p| over the row,
 *     q = 127 p / a, rounded to the nearest (ties to even),
 *     scale = a / (127 sqrt(sum h^2 / d + eps)),       y ~ scale q.
 * The norm's factor cancels in q, which is exact to the last tie (but for bf16
 * products below fp32's normal range, which lose bits).  A row of zeros has q 0 and
 * scale 0; a row with NaN or an infinity, or a bf16 one with products beyond fp32, has
 * q 0 and scale NaN.  Rows at multiples of 128 bytes are read fastest by the product.
 */
int sinkhorn_rms_norm_int8(const void *x, int dtype, int64_t ldx, const void *residual,
                           int64_t ldr, const void *weight, int T, int d, double eps, int8_t *q,
                           int64_t ldq, float *scale, void *h, int64_t ldh, void *stream);

/*
 * 8 bits without a norm, for weights (a row is an output channel) and other
 * activations: q = 127 x / max |x| rounded, scale = max |x| / 127; the same
 * rows of zeros, NaN and infinities.
 */
int sinkhorn_quantize_int8(const void *x, int dtype, int64_t ldx, int T, int d, int8_t *q,
                           int64_t ldq, float *scale, void *stream);

/*
 * Gradient of sinkhorn_rms_norm from dy = dL/dy and dh, what reaches h along
 * the residual stream (NULL: nothing).  With r = 1 / sqrt(sum h^2 / d + eps),
 * n = h r and u = dy weight,
 *     dx = r (u - n (r sum u h) / d) + dh               (x's and the residual's),
 *     dweight_j = sum over rows of dy_j n_j             (fp32 [d]; NULL: none).
 * dx may be dy, dh or h itself.  Sums within a row are fp64; those of dweight
 * are fp32 over up to T / 1024 + 1 rows (rounded up to whole work-groups) and fp64 beyond.
 * u is fp32: where it lies below 1e36 and within fp32's normal range, any row of finite h has
 * its gradient.  (The workspace is asked for without dweight, too.)
 */
int sinkhorn_rms_norm_backward(const void *dy, int dtype, int64_t lddy, const void *h,
                               int64_t ldh, const void *weight, const void *dh, int64_t lddh,
                               int T, int d, double eps, void *dx, int64_t lddx, float *dweight,
                               void *ws, size_t ws_bytes, void *stream);

/*
 * Product in 8-bit integers, a scale for each token and each channel:
 *     out[t][n] = xscale[t] wscale[n] sum_k x[t][k] w[n][k] + bias[n],
 * x [T][K], w [N][K] (1 <= K <= 131071, so that sums stay within 32 bits;
 * 1 <= N <= 2^24, T N <= 2^37), out [T][N] in `dtype`, bias [N] fp32 or NULL.  Rows of x and w
 * start at multiples of 16 bytes (addresses and ldx, ldw): a row's last 16 bytes
 * are read whole, and what lies behind the row in them has no effect.
 * The sum is exact; its conversion (beyond 2^24 a rounding), the scales' product, their
 * product with it and the bias's addition are fp32, rounded once to the type.
 */
int sinkhorn_int8_linear(const int8_t *x, int64_t ldx, const float *xscale, const int8_t *w,
                         int64_t ldw, const float *wscale, const float *bias, int T, int K, int N,
                         int dtype, void *out, int64_t ldo, void *ws, size_t ws_bytes,
                         void *stream);

/*
 * Scores of rows of logits [T][V] (1 <= V <= 2^24), with s = scale (an inverse
 * temperature, from 1e-20 to 1e20) and q = softmax(s z) of a row:
 *     lse[t] = log sum_v exp(s z_tv),    logp[t] = s z_{t,labels[t]} - lse[t],
 *     entropy[t] = -sum_v q_v log q_v,
 *     index[t][i], best[t][i]: the `top` largest logits (0 <= top <= 128) in
 *         falling order, among equal ones (0 and -0 are) the lower index first:
 *         their tokens and log-probabilities.
 * Outputs may be NULL (not all; index and best both or neither, with top > 0).
 * labels may be NULL: every row is scored, and there is no logp.  A negative
 * label marks a row that is not scored: its logits are not read, logp, lse and
 * entropy are 0 and its alternatives are empty.  A label of V or more gives a
 * logp of NaN alone.  A logit of -inf has no probability and is no alternative; an
 * empty place holds index -1 and best -inf, which sinkhorn_distill_loss takes as no
 * entry.  A row of nothing but -inf has logp 0 whatever its label, lse -inf, entropy 0.  A row with
 * NaN or +inf has logp, lse, entropy and best NaN; index then names the NaN
 * first, the infinities next.
 */
int sinkhorn_token_scores(const void *logits, int dtype, int64_t ld, const int32_t *labels,
                          int T, int V, double scale, int top, float *logp, float *lse,
                          float *entropy, int32_t *index, float *best, void *ws,
                          size_t ws_bytes, void *stream);

/*
 * The gradient of logp and entropy from grad [T] = dL/dlogp and grad_entropy
 * [T] = dL/dentropy (either may be NULL: 0; labels may be NULL without grad):
 *     dlogits[t][v] = s (grad (1[v = label] - q_v) - grad_entropy q_v (log q_v + entropy)).
 * A row of which both are 0, or that is not scored, is not read; its gradient is
 * 0.  dlogits [T][V] has the logits' type and may be the logits themselves.
 * The row's softmax is found again on the way (the row is read once).
 */
int sinkhorn_token_scores_backward(const void *logits, int dtype, int64_t ld,
                                   const int32_t *labels, const float *grad,
                                   const float *grad_entropy, int T, int V, double scale,
                                   void *dlogits, int64_t dld, void *ws, size_t ws_bytes,
                                   void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SINKHORN_HEAD_H */
