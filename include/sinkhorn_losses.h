/*
 * sinkhorn_losses.h -- losses over rows of logits, with their gradients: the
 * part of the library's C ABI that a training step uses beside the transport
 * losses of sinkhorn.h.
 *
 * Each is one streamed log-sum-exp per row, as a Sinkhorn half-iteration is,
 * and a gradient "coefficient x softmax + a few sparse terms", as the loss on a
 * sparse plan's support is.  The T x V softmax never exists in memory.
 *
 * Conventions (those of sinkhorn.h, and)
 *   - logits is [T][V] in `dtype` (SK_F32 or SK_BF16), rows `ld` elements apart
 *     (ld >= V; the elements behind V are neither read nor written), at any
 *     address that suits its type.  Rows whose dlogits lie at the same address
 *     modulo 128 bytes as their logits are written fastest.
 *   - dlogits has the logits' dtype and rows `dld` apart.  It may be the logits
 *     themselves (the same address and row distance): the gradient is then
 *     written over them.  NULL: no gradient.  Any other call in which outputs, the
 *     gradient or the workspace share memory with each other or with an input is
 *     refused; arrays between the rows of padded logits share none with them.
 *   - 0 <= T <= 2^24 rows and 1 <= V <= 2^24 values.  With T == 0 the pointers
 *     of row arrays may be NULL.
 *   - labels is [T] int32.  A negative label marks a row that is not scored (a
 *     prompt, padding): its logits are not read, its outputs are 0 and its
 *     gradient row is 0.  A label of V or more gives NaN where it enters,
 *     nothing is read out of range.
 *   - Packed sequences: offsets [n + 1] int64, non-decreasing; sequence i is
 *     rows offsets[i] <= t < offsets[i + 1] (empty ones are allowed; at most
 *     2^20 sequences, pairs or groups).  Rows
 *     before the first and behind the last sequence are left as they are in
 *     every row output, or get zeros with SK_LOSS_FILL.
 *   - A logit of -inf has no probability (masked vocabulary, disabled expert).
 *     A row of nothing but -inf has no distribution and drops out like a row
 *     that is not scored (of a mean's count too where the operation says so).  The
 *     type's lowest finite value is an ordinary number.  NaN or +inf gives NaN.
 *   - The returned losses include their weights, and the gradient is that of
 *     their sum.  A sequence, pair or row of weight 0 has loss (and KL) 0 and
 *     gradient 0, whatever its rows hold; the log-probabilities and rewards of a
 *     sequence or pair are reported all the same.
 *   - Precision.  The exponentials of a row of logits are fp32, and so are the
 *     sums of a thread and of 16 lanes; the joins of those, logarithms,
 *     log-probabilities, ratios and KL terms, clipping decisions, row weights and
 *     sums over rows are fp64, and a loss is rounded once.  A log-probability is
 *     off by about 1e-8 before it is rounded (up to 1e-7 where the scale puts
 *     log2(e) scale right above a power of two).  A gradient value is an fp32
 *     coefficient times an fp32 exponential, rounded to the logits' type.  A
 *     teacher's probabilities come from fp32 exponentials.  The balance loss is fp32
 *     within a row (softmax and f . p off by 1 to 2e-7 of themselves, a
 *     log-sum-exp by as much of the row's maximum) and fp64 over rows.
 *   - Same inputs at the same addresses modulo 128 bytes, same bits: no result
 *     depends on an order of atomics.
 *   - Every call enqueues kernels only and returns without waiting; it can be
 *     captured in a graph.  Calls that overlap need workspaces of their own,
 *     and a captured call's workspace has to outlive its graph.
 */
#ifndef SINKHORN_LOSSES_H
#define SINKHORN_LOSSES_H

#include <stddef.h>
#include <stdint.h>

#include "sinkhorn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Operation ids for sinkhorn_losses_workspace_bytes(). */
enum {
    SK_OP_TOKEN_LOGPROBS = 0,
    SK_OP_POLICY_LOSS = 1,
    SK_OP_PREFERENCE_LOSS = 2,
    SK_OP_DISTILL_LOSS = 3,
    SK_OP_BALANCE_LOSS = 4
};

/* Flags. */
#define SK_LOSS_MEAN 1u          /* a sequence's sum is divided by its number of labels */
#define SK_LOSS_FILL 2u          /* rows outside every sequence get zeros */
#define SK_LOSS_ROW_ADVANTAGE 4u /* adv is [T], one per row, instead of one per sequence */

/* Kinds of preference loss. */
enum { SK_PREFERENCE_SIGMOID = 0, SK_PREFERENCE_SQUARE = 1 };

/*
 * Workspace bytes of an operation (0 if the arguments are out of range): T rows
 * of V values (V = E for the balance loss), k = the teacher's K for the
 * distillation, the number of groups G for the balance loss, else 0.  No
 * initialisation needed; contents undefined after a call.
 */
size_t sinkhorn_losses_workspace_bytes(int op, int T, int V, int k, int dtype);

/*
 * Log-probabilities of tokens: with s = scale (an inverse temperature, from
 * 1e-20 to 1e20 here and below),
 *     logp[t] = s z_{t,labels[t]} - lse[t],   lse[t] = log sum_v exp(s z_tv).
 * Either output may be NULL (not both).  A row without a distribution has
 * logp 0 and lse -inf.
 */
int sinkhorn_token_logprobs(const void *logits, int dtype, int64_t ld, const int32_t *labels,
                            int T, int V, double scale, float *logp, float *lse,
                            void *ws, size_t ws_bytes, void *stream);

/*
 * Its gradient from grad [T] = dL/dlogp:
 *     dlogits[t][v] = grad[t] s (1[v = labels[t]] - exp(s z_tv - lse[t])).
 * With grad = -1/T this is the gradient of the mean cross-entropy.  The row's
 * softmax is found again on the way (the row is read once), so no rounded lse
 * enters.  A row of grad 0 is not read; its gradient is 0.  Workspace as for
 * SK_OP_TOKEN_LOGPROBS.
 */
int sinkhorn_token_logprobs_backward(const void *logits, int dtype, int64_t ld,
                                     const int32_t *labels, const float *grad, int T, int V,
                                     double scale, void *dlogits, int64_t dld,
                                     void *ws, size_t ws_bytes, void *stream);

/*
 * Clipped policy loss with a KL term, and its gradient in the logits, in one
 * pass over them.  Per scored row, logp as above, A = adv[i] of its sequence i
 * (adv[t] with SK_LOSS_ROW_ADVANTAGE), r = exp(logp - old[t]):
 *     l_t  = -min(r A, clip(r, 1 - clip_lo, 1 + clip_hi) A) + kl_coef k_t,
 *     k_t  = exp(d) - d - 1,  d = ref[t] - logp   (0 without ref),
 *     loss[i] = w_i sum_t l_t,   kl[i] = w_i sum_t k_t   over sequence i,
 * w_i = weights[i] (1 if NULL), divided by the sequence's number of labels with
 * SK_LOSS_MEAN.  At a border (r = 1 - clip_lo or 1 + clip_hi exactly) the row
 * is not clipped.  0 <= clip_lo < 1, clip_hi >= 0 (infinite: never), and
 * kl_coef finite (0: kl is reported alone).  loss, kl: [n]; logp [T] may be NULL.
 */
int sinkhorn_policy_loss(const void *logits, int dtype, int64_t ld, const int32_t *labels,
                         int T, int V, const int64_t *offsets, int n,
                         const float *old, const float *adv, const float *ref,
                         const float *weights, double scale, double clip_lo, double clip_hi,
                         double kl_coef, unsigned flags, float *loss, float *kl, float *logp,
                         void *dlogits, int64_t dld, void *ws, size_t ws_bytes, void *stream);

/*
 * Preference loss of pairs: sequence 2i is the preferred one of pair i and
 * sequence 2i + 1 the other (offsets has 2 pairs + 1 entries).  With
 *     R_j = sum_t (logp_t - ref[t]) over the scored rows of sequence j
 * (ref may be NULL: 0; with SK_LOSS_MEAN the mean over them, here without the
 * rows that have no distribution), D_i = R_2i - R_2i+1:
 *     sigmoid: loss[i] = w_i (-(1 - eps) log sigma(beta D) - eps log sigma(-beta D)),
 *     square:  loss[i] = w_i (D - 1 / (2 beta))^2,
 * eps = smoothing in [0, 1], beta > 0, w_i = weights[i] (1 if NULL).
 * reward [2 pairs] receives beta R_j, logp [T] the log-probabilities (needed).
 * The gradient needs the whole sequence, so the logits are read twice.
 */
int sinkhorn_preference_loss(const void *logits, int dtype, int64_t ld, const int32_t *labels,
                             int T, int V, const int64_t *offsets, int pairs,
                             const float *ref, const float *weights, double scale, int kind,
                             double beta, double smoothing, unsigned flags, float *loss,
                             float *reward, float *logp, void *dlogits, int64_t dld,
                             void *ws, size_t ws_bytes, void *stream);

/*
 * Distillation from a teacher's top logits: teacher [T][K] fp32 at tokens index
 * [T][K] (1 <= K <= 1024), tau = temperature > 0, q = softmax(z / tau) over the
 * whole row,
 *     p_k = exp(teacher_k / tau - U),  U = log sum_k exp(teacher_k / tau), or
 *           teacher_lse[t], the teacher's log-sum-exp of logits / tau over its
 *           whole vocabulary (may be NULL),
 *     loss[t] = w_t tau^2 sum_k p_k (log p_k - log q_{index_k}),
 *     dlogits[t][v] = w_t tau (q_v sum_k p_k - sum_{k: index_k = v} p_k),
 * w_t = weights[t] (1 if NULL).  A row of weight 0 is not read; its loss and
 * gradient are 0.  A negative index, or a teacher logit of -inf, is no entry; a
 * row without entries has loss and gradient 0.  A token may stand in the list
 * more than once.  An index of V or more, or a teacher logit of NaN or +inf,
 * makes the row NaN.
 */
int sinkhorn_distill_loss(const void *logits, int dtype, int64_t ld, int T, int V,
                          const int32_t *index, const float *teacher, int K,
                          const float *teacher_lse, const float *weights, double temperature,
                          float *loss, void *dlogits, int64_t dld,
                          void *ws, size_t ws_bytes, void *stream);

/*
 * Balance loss of an expert router and its counts.  logits [T][E] (E <= 1024),
 * index [T][K] the experts each row was sent to (K <= 64; negative: none), p =
 * softmax of a row.  Per group g of rows (offsets [G + 1] as above; NULL with
 * G = 1: every row), n = its rows with at least one index:
 *     counts[g][e] = how often e stands in the group's indices,
 *     f_e = E counts[g][e] / (K n),
 *     loss[g]  = (1/n) sum_t sum_e f_e p_te,      zloss[g] = (1/n) sum_t lse_t^2,
 *     dlogits  = d(balance loss[g] + z zloss[g]) with the counts held fixed.
 * A row without an index takes no part (gradient 0); one whose logits are all
 * -inf counts in n and counts alone.  loss and zloss [G] are without their
 * coefficients.  An index of E or more is left out of the counts and makes the
 * group's balance loss and its rows' gradients NaN.
 */
int sinkhorn_balance_loss(const void *logits, int dtype, int64_t ld, int T, int E,
                          const int32_t *index, int K, const int64_t *offsets, int G,
                          double balance, double z, unsigned flags, float *loss, float *zloss,
                          int32_t *counts, void *dlogits, int64_t dld,
                          void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SINKHORN_LOSSES_H */
