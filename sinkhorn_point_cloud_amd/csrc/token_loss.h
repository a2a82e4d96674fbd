// token_loss.h -- arguments and launchers of the losses over rows of logits
// (token_loss.hip, distill.hip), shared with the ABI (abi_losses.hip).
#pragma once

#include "common.h"

namespace sk {

// Rows of logits and, where a gradient is asked for, of its output.
struct LogitRows {
    const void *logits;
    int64_t ld;          // elements from one row to the next
    int dtype, T, V;
    double scale;        // the softmax is over scale * logits
    void *dlogits;       // NULL: no gradient
    int64_t dld;
};

// Packed sequences: rows [offsets[i], offsets[i + 1]) are sequence i.
struct Packed {
    const int64_t *offsets;   // [n + 1], or NULL: every row counts, no sequences
    int n;
    int fill;                 // rows outside every sequence get zeros (else are left alone)
};

// How many work-groups share a row, and whether a row's statistics and its
// gradient are one launch (parts == 1) or two.
int token_parts(int T, int V, int dtype);
// work-groups a row's gradient is dealt to where the statistics are known
int grad_parts(int T, int V, int dtype);

// (maximum, rest) of a part of a row: of a wave, or of a work-group.
struct RowPart {
    double r;
    float m;
};

struct TokenWs {
    RowPart *part;   // [T][parts] the parts' (maximum, rest); parts > 1 only
    float *zlab;     // [T] label's logit; parts > 1 only
};

// What a row's statistics leave for a later pass: its maximum, the rest of its
// sum (rounded to fp32, as the gradient's coefficient will be) and the label's
// log-probability before it is rounded.
struct RowStat {
    float M, R;
    double logp;
};

// Per row, each may be NULL.
struct LogpOut {
    float *logp, *lse;
    RowStat *stat;
};
hipError_t launch_logp(const LogitRows &r, const int32_t *labels, const Packed &p,
                       const TokenWs &w, const LogpOut &out, hipStream_t st);

// dlogits = G_t scale (1[v = label] - softmax), the softmax found on the way
hipError_t launch_logp_backward(const LogitRows &r, const int32_t *labels, const float *G,
                                const TokenWs &w, hipStream_t st);

// What a row needs of its sequence: its weight there, and the advantage.
struct PolicyRow {
    double w;
    float adv;
};
struct PolicyArgs {
    const float *old, *ref, *adv, *weights;
    int adv_per_token, mean;
    double lo, hi, log_lo, log_hi, kl;
    PolicyRow *info;   // [T] scratch, where it is found beforehand
    double2 *term;     // [T] scratch: weighted loss and KL of a row
    float *loss, *kl_out, *logp;
};
hipError_t launch_policy(const LogitRows &r, const int32_t *labels, const Packed &p,
                         const PolicyArgs &a, const TokenWs &w, hipStream_t st);

struct PreferenceArgs {
    const float *ref, *weights;
    int kind, mean;
    double beta, smoothing;
    float *coef;    // [T] scratch: dloss/dlogp of a row, one rounding of the gradient's own
    RowStat *stat;  // [T] scratch
    float *loss, *reward, *logp;
};
hipError_t launch_preference(const LogitRows &r, const int32_t *labels, const Packed &p,
                             const PreferenceArgs &a, const TokenWs &w, hipStream_t st);

struct DistillArgs {
    const int32_t *index;
    const float *teacher, *teacher_lse, *weights;
    int K;
    float *zk;      // [T][K] scratch: the student's logits at the teacher's tokens; parts > 1 only
    float *loss;
};
hipError_t launch_distill(const LogitRows &r, const DistillArgs &a, const TokenWs &w,
                          hipStream_t st);

// Router logits [T][E] with the chosen experts [T][K].
struct BalanceArgs {
    const void *logits;
    int64_t ld;
    int dtype, T, E, K;
    const int32_t *index;
    const int64_t *offsets;   // [G + 1] or NULL: one group of every row
    int G, fill;
    double balance, z;
    float *loss, *zloss;
    int32_t *counts;
    void *dlogits;
    int64_t dld;
};
// Chunks of rows within a group: the pieces of work of the two passes.
struct BalanceWs {
    int32_t *count_part;   // [count chunks][E + 2]: tokens per expert, rows, bad indices
    double *sum_part;      // [gradient chunks][2]: sums of f . p and of the squared log-sum-exp
    int32_t *rows;         // [G] rows that take part
    long count_chunks, grad_chunks;
};
long balance_count_chunks(int T, int G);
long balance_grad_chunks(int T, int G);
hipError_t launch_balance(const BalanceArgs &a, const BalanceWs &w, hipStream_t st);

constexpr int kMaxTopK = 1024;
constexpr int kMaxExperts = 1024;
constexpr int kMaxChosen = 64;

}  // namespace sk
