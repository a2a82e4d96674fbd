// head.h -- arguments and launchers of the output end of a model (norm.hip,
// int8_linear.hip, scores.hip), shared with the ABI (abi_head.hip).
#pragma once

#include "common.h"

namespace sk {

constexpr int kMaxNormRow = 32768;
constexpr int kMaxProductK = 131071;   // (-128)^2 K stays below 2^31
constexpr int kMaxTop = 128;

struct NormArgs {
    const void *x, *residual, *weight;   // residual, weight: NULL for none
    int64_t ldx, ldr;
    int dtype, T, d;
    double eps;
    void *y;             // the norm in x's type, or
    int64_t ldy;
    int8_t *q;           // in 8 bits with
    int64_t ldq;
    float *scale;        // [T]
    int norm;            // 0: 8 bits of x itself
    void *h;             // NULL: the sum is not kept
    int64_t ldh;
};
hipError_t launch_norm(const NormArgs &a, hipStream_t st);

struct NormGradArgs {
    const void *dy, *h, *weight, *dh;    // weight, dh: NULL for none
    int64_t lddy, ldh, lddh;
    int dtype, T, d;
    double eps;
    void *dx;
    int64_t lddx;
    float *dweight;      // [d], NULL: none
    float *part;         // [norm_groups][d] scratch: dweight of each group of rows
};
int norm_groups(int T, int d, int dtype);
hipError_t launch_norm_backward(const NormGradArgs &a, hipStream_t st);

struct ProductArgs {
    const int8_t *x, *w;
    int64_t ldx, ldw;
    const float *xscale, *wscale, *bias;
    int T, K, N, dtype;
    void *out;
    int64_t ldo;
    int32_t *part;       // [product_parts][T][N] scratch where the K axis is split over work-groups
};
int product_parts(int T, int K, int N);
hipError_t launch_product(const ProductArgs &a, hipStream_t st);

// (maximum, rest, weighted distance) of a part of a row.
struct ScorePart {
    double r, w;
    float m;
};
struct ScoreArgs {
    const void *logits;
    int64_t ld;
    int dtype, T, V, top;
    double scale;
    const int32_t *labels;
    float *logp, *lse, *entropy;
    int32_t *index;
    float *best;
    // the gradient
    const float *grad, *grad_entropy;
    void *dlogits;
    int64_t dld;
    // scratch where a row is dealt to several work-groups
    ScorePart *part;     // [T][parts]
    uint64_t *list;      // [T][parts][top] the parts' alternatives
    float *zlab;         // [T]
};
int score_parts(int T, int V, int dtype);
hipError_t launch_scores(const ScoreArgs &a, hipStream_t st);
hipError_t launch_scores_backward(const ScoreArgs &a, hipStream_t st);

}  // namespace sk
