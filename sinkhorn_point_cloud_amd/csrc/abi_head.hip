// abi_head.hip -- the C ABI declared in include/sinkhorn_head.h: argument checks,
// workspace carve-up and launches of the output end of a model.
#include "abi.h"
#include "head.h"
#include "sinkhorn_head.h"

#include <initializer_list>
#include <math.h>

namespace sk {
namespace {

constexpr int kMaxRows = 1 << 24;
constexpr int64_t kMaxStride = 1ll << 38;
constexpr int64_t kMaxSpan = 1ll << 58;
constexpr int64_t kMaxResults = 1ll << 37;   // 2^23 tiles of 128 x 128

size_t elem(int dtype) { return dtype == SK_BF16 ? 2 : 4; }

// Rows of a matrix in bytes, `distance` from one to the next; at == NULL: not given.
struct Rows {
    const char *name;
    const void *at;
    uint64_t rows, bytes, distance;
    uintptr_t first() const { return (uintptr_t)at; }
    uintptr_t end() const { return first() + (rows - 1) * distance + bytes; }
};

Rows rows_of(const char *name, const void *at, int64_t rows, int64_t len, int64_t ld, size_t size)
{
    return Rows{name, at, (uint64_t)rows, (uint64_t)len * size,
                rows > 1 ? (uint64_t)ld * size : (uint64_t)len * size};
}
Rows array_of(const char *name, const void *at, uint64_t bytes)
{
    return Rows{name, at, 1, bytes, bytes};
}

bool same(const Rows &a, const Rows &b)
{
    return a.at == b.at && a.rows == b.rows && a.bytes == b.bytes && a.distance == b.distance;
}

// Whether two share memory.  Rows of one distance may be columns side by side; of
// two matrices of other distances the hulls decide, a run of bytes has to lie
// within the gap of two rows.
bool meet(const Rows &a, const Rows &b)
{
    if (!a.at || !b.at || !a.rows || !b.rows || !a.bytes || !b.bytes)
        return false;
    if (a.end() <= b.first() || b.end() <= a.first())
        return false;
    if (a.rows == 1 || b.rows == 1 || a.distance == b.distance) {
        const Rows &m = a.rows > 1 ? a : b, &o = a.rows > 1 ? b : a;
        if (m.rows == 1)
            return true;
        // where o begins, from the row of m at or before it
        const int64_t gap = (int64_t)(o.first() - m.first()), ld = (int64_t)m.distance;
        const uint64_t in = (uint64_t)(((gap % ld) + ld) % ld);
        return in < m.bytes || in + o.bytes > m.distance;
    }
    return true;
}

// Outputs lie apart from inputs and from one another, but for an input that an
// output may be itself (`own`, a bit for each input).
struct Output {
    Rows rows;
    unsigned own;
};
int check_apart(std::initializer_list<Rows> inputs, std::initializer_list<Output> outputs)
{
    auto refuse = [](const Rows &a, const Rows &b) {
        return fail(SK_ERR_INVALID_ARG, "%s and %s overlap", a.name, b.name);
    };
    for (const Output *o = outputs.begin(); o != outputs.end(); ++o) {
        unsigned bit = 1;
        for (const Rows &i : inputs) {
            if (meet(o->rows, i) && !((o->own & bit) && same(o->rows, i)))
                return refuse(o->rows, i);
            bit <<= 1;
        }
        for (const Output *p = outputs.begin(); p != o; ++p)
            if (meet(o->rows, p->rows))
                return refuse(o->rows, p->rows);
    }
    return SK_OK;
}

int check_dtype(int dtype)
{
    if (dtype != SK_F32 && dtype != SK_BF16)
        return fail(SK_ERR_INVALID_ARG, "dtype %d is neither SK_F32 nor SK_BF16", dtype);
    return SK_OK;
}

int check_sizes(int T, int len, int most)
{
    if (T < 0 || T > kMaxRows || len < 1 || len > most)
        return fail(SK_ERR_INVALID_ARG, "bad sizes: %d rows of %d values (at most %d of %d)", T,
                    len, kMaxRows, most);
    return SK_OK;
}

// A matrix of a call: row distance, alignment, and that it is there.
int check_matrix(const char *name, const void *at, int64_t T, int64_t len, int64_t ld, size_t align,
                 bool needed)
{
    if (!at)
        return needed && T > 0
                   ? fail(SK_ERR_INVALID_ARG, "%s must be a non-NULL device pointer", name)
                   : SK_OK;
    if (ld < len || ld > kMaxStride || T * ld > kMaxSpan)
        return fail(SK_ERR_INVALID_ARG, "%s: %lld rows of %lld values cannot be %lld elements apart",
                    name, (long long)T, (long long)len, (long long)ld);
    if ((uintptr_t)at % align)
        return fail(SK_ERR_INVALID_ARG, "%s are not aligned to %zu bytes", name, align);
    return SK_OK;
}

int check_space(const void *ws, size_t ws_bytes, size_t need)
{
    if (!ws || ws_bytes < need)
        return fail(SK_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given%s", need, ws_bytes,
                    ws ? "" : " (ws is NULL)");
    return SK_OK;
}

int check_scale(double scale)
{
    if (!(scale >= 1e-20 && scale <= 1e20))
        return fail(SK_ERR_INVALID_ARG, "scale=%g must be in [1e-20, 1e20]", scale);
    return SK_OK;
}

int check_eps(double eps)
{
    if (!(eps >= 1e-30 && eps <= 1e30))
        return fail(SK_ERR_INVALID_ARG, "eps=%g must be in [1e-30, 1e30]", eps);
    return SK_OK;
}

struct Ws {
    float *norm = nullptr;
    int32_t *product = nullptr;
    ScorePart *part = nullptr;
    uint64_t *list = nullptr;
    float *zlab = nullptr;
};

Ws carve(Carve &c, int op, int T, int V, int k, int dtype)
{
    Ws w;
    if (op == SK_OP_RMS_NORM_BACKWARD) {
        w.norm = c.take<float>((size_t)norm_groups(T, V, dtype) * V);
    } else if (op == SK_OP_INT8_LINEAR) {
        const int parts = product_parts(T, k, V);
        if (parts > 1)
            w.product = c.take<int32_t>((size_t)parts * T * V);
    } else {
        const int parts = score_parts(T, V, dtype);
        if (parts > 1) {
            w.part = c.take<ScorePart>((size_t)T * parts);
            w.zlab = c.take<float>(T);
            w.list = c.take<uint64_t>((size_t)T * parts * k);
        }
    }
    return w;
}

size_t ws_bytes_of(int op, int T, int V, int k, int dtype)
{
    Carve c{nullptr};
    carve(c, op, T, V, k, dtype);
    return c.off + 256;
}

bool sizes_ok(int op, int T, int V, int k)
{
    if (T < 0 || T > kMaxRows || V < 1)
        return false;
    switch (op) {
    case SK_OP_RMS_NORM_BACKWARD: return V <= kMaxNormRow;
    case SK_OP_INT8_LINEAR:
        return V <= kMaxRows && k >= 1 && k <= kMaxProductK && (int64_t)T * V <= kMaxResults;
    case SK_OP_TOKEN_SCORES: return V <= kMaxRows && k >= 0 && k <= kMaxTop;
    default: return V <= kMaxRows && k == 0;
    }
}

// What the three forms of the norm have in common.
int check_norm(const NormArgs &a)
{
    const size_t size = elem(a.dtype);
    int rc;
    if ((rc = check_dtype(a.dtype)) || (rc = check_sizes(a.T, a.d, kMaxNormRow)) ||
        (rc = check_matrix("x", a.x, a.T, a.d, a.ldx, size, true)) ||
        (rc = check_matrix("residual", a.residual, a.T, a.d, a.ldr, size, false)) ||
        (rc = check_matrix("h", a.h, a.T, a.d, a.ldh, size, false)) ||
        (rc = check_matrix("weight", a.weight, 1, a.d, a.d, size, false)) ||
        (a.norm && (rc = check_eps(a.eps))))
        return rc;
    if (a.scale || a.q) {
        if ((rc = check_matrix("q", a.q, a.T, a.d, a.ldq, 1, true)) ||
            (rc = check_matrix("scale", a.scale, 1, a.T, a.T, 4, a.T > 0)))
            return rc;
    } else if ((rc = check_matrix("y", a.y, a.T, a.d, a.ldy, size, true))) {
        return rc;
    }
    if (a.T == 0)
        return SK_OK;
    return check_apart({rows_of("x", a.x, a.T, a.d, a.ldx, size),
                        rows_of("residual", a.residual, a.T, a.d, a.ldr, size),
                        array_of("weight", a.weight, a.d * size)},
                       {{rows_of("y", a.y, a.T, a.d, a.ldy, size), 3},
                        {rows_of("h", a.h, a.T, a.d, a.ldh, size), 3},
                        {rows_of("q", a.q, a.T, a.d, a.ldq, 1), 0},
                        {array_of("scale", a.scale, (uint64_t)a.T * 4), 0}});
}

// Rows of logits and what both directions check of them.
int check_logits(const void *logits, int dtype, int64_t ld, const int32_t *labels, int T, int V,
                 double scale)
{
    int rc;
    if ((rc = check_dtype(dtype)) || (rc = check_sizes(T, V, kMaxRows)) ||
        (rc = check_matrix("logits", logits, T, V, ld, elem(dtype), true)) ||
        (rc = check_scale(scale)))
        return rc;
    return check_matrix("labels", labels, 1, T, T, 4, false);
}

}  // namespace
}  // namespace sk

using namespace sk;

extern "C" {

size_t sinkhorn_head_workspace_bytes(int op, int T, int V, int k, int dtype)
{
    if (op < SK_OP_RMS_NORM_BACKWARD || op > SK_OP_TOKEN_SCORES_BACKWARD ||
        (dtype != SK_F32 && dtype != SK_BF16) || !sizes_ok(op, T, V, k))
        return 0;
    return ws_bytes_of(op, T, V, k, dtype);
}

int sinkhorn_rms_norm(const void *x, int dtype, int64_t ldx, const void *residual, int64_t ldr,
                      const void *weight, int T, int d, double eps, void *y, int64_t ldy, void *h,
                      int64_t ldh, void *stream)
{
    clear_error();
    NormArgs a{x, residual, weight, ldx, ldr, dtype, T, d, eps, y, ldy, nullptr, 0, nullptr, 1, h, ldh};
    const int rc = check_norm(a);
    if (rc || T == 0)
        return rc;
    const hipError_t e = launch_norm(a, (hipStream_t)stream);
    return e ? hip_fail(e, "norm") : SK_OK;
}

int sinkhorn_rms_norm_int8(const void *x, int dtype, int64_t ldx, const void *residual,
                           int64_t ldr, const void *weight, int T, int d, double eps, int8_t *q,
                           int64_t ldq, float *scale, void *h, int64_t ldh, void *stream)
{
    clear_error();
    if (T > 0 && (!q || !scale))
        return fail(SK_ERR_INVALID_ARG, "q and scale must be non-NULL");
    NormArgs a{x, residual, weight, ldx, ldr, dtype, T, d, eps, nullptr, 0, q, ldq, scale, 1, h, ldh};
    const int rc = check_norm(a);
    if (rc || T == 0)
        return rc;
    const hipError_t e = launch_norm(a, (hipStream_t)stream);
    return e ? hip_fail(e, "norm in 8 bits") : SK_OK;
}

int sinkhorn_quantize_int8(const void *x, int dtype, int64_t ldx, int T, int d, int8_t *q,
                           int64_t ldq, float *scale, void *stream)
{
    clear_error();
    if (T > 0 && (!q || !scale))
        return fail(SK_ERR_INVALID_ARG, "q and scale must be non-NULL");
    NormArgs a{x, nullptr, nullptr, ldx, 0, dtype, T, d, 0.0, nullptr, 0, q, ldq, scale, 0, nullptr, 0};
    const int rc = check_norm(a);
    if (rc || T == 0)
        return rc;
    const hipError_t e = launch_norm(a, (hipStream_t)stream);
    return e ? hip_fail(e, "8 bits") : SK_OK;
}

int sinkhorn_rms_norm_backward(const void *dy, int dtype, int64_t lddy, const void *h, int64_t ldh,
                               const void *weight, const void *dh, int64_t lddh, int T, int d,
                               double eps, void *dx, int64_t lddx, float *dweight, void *ws,
                               size_t ws_bytes, void *stream)
{
    clear_error();
    int rc;
    if ((rc = check_dtype(dtype)))
        return rc;
    const size_t size = elem(dtype);
    if ((rc = check_sizes(T, d, kMaxNormRow)) || (rc = check_eps(eps)) ||
        (rc = check_matrix("dy", dy, T, d, lddy, size, true)) ||
        (rc = check_matrix("h", h, T, d, ldh, size, true)) ||
        (rc = check_matrix("dh", dh, T, d, lddh, size, false)) ||
        (rc = check_matrix("dx", dx, T, d, lddx, size, true)) ||
        (rc = check_matrix("weight", weight, 1, d, d, size, false)) ||
        (rc = check_matrix("dweight", dweight, 1, d, d, 4, false)))
        return rc;
    const size_t need = ws_bytes_of(SK_OP_RMS_NORM_BACKWARD, T, d, 0, dtype);
    if ((rc = check_space(ws, ws_bytes, need)))
        return rc;
    if ((rc = check_apart({rows_of("dy", dy, T, d, lddy, size), rows_of("h", h, T, d, ldh, size),
                           rows_of("dh", dh, T, d, lddh, size),
                           array_of("weight", weight, d * size)},
                          {{rows_of("dx", dx, T, d, lddx, size), 7},
                           {array_of("dweight", dweight, (uint64_t)d * 4), 0},
                           {array_of("ws", ws, need), 0}})))
        return rc;
    if (T == 0 && !dweight)   // else it gets zeros
        return SK_OK;
    Carve c{(char *)ws};
    const Ws w = carve(c, SK_OP_RMS_NORM_BACKWARD, T, d, 0, dtype);
    const NormGradArgs a{dy, h, weight, dh, lddy, ldh, lddh, dtype, T, d, eps, dx, lddx, dweight, w.norm};
    const hipError_t e = launch_norm_backward(a, (hipStream_t)stream);
    return e ? hip_fail(e, "norm backward") : SK_OK;
}

int sinkhorn_int8_linear(const int8_t *x, int64_t ldx, const float *xscale, const int8_t *w,
                         int64_t ldw, const float *wscale, const float *bias, int T, int K, int N,
                         int dtype, void *out, int64_t ldo, void *ws, size_t ws_bytes, void *stream)
{
    clear_error();
    int rc;
    if ((rc = check_dtype(dtype)) || (rc = check_sizes(T, K, kMaxProductK)) ||
        (rc = check_sizes(N, K, kMaxProductK)))
        return rc;
    if (N < 1)
        return fail(SK_ERR_INVALID_ARG, "N=%d must be at least 1", N);
    // beyond any memory, and beyond the work-groups of one launch
    if ((int64_t)T * N > kMaxResults)
        return fail(SK_ERR_INVALID_ARG, "%d rows of %d results are too many", T, N);
    if ((rc = check_matrix("x", x, T, K, ldx, 16, true)) ||
        (rc = check_matrix("w", w, N, K, ldw, 16, true)) ||
        (rc = check_matrix("xscale", xscale, 1, T, T, 4, T > 0)) ||
        (rc = check_matrix("wscale", wscale, 1, N, N, 4, true)) ||
        (rc = check_matrix("bias", bias, 1, N, N, 4, false)) ||
        (rc = check_matrix("out", out, T, N, ldo, elem(dtype), true)))
        return rc;
    if (T > 0 && (ldx % 16 || ldw % 16))
        return fail(SK_ERR_INVALID_ARG, "ldx=%lld and ldw=%lld must be multiples of 16",
                    (long long)ldx, (long long)ldw);
    const size_t need = ws_bytes_of(SK_OP_INT8_LINEAR, T, N, K, dtype);
    if ((rc = check_space(ws, ws_bytes, need)))
        return rc;
    if (T == 0)
        return SK_OK;
    if ((rc = check_apart({rows_of("x", x, T, K, ldx, 1), rows_of("w", w, N, K, ldw, 1),
                           array_of("xscale", xscale, (uint64_t)T * 4),
                           array_of("wscale", wscale, (uint64_t)N * 4),
                           array_of("bias", bias, (uint64_t)N * 4)},
                          {{rows_of("out", out, T, N, ldo, elem(dtype)), 0},
                           {array_of("ws", ws, need), 0}})))
        return rc;
    Carve c{(char *)ws};
    const Ws s = carve(c, SK_OP_INT8_LINEAR, T, N, K, dtype);
    const ProductArgs a{x, w, ldx, ldw, xscale, wscale, bias, T, K, N, dtype, out, ldo, s.product};
    const hipError_t e = launch_product(a, (hipStream_t)stream);
    return e ? hip_fail(e, "8-bit product") : SK_OK;
}

int sinkhorn_token_scores(const void *logits, int dtype, int64_t ld, const int32_t *labels, int T,
                          int V, double scale, int top, float *logp, float *lse, float *entropy,
                          int32_t *index, float *best, void *ws, size_t ws_bytes, void *stream)
{
    clear_error();
    int rc;
    if ((rc = check_logits(logits, dtype, ld, labels, T, V, scale)))
        return rc;
    if (top < 0 || top > kMaxTop)
        return fail(SK_ERR_INVALID_ARG, "top=%d must be in [0, %d]", top, kMaxTop);
    const uint64_t rows = (uint64_t)T * 4;
    for (const Rows &o : {array_of("logp", logp, rows), array_of("lse", lse, rows),
                          array_of("entropy", entropy, rows), array_of("index", index, rows * top),
                          array_of("best", best, rows * top)})
        if (o.first() % 4)
            return fail(SK_ERR_INVALID_ARG, "%s is not aligned to 4 bytes", o.name);
    if (T > 0) {
        if (!logp && !lse && !entropy && !index)
            return fail(SK_ERR_INVALID_ARG, "one of the outputs must be non-NULL");
        if (logp && !labels)
            return fail(SK_ERR_INVALID_ARG, "logp needs labels");
        if ((top > 0) != (index != nullptr) || (top > 0) != (best != nullptr))
            return fail(SK_ERR_INVALID_ARG, "top=%d needs %s", top,
                        top ? "index and best" : "neither index nor best");
    }
    const size_t need = ws_bytes_of(SK_OP_TOKEN_SCORES, T, V, top, dtype);
    if ((rc = check_space(ws, ws_bytes, need)))
        return rc;
    if (T == 0)
        return SK_OK;
    if ((rc = check_apart({rows_of("logits", logits, T, V, ld, elem(dtype)),
                           array_of("labels", labels, rows)},
                          {{array_of("logp", logp, rows), 0},
                           {array_of("lse", lse, rows), 0},
                           {array_of("entropy", entropy, rows), 0},
                           {array_of("index", index, rows * top), 0},
                           {array_of("best", best, rows * top), 0},
                           {array_of("ws", ws, need), 0}})))
        return rc;
    Carve c{(char *)ws};
    const Ws w = carve(c, SK_OP_TOKEN_SCORES, T, V, top, dtype);
    const ScoreArgs a{logits, ld, dtype, T, V, top, scale, labels, logp, lse, entropy, index, best,
                      nullptr, nullptr, nullptr, 0, w.part, w.list, w.zlab};
    const hipError_t e = launch_scores(a, (hipStream_t)stream);
    return e ? hip_fail(e, "token scores") : SK_OK;
}

int sinkhorn_token_scores_backward(const void *logits, int dtype, int64_t ld,
                                   const int32_t *labels, const float *grad,
                                   const float *grad_entropy, int T, int V, double scale,
                                   void *dlogits, int64_t dld, void *ws, size_t ws_bytes,
                                   void *stream)
{
    clear_error();
    int rc;
    if ((rc = check_logits(logits, dtype, ld, labels, T, V, scale)) ||
        (rc = check_matrix("grad", grad, 1, T, T, 4, false)) ||
        (rc = check_matrix("grad_entropy", grad_entropy, 1, T, T, 4, false)) ||
        (rc = check_matrix("dlogits", dlogits, T, V, dld, elem(dtype), true)))
        return rc;
    if (T > 0 && !grad && !grad_entropy)
        return fail(SK_ERR_INVALID_ARG, "one of grad and grad_entropy must be non-NULL");
    if (T > 0 && grad && !labels)
        return fail(SK_ERR_INVALID_ARG, "grad needs labels");
    const size_t need = ws_bytes_of(SK_OP_TOKEN_SCORES_BACKWARD, T, V, 0, dtype);
    if ((rc = check_space(ws, ws_bytes, need)))
        return rc;
    if (T == 0)
        return SK_OK;
    const uint64_t rows = (uint64_t)T * 4;
    if ((rc = check_apart({rows_of("logits", logits, T, V, ld, elem(dtype)),
                           array_of("labels", labels, rows), array_of("grad", grad, rows),
                           array_of("grad_entropy", grad_entropy, rows)},
                          {{rows_of("dlogits", dlogits, T, V, dld, elem(dtype)), 1},
                           {array_of("ws", ws, need), 0}})))
        return rc;
    Carve c{(char *)ws};
    const Ws w = carve(c, SK_OP_TOKEN_SCORES_BACKWARD, T, V, 0, dtype);
    const ScoreArgs a{logits, ld, dtype, T, V, 0, scale, labels, nullptr, nullptr, nullptr, nullptr,
                      nullptr, grad, grad_entropy, dlogits, dld, w.part, w.list, w.zlab};
    const hipError_t e = launch_scores_backward(a, (hipStream_t)stream);
    return e ? hip_fail(e, "token scores backward") : SK_OK;
}

}  // extern "C"
