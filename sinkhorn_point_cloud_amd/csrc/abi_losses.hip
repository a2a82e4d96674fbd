// abi_losses.hip -- the C ABI declared in include/sinkhorn_losses.h: argument
// checks, workspace carve-up and launches of the losses over rows of logits.
#include "abi.h"
#include "common.h"
#include "sinkhorn_losses.h"
#include "token_loss.h"

#include <initializer_list>
#include <math.h>

namespace sk {
namespace {

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxSequences = 1 << 20;   // a work-group of 1024 threads each: 2^30 in a launch
constexpr int64_t kMaxStride = 1ll << 38;
constexpr int64_t kMaxSpan = 1ll << 58;      // elements: 2^60 bytes, beyond any address space

size_t elem(int dtype) { return dtype == SK_BF16 ? 2 : 4; }

struct Ws {
    TokenWs token{};
    PolicyRow *info = nullptr;
    double2 *term = nullptr;
    RowStat *stat = nullptr;
    float *coef = nullptr, *zk = nullptr;
    BalanceWs balance{};
};

Ws carve(Carve &c, int op, int T, int V, int k, int dtype)
{
    Ws w;
    const size_t rows = (size_t)T;
    if (op == SK_OP_BALANCE_LOSS) {
        w.balance.count_chunks = balance_count_chunks(T, k);
        w.balance.grad_chunks = balance_grad_chunks(T, k);
        w.balance.count_part = c.take<int32_t>((size_t)w.balance.count_chunks * (V + 2));
        w.balance.sum_part = c.take<double>((size_t)w.balance.grad_chunks * 2);
        w.balance.rows = c.take<int32_t>(k);
        return w;
    }
    const int parts = token_parts(T, V, dtype);
    if (parts > 1) {
        w.token.part = c.take<RowPart>(rows * parts);
        if (op == SK_OP_DISTILL_LOSS)
            w.zk = c.take<float>(rows * k);
        else
            w.token.zlab = c.take<float>(rows);
    }
    if (op == SK_OP_POLICY_LOSS) {
        w.info = c.take<PolicyRow>(rows);
        w.term = c.take<double2>(rows);
    } else if (op == SK_OP_PREFERENCE_LOSS) {
        w.stat = c.take<RowStat>(rows);
        w.coef = c.take<float>(rows);
    }
    return w;
}

bool sizes_ok(int op, int T, int V, int k)
{
    if (T < 0 || T > kMaxRows || V < 1)
        return false;
    if (op == SK_OP_BALANCE_LOSS)
        return V <= kMaxExperts && k >= 1 && k <= kMaxSequences;
    return V <= kMaxRows && (op != SK_OP_DISTILL_LOSS || (k >= 1 && k <= kMaxTopK));
}

size_t ws_bytes_of(int op, int T, int V, int k, int dtype)
{
    Carve c{nullptr};
    carve(c, op, T, V, k, dtype);
    return c.off + 256;
}

int check_rows(const void *logits, int dtype, int64_t ld, int T, int V, int max_V)
{
    if (dtype != SK_F32 && dtype != SK_BF16)
        return fail(SK_ERR_INVALID_ARG, "dtype %d is neither SK_F32 nor SK_BF16", dtype);
    if (T < 0 || T > kMaxRows || V < 1 || V > max_V)
        return fail(SK_ERR_INVALID_ARG, "bad sizes: %d rows of %d values (at most %d of %d)", T,
                    V, kMaxRows, max_V);
    if (T > 0 && !logits)
        return fail(SK_ERR_INVALID_ARG, "logits must be a non-NULL device pointer");
    if (ld < V || ld > kMaxStride || T * ld > kMaxSpan)
        return fail(SK_ERR_INVALID_ARG, "%d rows of %d values cannot be %lld elements apart",
                    T, V, (long long)ld);
    if ((uintptr_t)logits % elem(dtype))
        return fail(SK_ERR_INVALID_ARG, "logits are not aligned to their type");
    return SK_OK;
}

// dlogits may be the logits themselves, or lie apart from them.
int check_grad(const void *logits, int64_t ld, const void *dlogits, int64_t dld, int dtype, int T,
               int V)
{
    if (!dlogits || T == 0)
        return SK_OK;
    const int64_t size = (int64_t)elem(dtype);
    if (dld < V || dld > kMaxStride || T * dld > kMaxSpan)
        return fail(SK_ERR_INVALID_ARG, "%d gradient rows of %d values cannot be %lld elements apart",
                    T, V, (long long)dld);
    if ((uintptr_t)dlogits % (uintptr_t)size)
        return fail(SK_ERR_INVALID_ARG, "dlogits are not aligned to their type");
    const int64_t a = (int64_t)(uintptr_t)logits, b = (int64_t)(uintptr_t)dlogits;
    if (a == b && (ld == dld || T == 1))
        return SK_OK;
    const int64_t a1 = a + ((T - 1) * ld + V) * size, b1 = b + ((T - 1) * dld + V) * size;
    if (a1 <= b || b1 <= a)
        return SK_OK;
    if (ld == dld && (a - b) % size == 0) {
        // columns of one buffer side by side
        const int64_t off = (((b - a) / size) % ld + ld) % ld;
        if (off >= V && ld - off >= V)
            return SK_OK;
    }
    return fail(SK_ERR_INVALID_ARG,
                "dlogits overlap the logits without being them (same address and row distance)");
}

// The range in which both pieces of scale log2(e) are ordinary fp32 numbers.
int check_scale(double scale, const char *what)
{
    if (!(scale >= 1e-20 && scale <= 1e20))
        return fail(SK_ERR_INVALID_ARG, "%s=%g must be in [1e-20, 1e20]", what, scale);
    return SK_OK;
}

int check_packed(const int64_t *offsets, int n, unsigned flags, unsigned known)
{
    if (!offsets || n < 1 || n > kMaxSequences)
        return fail(SK_ERR_INVALID_ARG, "%d sequences need 1 <= n <= %d and device offsets", n,
                    kMaxSequences);
    if (flags & ~known)
        return fail(SK_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    return SK_OK;
}

int check_space(const void *ws, size_t ws_bytes, size_t need)
{
    if (!ws || ws_bytes < need)
        return fail(SK_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given%s", need,
                    ws_bytes, ws ? "" : " (ws is NULL)");
    return SK_OK;
}

// An array of a call (at == NULL: not given).
struct Span {
    const char *name;
    const void *at;
    size_t bytes;
    uintptr_t first() const { return (uintptr_t)at; }
    uintptr_t end() const { return first() + bytes; }
};

// Rows of a matrix, `distance` bytes from one to the next; what lies between them is
// another's.
struct Rows {
    const char *name;
    const void *at;
    uint64_t rows, bytes, distance;
};

bool meet(const Span &a, const Span &b)
{
    return a.at && b.at && a.bytes && b.bytes && a.first() < b.end() && b.first() < a.end();
}

bool meet(const Span &a, const Rows &r)
{
    if (!a.at || !a.bytes || !r.at || !r.rows)
        return false;
    const uintptr_t first = (uintptr_t)r.at;
    if (a.end() <= first || a.first() >= first + (r.rows - 1) * r.distance + r.bytes)
        return false;
    if (a.first() < first)
        return true;
    const uint64_t in = (a.first() - first) % r.distance;
    return in < r.bytes || in + a.bytes > r.distance;
}

// Outputs, the workspace among them, lie apart from the inputs and from one another
// (work-groups that share a row read what others would have overwritten), and the
// gradient apart from all but the logits.
int check_apart(const LogitRows &r, std::initializer_list<Span> inputs,
                std::initializer_list<Span> outputs)
{
    const uint64_t size = elem(r.dtype), T = (uint64_t)r.T, bytes = (uint64_t)r.V * size;
    const Rows logits{"logits", r.logits, T, bytes, (uint64_t)r.ld * size};
    const Rows dlogits{"dlogits", r.dlogits, T, bytes, (uint64_t)r.dld * size};
    auto refuse = [](const char *a, const char *b) {
        return fail(SK_ERR_INVALID_ARG, "%s and %s overlap", a, b);
    };
    for (const Span *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span &i : inputs)
            if (meet(*o, i))
                return refuse(o->name, i.name);
        for (const Span *q = outputs.begin(); q != o; ++q)
            if (meet(*o, *q))
                return refuse(o->name, q->name);
        for (const Rows *m : {&logits, &dlogits})
            if (meet(*o, *m))
                return refuse(o->name, m->name);
    }
    for (const Span &i : inputs)
        if (meet(i, dlogits))
            return refuse(dlogits.name, i.name);
    return SK_OK;
}

}  // namespace
}  // namespace sk

using namespace sk;

extern "C" {

size_t sinkhorn_losses_workspace_bytes(int op, int T, int V, int k, int dtype)
{
    if (op < SK_OP_TOKEN_LOGPROBS || op > SK_OP_BALANCE_LOSS ||
        (dtype != SK_F32 && dtype != SK_BF16) || !sizes_ok(op, T, V, k))
        return 0;
    return ws_bytes_of(op, T, V, k, dtype);
}

int sinkhorn_token_logprobs(const void *logits, int dtype, int64_t ld, const int32_t *labels,
                            int T, int V, double scale, float *logp, float *lse, void *ws,
                            size_t ws_bytes, void *stream)
{
    clear_error();
    int rc;
    if ((rc = check_rows(logits, dtype, ld, T, V, kMaxRows)) || (rc = check_scale(scale, "scale")))
        return rc;
    if (T > 0 && (!labels || (!logp && !lse)))
        return fail(SK_ERR_INVALID_ARG, "labels and one of logp and lse must be non-NULL");
    if ((rc = check_space(ws, ws_bytes, ws_bytes_of(SK_OP_TOKEN_LOGPROBS, T, V, 0, dtype))))
        return rc;
    if (T == 0)
        return SK_OK;
    const LogitRows r{logits, ld, dtype, T, V, scale, nullptr, 0};
    const size_t rows = (size_t)T * 4;
    if ((rc = check_apart(r, {{"labels", labels, rows}},
                          {{"logp", logp, rows},
                           {"lse", lse, rows},
                           {"ws", ws, ws_bytes_of(SK_OP_TOKEN_LOGPROBS, T, V, 0, dtype)}})))
        return rc;
    Carve c{(char *)ws};
    const Ws w = carve(c, SK_OP_TOKEN_LOGPROBS, T, V, 0, dtype);
    const hipError_t e = launch_logp(r, labels, Packed{nullptr, 0, 0}, w.token,
                                     LogpOut{logp, lse, nullptr}, (hipStream_t)stream);
    return e ? hip_fail(e, "token log-probabilities") : SK_OK;
}

int sinkhorn_token_logprobs_backward(const void *logits, int dtype, int64_t ld,
                                     const int32_t *labels, const float *grad, int T, int V,
                                     double scale, void *dlogits, int64_t dld, void *ws,
                                     size_t ws_bytes, void *stream)
{
    clear_error();
    int rc;
    if ((rc = check_rows(logits, dtype, ld, T, V, kMaxRows)) || (rc = check_scale(scale, "scale")))
        return rc;
    if (T > 0 && (!labels || !grad || !dlogits))
        return fail(SK_ERR_INVALID_ARG, "labels, grad and dlogits must be non-NULL");
    if ((rc = check_grad(logits, ld, dlogits, dld, dtype, T, V)) ||
        (rc = check_space(ws, ws_bytes, ws_bytes_of(SK_OP_TOKEN_LOGPROBS, T, V, 0, dtype))))
        return rc;
    if (T == 0)
        return SK_OK;
    const LogitRows r{logits, ld, dtype, T, V, scale, dlogits, dld};
    const size_t rows = (size_t)T * 4;
    if ((rc = check_apart(r, {{"labels", labels, rows}, {"grad", grad, rows}},
                          {{"ws", ws, ws_bytes_of(SK_OP_TOKEN_LOGPROBS, T, V, 0, dtype)}})))
        return rc;
    Carve c{(char *)ws};
    const Ws w = carve(c, SK_OP_TOKEN_LOGPROBS, T, V, 0, dtype);
    const hipError_t e = launch_logp_backward(r, labels, grad, w.token, (hipStream_t)stream);
    return e ? hip_fail(e, "token log-probabilities backward") : SK_OK;
}

int sinkhorn_policy_loss(const void *logits, int dtype, int64_t ld, const int32_t *labels, int T,
                         int V, const int64_t *offsets, int n, const float *old, const float *adv,
                         const float *ref, const float *weights, double scale, double clip_lo,
                         double clip_hi, double kl_coef, unsigned flags, float *loss, float *kl,
                         float *logp, void *dlogits, int64_t dld, void *ws, size_t ws_bytes,
                         void *stream)
{
    clear_error();
    int rc;
    if ((rc = check_rows(logits, dtype, ld, T, V, kMaxRows)) ||
        (rc = check_scale(scale, "scale")) ||
        (rc = check_packed(offsets, n, flags,
                           SK_LOSS_MEAN | SK_LOSS_FILL | SK_LOSS_ROW_ADVANTAGE)))
        return rc;
    if (!loss || !kl || (T > 0 && (!labels || !old || !adv)))
        return fail(SK_ERR_INVALID_ARG, "labels, old, adv, loss and kl must be non-NULL");
    if (!(clip_lo >= 0.0 && clip_lo < 1.0) || !(clip_hi >= 0.0))
        return fail(SK_ERR_INVALID_ARG, "clip_lo=%g must be in [0, 1) and clip_hi=%g >= 0",
                    clip_lo, clip_hi);
    if (!isfinite(kl_coef))
        return fail(SK_ERR_INVALID_ARG, "kl_coef=%g must be finite", kl_coef);
    if ((rc = check_grad(logits, ld, dlogits, dld, dtype, T, V)) ||
        (rc = check_space(ws, ws_bytes, ws_bytes_of(SK_OP_POLICY_LOSS, T, V, 0, dtype))))
        return rc;
    const LogitRows r{logits, ld, dtype, T, V, scale, dlogits, dld};
    const size_t rows = (size_t)T * 4, seqs = (size_t)n * 4;
    if ((rc = check_apart(r, {{"labels", labels, rows},
                              {"offsets", offsets, 2 * seqs + 8},
                              {"old", old, rows},
                              {"adv", adv, flags & SK_LOSS_ROW_ADVANTAGE ? rows : seqs},
                              {"ref", ref, rows},
                              {"weights", weights, seqs}},
                          {{"loss", loss, seqs},
                           {"kl", kl, seqs},
                           {"logp", logp, rows},
                           {"ws", ws, ws_bytes_of(SK_OP_POLICY_LOSS, T, V, 0, dtype)}})))
        return rc;
    Carve c{(char *)ws};
    const Ws w = carve(c, SK_OP_POLICY_LOSS, T, V, 0, dtype);
    PolicyArgs a{};
    a.old = old;
    a.ref = ref;
    a.adv = adv;
    a.weights = weights;
    a.adv_per_token = (flags & SK_LOSS_ROW_ADVANTAGE) != 0;
    a.mean = (flags & SK_LOSS_MEAN) != 0;
    a.lo = 1.0 - clip_lo;
    a.hi = 1.0 + clip_hi;
    a.log_lo = log1p(-clip_lo);
    a.log_hi = log1p(clip_hi);
    a.kl = kl_coef;
    a.info = w.info;
    a.term = w.term;
    a.loss = loss;
    a.kl_out = kl;
    a.logp = logp;
    const hipError_t e = launch_policy(r, labels, Packed{offsets, n, (flags & SK_LOSS_FILL) != 0},
                                       a, w.token, (hipStream_t)stream);
    return e ? hip_fail(e, "policy loss") : SK_OK;
}

int sinkhorn_preference_loss(const void *logits, int dtype, int64_t ld, const int32_t *labels,
                             int T, int V, const int64_t *offsets, int pairs, const float *ref,
                             const float *weights, double scale, int kind, double beta,
                             double smoothing, unsigned flags, float *loss, float *reward,
                             float *logp, void *dlogits, int64_t dld, void *ws, size_t ws_bytes,
                             void *stream)
{
    clear_error();
    int rc;
    if ((rc = check_rows(logits, dtype, ld, T, V, kMaxRows)) ||
        (rc = check_scale(scale, "scale")) ||
        (rc = check_packed(offsets, pairs, flags, SK_LOSS_MEAN | SK_LOSS_FILL)))
        return rc;
    if (!loss || !reward || (T > 0 && (!labels || !logp)))
        return fail(SK_ERR_INVALID_ARG, "labels, loss, reward and logp must be non-NULL");
    if (kind != SK_PREFERENCE_SIGMOID && kind != SK_PREFERENCE_SQUARE)
        return fail(SK_ERR_INVALID_ARG, "kind %d is no preference loss", kind);
    if (!(beta > 0.0) || !isfinite(beta) || !(smoothing >= 0.0 && smoothing <= 1.0))
        return fail(SK_ERR_INVALID_ARG, "beta=%g must be finite and > 0, smoothing=%g in [0, 1]",
                    beta, smoothing);
    if ((rc = check_grad(logits, ld, dlogits, dld, dtype, T, V)) ||
        (rc = check_space(ws, ws_bytes, ws_bytes_of(SK_OP_PREFERENCE_LOSS, T, V, 0, dtype))))
        return rc;
    const LogitRows r{logits, ld, dtype, T, V, scale, dlogits, dld};
    const size_t rows = (size_t)T * 4, each = (size_t)pairs * 4;
    if ((rc = check_apart(r, {{"labels", labels, rows},
                              {"offsets", offsets, 4 * each + 8},
                              {"ref", ref, rows},
                              {"weights", weights, each}},
                          {{"loss", loss, each},
                           {"reward", reward, 2 * each},
                           {"logp", logp, rows},
                           {"ws", ws, ws_bytes_of(SK_OP_PREFERENCE_LOSS, T, V, 0, dtype)}})))
        return rc;
    Carve c{(char *)ws};
    const Ws w = carve(c, SK_OP_PREFERENCE_LOSS, T, V, 0, dtype);
    const PreferenceArgs a{ref,       weights, kind,   (flags & SK_LOSS_MEAN) != 0,
                           beta,      smoothing, w.coef, w.stat,
                           loss,      reward,  logp};
    const hipError_t e =
        launch_preference(r, labels, Packed{offsets, 2 * pairs, (flags & SK_LOSS_FILL) != 0}, a,
                          w.token, (hipStream_t)stream);
    return e ? hip_fail(e, "preference loss") : SK_OK;
}

int sinkhorn_distill_loss(const void *logits, int dtype, int64_t ld, int T, int V,
                          const int32_t *index, const float *teacher, int K,
                          const float *teacher_lse, const float *weights, double temperature,
                          float *loss, void *dlogits, int64_t dld, void *ws, size_t ws_bytes,
                          void *stream)
{
    clear_error();
    int rc;
    if ((rc = check_rows(logits, dtype, ld, T, V, kMaxRows)) ||
        (rc = check_scale(1.0 / temperature, "1 / temperature")))
        return rc;
    if (K < 1 || K > kMaxTopK)
        return fail(SK_ERR_INVALID_ARG, "K=%d must be in [1, %d]", K, kMaxTopK);
    if (T > 0 && (!index || !teacher || !loss))
        return fail(SK_ERR_INVALID_ARG, "index, teacher and loss must be non-NULL");
    if ((rc = check_grad(logits, ld, dlogits, dld, dtype, T, V)) ||
        (rc = check_space(ws, ws_bytes, ws_bytes_of(SK_OP_DISTILL_LOSS, T, V, K, dtype))))
        return rc;
    if (T == 0)
        return SK_OK;
    const LogitRows r{logits, ld, dtype, T, V, 1.0 / temperature, dlogits, dld};
    const size_t rows = (size_t)T * 4;
    if ((rc = check_apart(r, {{"index", index, rows * K},
                              {"teacher", teacher, rows * K},
                              {"teacher_lse", teacher_lse, rows},
                              {"weights", weights, rows}},
                          {{"loss", loss, rows},
                           {"ws", ws, ws_bytes_of(SK_OP_DISTILL_LOSS, T, V, K, dtype)}})))
        return rc;
    Carve c{(char *)ws};
    const Ws w = carve(c, SK_OP_DISTILL_LOSS, T, V, K, dtype);
    const DistillArgs a{index, teacher, teacher_lse, weights, K, w.zk, loss};
    const hipError_t e = launch_distill(r, a, w.token, (hipStream_t)stream);
    return e ? hip_fail(e, "distillation loss") : SK_OK;
}

int sinkhorn_balance_loss(const void *logits, int dtype, int64_t ld, int T, int E,
                          const int32_t *index, int K, const int64_t *offsets, int G,
                          double balance, double z, unsigned flags, float *loss, float *zloss,
                          int32_t *counts, void *dlogits, int64_t dld, void *ws, size_t ws_bytes,
                          void *stream)
{
    clear_error();
    int rc;
    if ((rc = check_rows(logits, dtype, ld, T, E, kMaxExperts)))
        return rc;
    if (K < 1 || K > kMaxChosen)
        return fail(SK_ERR_INVALID_ARG, "K=%d must be in [1, %d]", K, kMaxChosen);
    if (G < 1 || G > kMaxSequences || (!offsets && G != 1))
        return fail(SK_ERR_INVALID_ARG, "%d groups need 1 <= G <= %d, and offsets unless G is 1",
                    G, kMaxSequences);
    if (flags & ~SK_LOSS_FILL)
        return fail(SK_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (!loss || !zloss || !counts || (T > 0 && !index))
        return fail(SK_ERR_INVALID_ARG, "index, loss, zloss and counts must be non-NULL");
    if (!isfinite(balance) || !isfinite(z))
        return fail(SK_ERR_INVALID_ARG, "balance=%g and z=%g must be finite", balance, z);
    if ((rc = check_grad(logits, ld, dlogits, dld, dtype, T, E)) ||
        (rc = check_space(ws, ws_bytes, ws_bytes_of(SK_OP_BALANCE_LOSS, T, E, G, dtype))))
        return rc;
    const size_t groups = (size_t)G * 4;
    if ((rc = check_apart(LogitRows{logits, ld, dtype, T, E, 1.0, dlogits, dld},
                          {{"index", index, (size_t)T * K * 4},
                           {"offsets", offsets, 2 * groups + 8}},
                          {{"loss", loss, groups},
                           {"zloss", zloss, groups},
                           {"counts", counts, groups * E},
                           {"ws", ws, ws_bytes_of(SK_OP_BALANCE_LOSS, T, E, G, dtype)}})))
        return rc;
    Carve c{(char *)ws};
    const Ws w = carve(c, SK_OP_BALANCE_LOSS, T, E, G, dtype);
    BalanceArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.dtype = dtype;
    a.T = T;
    a.E = E;
    a.K = K;
    a.index = index;
    a.offsets = offsets;
    a.G = G;
    a.fill = (flags & SK_LOSS_FILL) != 0;
    a.balance = balance;
    a.z = z;
    a.loss = loss;
    a.zloss = zloss;
    a.counts = counts;
    a.dlogits = dlogits;
    a.dld = dld;
    const hipError_t e = launch_balance(a, w.balance, (hipStream_t)stream);
    return e ? hip_fail(e, "balance loss") : SK_OK;
}

}  // extern "C"
