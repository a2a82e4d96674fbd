"""The losses over logits from their formulas, in float64 on the CPU, with the error
that fp32 softmax sums may bring.

Bounds.  With M the row maximum, a term e_v = 2^((s z_v - s M) log2 e) is off, relative, by the
hardware exponential (one unit, 2^-23) and by its argument: the difference, the product and the
constant are each rounded once, 3 * 2^-24 * |argument| * ln 2.  Weighted by the softmax, the mean
|argument| is at most log2 V.  A thread adds at most V/512 + 64 terms one after another and the
joins add 30 more, each rounding by 2^-24.  So the sum S is off, relative, by at most
    eps_S = 2^-24 (2 + 2.1 log2 V + V/512 + 100),
lse and logp by eps_S and their own rounding (2^-24 relative), and an element q_v of the softmax,
relative, by eps_S + 2^-23 + 3 ln 2 2^-24 |argument| + 4 roundings.

The logarithm of S is taken in fp64.

A teacher's probability p_k is an fp32 exponential of an argument rounded once (2^-24 |argument|)
and, where the K are normalised among themselves, over a sum of such (K/64 + 10 additions): off,
relative, by at most 2^-24 (14 + K/64 + |argument|).
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8,   # a rounding, relative
        torch.float64: 0.0}


def eps_sum(V):
    return U * (2 + 2.1 * math.log2(max(V, 2)) + V / 512 + 100)


class Rows:
    """Softmax of scale * logits per row, float64; empty rows (nothing finite) marked."""

    def __init__(self, logits, scale=1.0):
        self.dtype = logits.dtype
        z = logits.detach().cpu().double()
        self.T, self.V = z.shape
        self.scale = scale
        self.z = z
        x = z * scale
        self.M = x.amax(1) if self.T else x.sum(1)
        self.empty = self.M == -math.inf
        shift = torch.where(self.empty, 0.0, self.M)
        e = torch.exp(x - shift[:, None])
        S = e.sum(1)
        self.lse = torch.where(self.empty, -math.inf, shift + torch.log(S))
        self.lnS = torch.where(self.empty, 0.0, torch.log(S))
        self.q = torch.where(self.empty[:, None], 0.0, e / torch.where(self.empty, 1.0, S)[:, None])
        arg = torch.where(e > 0, (x - shift[:, None]).abs(), 0.0)
        self.q_tol = self.q * (eps_sum(self.V) + U * (2 + 4 + 3 * arg)) + 2.0 ** -126

    def logp(self, labels):
        """(value, tolerance) at the labels; 0 where not scored or without a distribution."""
        y = labels.cpu().long()
        at = y.clamp(min=0, max=self.V - 1)
        # the maximum first: a row of huge values keeps its differences
        zy = self.z.gather(1, at[:, None])[:, 0] * self.scale
        lp = zy - torch.where(self.empty, 0.0, self.M) - self.lnS
        lp = torch.where(y >= self.V, math.nan, lp)
        used = (y >= 0) & ~self.empty
        lp = torch.where(used, lp, 0.0)
        gap = torch.where(lp.isfinite(), lp.abs(), 0.0)
        return lp, eps_sum(self.V) + U * gap * 2

    def label_grad(self, labels, coef, coef_tol):
        """coef scale (1[v = label] - q) and its tolerance, rounding to the logits' type included."""
        y = labels.cpu().long()
        coef = torch.where((y >= 0) & ~self.empty, coef, 0.0) * self.scale
        tol = torch.where((y >= 0) & ~self.empty, coef_tol, 0.0) * abs(self.scale)
        hot = torch.zeros_like(self.q)
        ok = (y >= 0) & (y < self.V)
        hot[torch.arange(self.T)[ok], y[ok]] = 1.0
        g = torch.where(coef[:, None] == 0, 0.0, coef[:, None] * (hot - self.q))
        g = torch.where((y >= self.V)[:, None], math.nan, g)
        # 4 U: the coefficient, its product with 1 / S, the last product and the label's sum
        t = coef.abs()[:, None] * (self.q_tol + 4 * U * (hot + self.q)) + tol[:, None] * (hot + self.q)
        t = t + HALF[self.dtype] * (g.abs() + t) * 1.01 + 1e-38
        return g, t


def ranges(offsets, T):
    o = [min(max(int(v), 0), T) for v in offsets.cpu().tolist()]
    return [(a, max(a, b)) for a, b in zip(o[:-1], o[1:])]


def policy(logits, labels, offsets, old, adv, ref=None, clip=(0.2, 0.2), kl=0.0, scale=1.0,
           weights=None, mean=True):
    """Per output (value, tolerance): loss [n], kl [n], logp [T], gradient [T, V]; and the
    distance of each ratio from the nearest clipping border."""
    R = Rows(logits, scale)
    lp, lp_tol = R.logp(labels)
    T, n = R.T, offsets.numel() - 1
    old, adv = old.cpu().double(), adv.cpu().double()
    y = labels.cpu().long()
    used = (y >= 0) & ~R.empty
    A = adv if adv.shape == (T,) else None
    loss, kls = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    loss_tol, kl_tol = loss.clone(), loss.clone()
    coef, coef_tol = torch.zeros(T, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    r = torch.exp(lp - old)
    lo, hi = 1 - clip[0], 1 + clip[1]
    border = torch.minimum((r - lo).abs(), (r - hi).abs())
    for i, (a, b) in enumerate(ranges(offsets, T)):
        w = 1.0 if weights is None else float(weights[i])
        if mean:
            k = int((y[a:b] >= 0).sum())
            w = w / k if k else 0.0
        for t in range(a, b):
            if not used[t]:
                continue
            Ai = float(A[t]) if A is not None else float(adv[i])
            rt, d = float(r[t]), float(lp_tol[t])
            cut = (Ai > 0 and rt > hi) or (Ai < 0 and rt < lo)
            gain = min(max(rt, lo), hi) * Ai if cut else rt * Ai
            slope = 0.0 if cut else -rt * Ai
            st = 0.0 if cut else abs(rt * Ai) * d * 1.01
            kt = ktol = 0.0
            if ref is not None:
                g = float(ref[t]) - float(lp[t])
                kt, ktol = math.expm1(g) - g, abs(math.expm1(g)) * d * 1.01 + d * d
                slope -= kl * math.expm1(g)
                st += abs(kl) * math.exp(g) * d * 1.01
            loss[i] += w * (kl * kt - gain)
            kls[i] += w * kt
            # the weight and each row's two terms are rounded to fp32 once
            loss_tol[i] += abs(w) * (st + abs(kl) * ktol + 3 * U * abs(kl * kt - gain)
                                     + U * (abs(kl * kt) + abs(gain)))
            kl_tol[i] += abs(w) * (ktol + 3 * U * abs(kt))
            coef[t], coef_tol[t] = slope * w, abs(w) * (st + 2 * U * abs(slope))
    loss_tol += U * loss.abs() * 2
    kl_tol += U * kls.abs() * 2
    return (loss, loss_tol), (kls, kl_tol), (lp, lp_tol), R.label_grad(labels, coef, coef_tol), border


def preference(logits, labels, offsets, ref=None, beta=0.1, smoothing=0.0, kind="sigmoid",
               scale=1.0, weights=None, mean=False):
    """Per output (value, tolerance): loss [P], reward [2 P], logp [T], gradient [T, V]."""
    R = Rows(logits, scale)
    lp, lp_tol = R.logp(labels)
    y = labels.cpu().long()
    used = (y >= 0) & ~R.empty
    rng = ranges(offsets, R.T)
    P = len(rng) // 2
    ratio, tol, part = [], [], []
    for a, b in rng:
        u = used[a:b]
        v = lp[a:b][u] - (ref.cpu().double()[a:b][u] if ref is not None else 0.0)
        k = 1.0 / max(1, int(u.sum())) if mean else 1.0
        ratio.append(float(v.sum()) * k)
        tol.append(float((lp_tol[a:b][u] + U * lp[a:b][u].abs()).sum()) * k)
        part.append(k if int(u.sum()) else (0.0 if mean else 1.0))
    loss, loss_tol, coef, coef_tol = [], [], torch.zeros(R.T, dtype=torch.float64), \
        torch.zeros(R.T, dtype=torch.float64)
    for i in range(P):
        w = 1.0 if weights is None else float(weights[i])
        gap, d = ratio[2 * i] - ratio[2 * i + 1], tol[2 * i] + tol[2 * i + 1]
        if kind == "sigmoid":
            h = beta * gap
            softplus = lambda x: max(x, 0.0) + math.log1p(math.exp(-abs(x)))  # noqa: E731
            value = (1 - smoothing) * softplus(-h) + smoothing * softplus(h)
            sig = 1 / (1 + math.exp(h)) if h < 700 else 0.0
            slope, bend = beta * (smoothing - sig), beta * beta / 4
        else:
            value, slope, bend = (gap - 0.5 / beta) ** 2, 2 * (gap - 0.5 / beta), 2.0
        loss.append(w * value)
        loss_tol.append(abs(w) * (abs(slope) * d + bend * d * d + 2 * U * abs(value)))
        for j, sign in ((2 * i, 1.0), (2 * i + 1, -1.0)):
            a, b = rng[j]
            coef[a:b] = sign * slope * w * part[j]
            coef_tol[a:b] = abs(w) * part[j] * (bend * d + 2 * U * abs(slope))
    t64 = lambda v: torch.tensor(v, dtype=torch.float64)  # noqa: E731
    reward = t64(ratio) * beta
    return ((t64(loss), t64(loss_tol)), (reward, t64(tol) * beta + 2 * U * reward.abs()),
            (lp, lp_tol), R.label_grad(labels, coef, coef_tol))


def distill(logits, index, teacher, teacher_lse=None, temperature=1.0, weights=None):
    """(value, tolerance) of loss [T] and of the gradient [T, V]."""
    tau = temperature
    R = Rows(logits, 1.0 / tau)
    T, V = R.T, R.V
    loss, loss_tol = torch.zeros(T, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    grad, tol = torch.zeros(T, V, dtype=torch.float64), torch.zeros(T, V, dtype=torch.float64)
    idx, u = index.cpu().long(), teacher.cpu().double() / tau
    for t in range(T):
        w = 1.0 if weights is None else float(weights[t])
        keep = (idx[t] >= 0) & (u[t] != -math.inf)
        if w == 0 or R.empty[t] or not keep.any():
            continue
        if (idx[t] >= V).any():
            loss[t], grad[t] = math.nan, math.nan
            continue
        at, v = idx[t][keep], u[t][keep]
        U0 = torch.logsumexp(v, 0) if teacher_lse is None else teacher_lse.cpu().double()[t]
        p = torch.exp(v - U0)
        lq = R.z[t, at] * R.scale - R.M[t] - R.lnS[t]
        terms = p * (v - U0 - lq)
        loss[t] = w * tau * tau * torch.where(p > 0, terms, 0.0).sum()
        C = float(p.sum())
        base = v.max() if teacher_lse is None else U0
        p_off = U * (14 + idx.shape[1] / 64 + (v - base).abs())
        # the terms follow p; log q and the teacher's own logarithm are off by eps_S at most
        loss_tol[t] = abs(w) * tau * tau * (2 * C * eps_sum(V) + float((p_off * terms.abs()).sum())) \
            + 2 * U * abs(loss[t])
        sparse = torch.zeros(V, dtype=torch.float64).index_add_(0, at, p)
        grad[t] = w * tau * (C * R.q[t] - sparse)
        entries = int(keep.sum())
        off = torch.zeros(V, dtype=torch.float64).index_add_(0, at, p * p_off)
        tol[t] = abs(w) * tau * (C * (R.q_tol[t] + 5 * U * R.q[t]) + (5 + entries) * U * sparse
                                 + off + float(off.sum()) * R.q[t])
    tol = tol + HALF[R.dtype] * (grad.abs() + tol) * 1.01 + 1e-38
    return (loss, loss_tol), (grad, tol)


def balance(logits, index, offsets=None, balance=1.0, z=0.0):
    """(value, tolerance) of loss [G], zloss [G], counts [G, E] (exact) and the gradient."""
    R = Rows(logits)
    T, E = R.T, R.V
    idx = index.cpu().long()
    K = idx.shape[1]
    if offsets is None:
        offsets = torch.tensor([0, T])
    rng = ranges(offsets, T)
    G = len(rng)
    f64 = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    loss, loss_tol, zloss, z_tol = f64(G), f64(G), f64(G), f64(G)
    counts, grad, tol = torch.zeros(G, E, dtype=torch.int32), f64(T, E), f64(T, E)
    e = eps_sum(E)
    for g, (a, b) in enumerate(rng):
        ok = (idx[a:b] >= 0) & (idx[a:b] < E)
        n = int(ok.any(1).sum())
        flat = idx[a:b][ok]
        counts[g] = torch.bincount(flat, minlength=E).int()
        if not n:
            continue
        if (idx[a:b] >= E).any():
            loss[g] = math.nan
        f = counts[g].double() * E / (K * n)
        rows = torch.arange(a, b)[(idx[a:b] >= 0).any(1) & ~R.empty[a:b]]
        q, lse = R.q[rows], R.lse[rows]
        dot = (q * f).sum(1)
        loss[g] = loss[g] + dot.sum() / n
        # each f is rounded once, as f - 1; sum q f is off by f's and q's roundings
        size = (q * (f - 1).abs()).sum(1)
        d = size * (e + 24 * U) + E * U * size + (R.q_tol[rows] * (f - 1).abs()).sum(1)
        loss_tol[g] = d.sum() / n + 4 * U * abs(loss[g])
        zloss[g] = (lse ** 2).sum() / n
        lt = e + 4 * U * (lse.abs() + R.M[rows].abs())
        z_tol[g] = (2 * lse.abs() * lt + lt * lt).sum() / n + 4 * U * zloss[g]
        inner = balance * (f[None] - dot[:, None]) + 2 * z * lse[:, None]
        it = abs(balance) * (d[:, None] + 6 * U * ((f - 1).abs()[None] + size[:, None])) \
            + 2 * abs(z) * (lt + 4 * U * lse.abs())[:, None]
        if math.isnan(loss[g]):
            inner = inner * math.nan
        grad[rows] = q * inner / n
        tol[rows] = (q * it + (R.q_tol[rows] + 6 * U * q) * (inner.abs() + it)) / n
    tol = tol + HALF[R.dtype] * (grad.abs() + tol) * 1.01 + 1e-38
    return (loss, loss_tol), (zloss, z_tol), counts, (grad, tol)


def check(got, want, what):
    """got within the tolerance of want = (value, tolerance); NaN and infinities alike."""
    value, tol = want
    got = got.detach().cpu().double()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    # beyond the largest finite fp32 the result is infinite
    value = torch.where(value.abs() > 3.4028235677973366e38, value.sign() * math.inf, value)
    odd = ~value.isfinite()
    same = (got == value) | (got.isnan() & value.isnan())
    assert bool(same[odd].all()), f"{what}: {got[odd]} where {value[odd]} is due"
    off = torch.where(odd, 0.0, (got - value).abs())
    tol = torch.where(odd, 1.0, tol.expand_as(value) if torch.is_tensor(tol) else tol)
    worst = (off / tol.clamp(min=1e-300)).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times its tolerance, off by {off.max():.3g}"
