"""The output end of a model from its formulas, in float64 on the CPU, with the error that the
fp32 steps may bring.

Norm.  Sums of a row and its factor r are fp64; r, the products with it and with the weight are
fp32, each rounded once (U = 2^-24), and the result once to its type.
The 8-bit values are exact: 127 p / a to the nearest, ties to even.

Product.  The sum is exact; its conversion, the scales' product, their product with it and the
bias's addition round once each, and the result once to its type.

Scores.  As for the losses: eps_S bounds the sum S of a row, relative.  W, the sum of e_v d_v with
d_v = s (M - z_v), has terms of one sign.  An e_v is off, relative, by 2^-23 and by its exponent's
three roundings, 3 U d_v; d_v by 3 U; additions, two roundings each, as many as for S.  So
D = W / S is off by at most  D (3 eps_S + 8 U) + 3 U sum q d^2.
"""
import math

import torch

import losses_formulas as L

U, HALF, check = L.U, L.HALF, L.check
TINY = 1e-38


def stream(x, residual):
    """h: the sum, rounded to the type (fp64 holds it exactly or far beyond a rounding's middle)."""
    if residual is None:
        return x.detach().cpu()
    return (x.detach().cpu().double() + residual.detach().cpu().double()).to(x.dtype)


def factor(h, eps):
    h = h.double()
    return 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)


def norm(h, weight, eps, dtype):
    """(y, tolerance) of the norm of h (CPU, its type)."""
    y = h.double() * factor(h, eps)
    if weight is not None:
        y = y * weight.cpu().double()
    return y, y.abs() * (3 * U + HALF[dtype]) * 1.01 + TINY


def eight(h, weight, eps):
    """(q, scale, its tolerance); eps None: without the norm."""
    p = h.double()
    if weight is not None:
        p = p * weight.cpu().double()
    a = p.abs().amax(1, keepdim=True)
    sound = a.isfinite()
    q = torch.where(sound & (a > 0), torch.round(127.0 * p / torch.where(a > 0, a, 1.0)), 0.0)
    scale = a / 127.0
    if eps is not None:
        scale = scale * factor(h, eps)
    scale = torch.where(sound, scale, math.nan)[:, 0]
    return q.to(torch.int8), scale, scale.abs() * U * 1.01 + 2.0 ** -149


def norm_backward(dy, h, weight, dh, eps, workers=1):
    """((dx, tolerance), (dweight, tolerance)); `workers`: how many share the rows."""
    dtype = h.dtype
    h, dy = h.cpu().double(), dy.cpu().double()
    d = h.shape[1]
    r = factor(h, eps)
    u = dy if weight is None else dy * weight.cpu().double()
    first = r * u
    c = r ** 3 * (u * h).sum(1, keepdim=True) / d
    c_tol = U * c.abs() + r ** 3 * U * (u * h).abs().sum(1, keepdim=True) / d
    v = first - c * h
    dx = v if dh is None else v + dh.cpu().double()
    tol = 3 * U * first.abs() + (c_tol + U * c.abs()) * h.abs() + 2 * U * v.abs() + U * dx.abs()
    tol = tol + HALF[dtype] * (dx.abs() + tol) * 1.01 + TINY
    n = dy * h * r
    dw = n.sum(0)
    adds = math.ceil(max(1, h.shape[0]) / workers) + 3
    return (dx, tol), (dw, U * (adds * n.abs().sum(0) + dw.abs()) * 1.01 + TINY)


def linear(x, xscale, w, wscale, bias, dtype):
    """(out, tolerance)."""
    s = x.cpu().double() @ w.cpu().double().t()
    v = s * (xscale.cpu().double()[:, None] * wscale.cpu().double())
    out = v if bias is None else v + bias.cpu().double()
    tol = 3 * U * v.abs() + (0 if bias is None else U * out.abs())
    return out, (tol + HALF[dtype] * (out.abs() + tol)) * 1.01 + TINY


def alternatives(z, used, lse, scale, top):
    """(index, best) by a stable sort of each row: NaN first, then falling values."""
    T, V = z.shape
    index = torch.full((T, top), -1, dtype=torch.int32)
    best = torch.full((T, top), -math.inf, dtype=torch.float64)
    for t in range(T):
        if not used[t]:
            continue
        x = z[t].cpu().double() + 0.0
        order = torch.sort(torch.where(x.isnan(), math.inf, x), descending=True, stable=True).indices
        nan = x[order].isnan()
        order = torch.cat([order[nan], order[~nan]])[:top]
        order = order[~(x[order] == -math.inf)]
        index[t, :len(order)] = order.int()
        best[t, :len(order)] = x[order] * scale - lse[t]
    return index, best


class Scores:
    """Everything that the scores of rows are, with tolerances."""

    def __init__(self, logits, labels=None, scale=1.0, top=0):
        R = self.R = L.Rows(logits, scale)
        T, V = R.T, R.V
        y = torch.zeros(T, dtype=torch.int32) if labels is None else labels.cpu()
        self.used = torch.ones(T, dtype=torch.bool) if labels is None else y >= 0
        e = self.eps = L.eps_sum(V)
        self.logp = R.logp(y)
        lse = torch.where(self.used, R.lse, 0.0)
        self.lse = lse, e + 2 * U * torch.where(lse.isfinite(), lse.abs(), 0.0)
        d = torch.where(R.empty[:, None], 0.0, torch.where(R.empty, 0.0, R.M)[:, None] - R.z * scale)
        # the row's nats of distance; what has no probability has no part
        d = torch.where(R.q > 0, d, 0.0)
        self.d = d
        self.D = (R.q * d).sum(1)
        self.D_tol = self.D * (3 * e + 8 * U) + 3 * U * (R.q * d * d).sum(1)
        H = torch.where(self.used & ~R.empty, R.lnS + self.D, 0.0)
        self.entropy = H, e + self.D_tol + 2 * U * H.abs()
        if top:
            index, best = alternatives(logits, self.used, R.lse, scale, top)
            self.index = index
            self.best = best, (e + 2 * U * torch.where(best.isfinite(), best.abs(), 0.0)
                               + 2 * U * torch.where(R.lse.isfinite(), R.lse.abs(), 0.0)[:, None])

    def backward(self, labels, grad, grad_entropy):
        """(dlogits, tolerance)."""
        R, s, e = self.R, self.R.scale, self.eps
        live = (self.used & ~R.empty)[:, None]
        zero = torch.zeros(R.T, dtype=torch.float64)
        gl = (zero if grad is None else grad.cpu().double())[:, None] * s
        ge = (zero if grad_entropy is None else grad_entropy.cpu().double())[:, None] * s
        hot = torch.zeros_like(R.q)
        if labels is not None:
            y = labels.cpu().long()
            ok = (y >= 0) & (y < R.V)
            hot[torch.arange(R.T)[ok], y[ok]] = 1.0
        D, d, q = self.D[:, None], self.d, R.q
        g = torch.where(live, gl * (hot - q) + ge * q * (d - D), 0.0)
        if labels is not None:
            g = torch.where(live & (labels.cpu()[:, None] >= R.V) & (gl != 0), math.nan, g)
        rel = e + U * (8 + 3 * d)
        tol = gl.abs() * (q * rel + hot * (e + 8 * U)) \
            + ge.abs() * q * ((D + d) * (rel + 4 * U) + self.D_tol[:, None])
        tol = torch.where(live, tol, 0.0)
        return g, tol + HALF[R.dtype] * (g.abs() + tol) * 1.01 + TINY
