"""Edges of the output end of a model on the GPU: gradients of rows near the ends of fp32, 8-bit
values decided to the last bit, gradients against differences in directions that show them, outputs
over inputs, many rows, and rows far into their matrices.  Formulas and tolerances:
head_formulas.py."""
import math

import pytest
import torch

import head_formulas as H
import sinkhorn_point_cloud_amd as sk
from test_head_gpu import TYPES, norm_case, padded, rng

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _say(request):
    print(request.node.name, flush=True)
    yield


# --- the norm's gradient at the ends of fp32

# the size of a row's values and that of its dy: dx is of the size of their quotient (of dy / sqrt(eps)
# for the smallest), which lies well within fp32 each time
EXTREMES = [(1e30, 1.0), (1e30, 1e-5), (1e20, 1e-6), (1e18, 1e-6), (1e16, 1e-9), (1e10, 1e10), (1.0, 1e30),
            (1e-10, 1e-10), (1e-14, 1e15), (1e-30, 1e-20)]


def extreme_case(dt, d, g):
    """h, and a dy that follows it: the projection on h is a large part of the gradient."""
    h = torch.randn(len(EXTREMES) + 2, d, generator=g)
    dy = h.sign() * (0.5 + torch.rand(h.shape, generator=g))
    for t, (size, grad) in enumerate(EXTREMES):
        h[t] *= size
        dy[t] *= grad
    h[-2], dy[-2] = torch.finfo(TYPES[dt]).max / 8 * h[-2].sign(), dy[-2] * 1e6
    h[-1, d // 2] = 2.0 ** 100
    w = 1 + 0.3 * torch.randn(d, generator=g)
    return h.to(TYPES[dt]), dy.to(TYPES[dt]), w.to(TYPES[dt])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("d", [37, 515, 2501, 20000])
def test_norm_gradient_of_extreme_rows(d, dt):
    """dx = r (u - n m) + dh in fp32: u is off by U, n by 2 U (r and its product), m by U and what u's
    roundings bring to its sum, the inner difference and r by U of it each, the whole by U.  That is
    U |r u| + 3 U |r n m| + 2 U |v| + U |dx| beside the sum's part, against the formula's 3 U |r u| + 2 U
    |r n m| + 2 U |v| + 2 U |dx|: within it, since |r n m| <= |r u| + |dx| without dh."""
    h, dy, w = extreme_case(dt, d, rng(d))
    for weight in (w, None):
        wd = None if weight is None else weight.cuda()
        for eps in (1e-6, 1e-30):
            (ref, tol), _ = H.norm_backward(dy, h, weight, None, eps)
            # a gradient without its projection would be seen in every row but those that eps rules
            u = dy.double() if weight is None else dy.double() * weight.double()
            part = ((H.factor(h, eps) * u - ref).abs() / tol).amax(1)
            seen = H.factor(h, eps)[:, 0] * h.double().square().mean(1).sqrt() > 0.9
            assert seen.sum() >= 9 and (part[seen] > 100).all()
            dx, _ = sk.rms_norm_backward(dy.cuda(), h.cuda(), wd, eps=eps)
            H.check(dx, (ref, tol), "dx")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("size,grad", [(1e30, 1e-12), (1e30, 1e5), (1e-14, 1e-28), (1.0, 1e-30)])
def test_weight_gradient_of_extreme_rows(size, grad, dt):
    """dy r can lie below fp32's normal range while dy h r does not."""
    g = rng(31)
    h = (torch.randn(1, 700, generator=g) * size).to(TYPES[dt])
    dy = (torch.randn(1, 700, generator=g) * grad).to(TYPES[dt])
    w = torch.ones(700, dtype=h.dtype)
    _, dw = sk.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), eps=1e-30)
    H.check(dw, H.norm_backward(dy, h, w, None, 1e-30)[1], "dweight")


@pytest.mark.parametrize("dt", TYPES)
def test_norm_of_rows_whose_factor_is_subnormal(dt):
    """Root mean squares beyond 2^126, whose inverse has fewer bits in fp32: off by 2^-150, at most
    2^-22 of itself, once in y, and in the gradient in both factors of the projection and in one of u."""
    g = rng(33)
    top = torch.finfo(TYPES[dt]).max
    h = torch.randn(9, 700, generator=g).sign() * (0.98 + 0.02 * torch.rand(9, 700, generator=g))
    h = (h.double() * (torch.linspace(0.26, 1, 9)[:, None] * top)).to(TYPES[dt])
    assert h.isfinite().all() and (h.double().square().mean(1).sqrt() > 2.0 ** 126).all()
    dy = (h.sign() * (0.5 + torch.rand(9, 700, generator=g)) * 1e6).to(h.dtype)
    w = torch.ones(700, dtype=h.dtype)
    y, _ = sk.rms_norm(h.cuda(), w.cuda())
    ref, tol = H.norm(h, w, 1e-6, h.dtype)
    H.check(y, (ref, tol + 2.0 ** -22 * ref.abs()), "y")
    dx, dw = sk.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda())
    (ref, tol), (wref, wtol) = H.norm_backward(dy, h, w, None, 1e-6, workers=9)
    away = H.factor(h, 1e-6) * dy.double() - ref        # the projection
    H.check(dx, (ref, tol + 2.0 ** -22 * (ref.abs() + away.abs()) * 1.01), "dx")
    n = dy.double() * h.double() * H.factor(h, 1e-6)
    H.check(dw, (wref, wtol + 2.0 ** -22 * n.abs().sum(0)), "dweight")


# --- 8 bits to the last bit

def nearest(p, a):
    """127 p / a in whole numbers, ties to even."""
    k, rest = divmod(254 * p, 2 * a)
    return k + (rest > a or (rest == a and k & 1))


def test_eight_bits_of_weighted_fp32_rows_at_exact_ties():
    """p = h weight has up to 48 bits and 127 p up to 55, more than fp64's 53.  With a = 254 m n and
    p = (2 k + 1) m n, 127 p / a is k + 1/2 to the last bit."""
    ms = (66049, 66047, 65537, 40503, 33333, 1)
    steps = [2 * k + 1 for k in range(127)]
    h = torch.tensor([[254 * m] + [s * m for s in steps] + [-s * m for s in steps] for m in ms],
                     dtype=torch.float32)
    for n in (16777213, 16777215, 15485863, 8388609, 3):
        w = torch.full((h.shape[1],), float(n))
        q, _, _ = sk.rms_norm_int8(h.cuda(), w.cuda())
        even = [nearest(s, 254) for s in steps]
        want = torch.tensor([127] + even + [-k for k in even], dtype=torch.int8)
        assert torch.equal(q.cpu(), want.expand(len(ms), -1)), n


def test_eight_bits_of_weighted_fp32_rows_beside_ties():
    """Pairs (h, weight) of whole numbers of 24 bits whose products a and p have 254 p - (2 k + 1) a
    = 1 or 3, or -1 or -3: 2^-55 of itself off the middle of two steps.  A pair each row."""
    cases = [(13696173, 13550015, 12136601, 14147382), (10662761, 12013235, 12995323, 5704613),
             (15649377, 13613437, 13085221, 14550433), (9298943, 12177657, 8753761, 11051689),
             (11325871, 10886089, 8666695, 13946191), (13343589, 14999343, 9920321, 16124323)]
    n = len(cases)
    for sign, scale in ((1, 1.0), (-1, 2.0 ** 70), (1, 2.0 ** -90)):
        h, w = torch.zeros(n, 2 * n), torch.zeros(2 * n)
        want = torch.zeros(n, 2 * n, dtype=torch.int8)
        for t, (ha, wa, hp, wp) in enumerate(cases):
            h[t, 2 * t], h[t, 2 * t + 1] = ha, sign * hp
            w[2 * t], w[2 * t + 1] = wa, wp
            want[t, 2 * t], want[t, 2 * t + 1] = 127, sign * nearest(hp * wp, ha * wa)
        q, _, _ = sk.rms_norm_int8((h * scale).cuda(), w.cuda())
        assert torch.equal(q.cpu(), want), (sign, scale)


# --- gradients against differences

def score_directions(dt):
    """Few, peaked logits on a grid of 2^-5 (7 bits and a sign below 4, exact also one step away), a
    label that is not the likeliest, and weights of logp and entropy."""
    g = rng(41)
    T, V = 5, 12
    z = torch.randint(-90, 91, (T, V), generator=g).float() / 32
    y = z.argsort(1)[:, V // 2].int()
    return (z.to(TYPES[dt]), y, 0.5 + torch.rand(T, generator=g), -0.5 - torch.rand(T, generator=g))


def slack_of(z, wl, we, grad, h):
    """What a central difference of step h along +-1 may be off from grad's part in that direction.
    With x the direction and Z the logits (range R) under the row's q, logp''' = -k3(x) and
    H''' = -(k(Z, x, x, x) + 2 k3(x)), joint cumulants: |k3| <= 0.77 for |x| <= 1, and
    |k(Z, x, x, x)| <= E|Z - EZ||x - Ex|^3 + 3 |cov(Z, x)| var(x) <= 2 R + 3 R / 2, since |x - Ex| <= 2,
    var(x) <= 1, |cov(Z, x)| <= R / 2.  The central difference is off by h^2 / 6 times that.  Outputs of
    at most 16 are off by less than 16 U + 2e-7, twice, over 2 h; gradient entries by half a step of
    their type and 2e-6 of fp32 arithmetic."""
    R = (z.double().amax(1) - z.double().amin(1)).max() + 2 * h
    wl, we = wl.abs().double().sum(), we.abs().double().sum()
    return h * h / 6 * (wl * 0.77 + we * (3.5 * R + 1.54)) + (wl + we) * (16 * H.U + 2e-7) / h \
        + (H.HALF[z.dtype] + 2e-6) * grad.double().abs().sum()


@pytest.mark.parametrize("dt", TYPES)
def test_score_gradients_against_differences(dt):
    """Along the signs of the gradient, where the difference is the sum of its magnitudes: logp and
    entropy alone and together.  A gradient of zeros and one of the entropy's sign reversed are far
    outside of the slack."""
    z, y, wl, we = score_directions(dt)
    h = 2.0 ** -5
    yd, wld, wed = y.cuda(), wl.cuda(), we.cuda()

    def grad(a, b):
        return sk.token_scores_backward(z.cuda(), yd, a, b).cpu().double()

    def difference(a, b, x):
        def total(s):
            moved = (z.float() + s * x).to(z.dtype)
            assert torch.equal(moved.double(), z.double() + s * x.double())
            o = sk.token_scores(moved.cuda(), yd)
            return (a.double() * o[0].cpu().double() + b.double() * o[2].cpu().double()).sum()
        return (total(h) - total(-h)) / (2 * h)
    zero = torch.zeros_like(wl)
    dl, de, both = grad(wld, None), grad(None, wed), grad(wld, wed)
    for d, a, b in ((dl, wl, zero), (de, zero, we), (both, wl, we)):
        x = d.sign().float()
        diff, slack = difference(a, b, x), slack_of(z, a, b, d, h)
        assert abs(diff - (d * x).sum()) < slack
        assert abs(diff) > 8 * slack                                   # zeros
    x = both.sign().float()
    # the slack of both, and how far the entropy's part reversed or left out would be off
    assert abs((de * x).sum()) > 2 * slack_of(z, wl, we, both, h)
    for d, x in ((dl, dl.sign().float()), (de, de.sign().float())):
        assert abs((both * x).sum() - (d * x).sum()) > 2 * slack_of(z, wl, we, both, h)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("weighted", [False, True])
def test_norm_gradients_against_differences(weighted, dt):
    """dx along its own signs, dweight along its own: sums of magnitudes.  The difference's own error
    is that of the formula in fp64; y is off by half a step and 3 U, its sums with dy are fp64."""
    g = rng(42)
    T, d, h, eps = 4, 48, 2.0 ** -3, 0.5
    x = (torch.randint(-12, 13, (T, d), generator=g).float() / 8).to(TYPES[dt])
    w = ((torch.randint(4, 13, (d,), generator=g).float() / 8) if weighted else torch.ones(d)).to(x.dtype)
    # half of dy follows x, so that the projection is a large part
    dy = (torch.randint(-4, 5, (T, d), generator=g).float() / 8 + x.float()).to(x.dtype)
    dh = (torch.randint(-4, 5, (T, d), generator=g).float() / 8).to(x.dtype)
    dx, dw = sk.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), dh=dh.cuda(), eps=eps)
    dx, dw = dx.cpu().double(), dw.cpu().double()

    def total(x_, w_, here):
        y = sk.rms_norm(x_.cuda(), w_.cuda(), eps=eps)[0].cpu().double() if here \
            else H.norm(x_, w_, eps, torch.float64)[0]
        return (y * dy.double()).sum() + (x_.double() * dh.double()).sum()

    def moved(a, s, way):
        b = (a.float() + s * way.float()).to(a.dtype)
        assert torch.equal(b.double(), a.double() + s * way.double())
        return b

    way = dx.sign()
    here, there = ((total(moved(x, h, way), w, k) - total(moved(x, -h, way), w, k)) / (2 * h)
                   for k in (True, False))
    size = H.norm(x, w, eps, torch.float64)[0].abs() + h * w.double()
    rounding = ((H.HALF[x.dtype] + 4 * H.U) * size * dy.double().abs()).sum() / h
    (ref, tol), _ = H.norm_backward(dy, x, w, dh, eps)
    slack = rounding + abs(there - (ref * way).sum()) + tol.sum()
    assert abs(here - dx.abs().sum()) < slack and dx.abs().sum() > 4 * slack
    # without its projection on h it would be seen
    u = dy.double() * w.double()
    bare = H.factor(x, eps) * u + dh.double()
    assert abs((bare * way).sum() - dx.abs().sum()) > 2 * slack
    way = dw.sign()
    here = (total(x, moved(w, h, way), True) - total(x, moved(w, -h, way), True)) / (2 * h)
    assert abs(here - dw.abs().sum()) < rounding + 1e-5 * dw.abs().sum()
    assert dw.abs().sum() > 4 * rounding


# --- outputs over inputs

# lengths that end inside a chunk (of 8 bf16 or 4 fp32 values), of each launch shape
OVER = [(9, 61), (5, 515), (4, 1029), (3, 4099), (3, 16389), (2, 32765)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,d", OVER)
def test_norm_outputs_over_inputs(T, d, dt):
    """y and h over x and the residual, either way, and h over either with y in 8 bits: the bits of
    outputs of their own."""
    g = rng(T + d)
    x, r, w = norm_case(T, d, dt, g)
    wd = w.cuda()

    def inputs():
        return padded(x, 3, 1)[0], padded(r, 3, 1)[0]
    xd, rd = inputs()
    y, h = sk.rms_norm(xd, wd, rd)
    q, scale, _ = sk.rms_norm_int8(xd, wd, rd)
    assert torch.equal(h.cpu(), H.stream(x, r))
    for swap in (False, True):
        xd, rd = inputs()
        to = (rd, xd) if swap else (xd, rd)
        got = sk.rms_norm(xd, wd, rd, out=to)
        assert torch.equal(to[0], y) and torch.equal(to[1], h) and got[0] is to[0]
        xd, rd = inputs()
        over, other, kept = (rd, xd, x) if swap else (xd, rd, r)
        got = sk.rms_norm_int8(xd, wd, rd, out=(torch.empty_like(q), torch.empty_like(scale), over))
        assert torch.equal(got[0], q) and torch.equal(got[1], scale) and torch.equal(over, h)
        assert torch.equal(other.cpu(), kept)
        xd, rd = inputs()
        over = rd if swap else xd
        sk.rms_norm(xd, wd, rd, out=(over, None))
        assert torch.equal(over, y)
    xd, _ = inputs()
    y, _ = sk.rms_norm(xd, wd)
    q, scale, _ = sk.rms_norm_int8(xd, wd)
    got = sk.rms_norm_int8(xd, wd, out=(torch.empty_like(q), torch.empty_like(scale), xd))
    assert torch.equal(got[0], q) and torch.equal(xd.cpu(), x)
    # y in 8 bits where x was is no input itself
    with pytest.raises(sk.SinkhornError):
        sk.rms_norm_int8(xd, wd, out=(xd.view(torch.int8)[:, :d], scale, None))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,d", OVER)
def test_norm_gradient_over_inputs(T, d, dt):
    g = rng(T * 3 + d)
    h, dh, w = norm_case(T, d, dt, g)
    dy = torch.randn(T, d, generator=g).to(h.dtype)
    wd = w.cuda()

    def inputs():
        return [padded(a, 5, 1)[0] for a in (dy, h, dh)]
    a, b, c = inputs()
    dx, dw = sk.rms_norm_backward(a, b, wd, dh=c)
    H.check(dx, H.norm_backward(dy, h, w, dh, 1e-6)[0], "dx")
    for k in range(3):
        a, b, c = inputs()
        over = (a, b, c)[k]
        got, dw2 = sk.rms_norm_backward(a, b, wd, dh=c, out=(over, torch.empty_like(dw)))
        assert torch.equal(over, dx) and torch.equal(dw2, dw)


# --- many rows

@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,d", [(2500, 96), (1023, 300), (1025, 2056), (9001, 40), (70001, 24),
                                 (131072, 8), (20000, 1100), (300001, 3)])
def test_weight_gradient_of_many_rows(T, d, dt):
    """No worker of the T rows adds up more than T / 1024 + 1 of them in fp32."""
    g = rng(T + d)
    h = torch.randn(T, d, generator=g).to(TYPES[dt])
    dy = torch.randn(T, d, generator=g).to(TYPES[dt])
    dy += 0.5           # sums that grow with T
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(TYPES[dt])
    dx, dw = sk.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda())
    wx, ww = H.norm_backward(dy, h, w, None, 1e-6, workers=min(T, 1024))
    H.check(dw, ww, "dweight")
    H.check(dx, wx, "dx")


# --- rows far into their matrices

def test_gradients_of_rows_beyond_32_bit_offsets():
    """The last of rows that lie 2^33 bytes into their matrices, in the norm with its residual and in
    both gradients; gradients over their inputs."""
    T, d, V = 131073, 32768, 70001
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    g = rng(10)
    a = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros_like(a)
    x, r, dy = (torch.randn(3, d, generator=g).bfloat16() for _ in range(3))
    w = (1 + 0.3 * torch.randn(d, generator=g)).bfloat16()
    a[-3:], b[-3:] = x.cuda(), r.cuda()
    h = H.stream(x, r)
    y, hd = sk.rms_norm(a, w.cuda(), b, out=(a, b))
    H.check(y[-3:], H.norm(h, w, 1e-6, torch.bfloat16), "y")
    assert torch.equal(hd[-3:].cpu(), h) and (y[:-3] == 0).all()
    a[-3:] = dy.cuda()
    dx, dw = sk.rms_norm_backward(a, b, w.cuda(), out=(a, torch.empty(d, device="cuda")))
    wx, ww = H.norm_backward(dy, h, w, None, 1e-6)
    H.check(dx[-3:], wx, "dx")
    H.check(dw, ww, "dweight")
    assert (dx[:-3] == 0).all()
    del b, hd, y, dx
    z = a.view(-1)[: T * d // V * V].view(-1, V)
    rows = z.shape[0]
    z[-2:] = torch.randn(2, V, generator=g).bfloat16().cuda()
    last = z[-2:].clone()
    labels = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    labels[-2:] = torch.tensor([5, V - 1], dtype=torch.int32)
    gl, ge = torch.randn(2, rows, generator=g)
    dz = sk.token_scores_backward(z, labels, gl.cuda(), ge.cuda(), out=z)
    S = H.Scores(last, labels[-2:], 1.0)
    H.check(dz[-2:], S.backward(labels[-2:], gl[-2:], ge[-2:]), "dlogits")
    assert (dz[:-2] == 0).all()


def test_labels_of_rows_without_a_distribution():
    """A row of nothing but -inf drops out whatever its label: logp 0, gradient 0, no alternatives."""
    for T, V in ((4, 300), (4, 9000), (4, 70000)):
        for dtype in TYPES.values():
            z = torch.full((T, V), -math.inf, dtype=dtype, device="cuda")
            y = torch.tensor([0, V - 1, V, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
            logp, lse, ent, index, best = sk.token_scores(z, y, top=3)
            assert (logp == 0).all() and (lse == -math.inf).all() and (ent == 0).all()
            assert (index == -1).all() and (best == -math.inf).all()
            one = torch.ones(T, device="cuda")
            assert (sk.token_scores_backward(z, y, one, one) == 0).all()
