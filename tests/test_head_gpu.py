"""The output end of a model on the GPU against its formulas in float64 (head_formulas.py, where
the tolerances are derived)."""
import math

import pytest
import torch

import head_formulas as H
import losses_formulas as L
import sinkhorn_point_cloud_amd as sk

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(autouse=True)
def _say(request):
    print(request.node.name, flush=True)
    yield


def rng(seed):
    return torch.Generator().manual_seed(seed)


def padded(x, pad, shift, fill=7.0):
    """x on the GPU in rows x.shape[1] + pad apart, the first `shift` elements into a buffer; and
    the buffer."""
    T, d = x.shape
    buf = torch.full((T * (d + pad) + shift,), fill, dtype=x.dtype)
    buf[shift:].view(T, d + pad)[:, :d].copy_(x)
    dev = buf.cuda()
    return dev[shift:].view(T, d + pad)[:, :d], dev


def gaps_kept(view, buf, fill=7.0):
    """Nothing but the rows of `view` was written in its buffer."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    off = view.storage_offset()
    torch.as_strided(mask, view.shape, view.stride(), off).fill_(False)
    return bool((buf[mask] == fill).all())


# --- the norm

# rows x values: one, odd lengths, the limits of each launch shape (chunks of 8 bf16 or 4 fp32
# values: 64, 128, 256, 512, 1024, 2048, 4096 of them and one value more or less), the longest
NORM_SIZES = [(1, 1), (3, 2), (5, 7), (9, 64), (4, 257), (130, 513), (7, 1023), (6, 1025), (3, 2047),
              (3, 2049), (2, 4096), (3, 4099), (3, 8191), (2, 8193), (2, 16384), (2, 16385),
              (1, 32767), (2, 32768), (2500, 96), (1100, 1288)]


def norm_case(T, d, dt, g, residual=True, weight=True):
    dtype = TYPES[dt]
    x = (torch.randn(T, d, generator=g) * 3).to(dtype)
    r = (torch.randn(T, d, generator=g) * torch.exp(torch.randn(d, generator=g))).to(dtype)
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    if T > 2:
        x[1] = 0
        r[1] = 0
    return x, r if residual else None, w if weight else None


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,d", NORM_SIZES)
def test_rms_norm(T, d, dt):
    g = rng(T * 3 + d)
    x, r, w = norm_case(T, d, dt, g, residual=(T + d) % 3 > 0, weight=d % 4 > 0)
    xd, _ = padded(x, T % 3, d % 5)
    rd = None if r is None else padded(r, d % 2, T % 7)[0]
    wd = None if w is None else w.cuda()
    h = H.stream(x, r)
    y, hd = sk.rms_norm(xd, wd, rd, eps=EPS)
    assert torch.equal(hd.cpu(), h)
    H.check(y, H.norm(h, w, EPS, x.dtype), "y")
    # into padded buffers, one of them an input itself
    yv, ybuf = padded(torch.zeros_like(x), 3, 1)
    target = xd if rd is None else rd
    y2, h2 = sk.rms_norm(xd, wd, rd, eps=EPS, out=(yv, target if r is not None else None))
    assert torch.equal(y2, y) and gaps_kept(yv, ybuf)
    if r is not None:
        assert h2.data_ptr() == rd.data_ptr() and torch.equal(rd.cpu(), h)
    y3, _ = sk.rms_norm(xd, wd, None, eps=EPS, out=(xd, None))
    H.check(y3, H.norm(x, w, EPS, x.dtype), "y over x")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,d", NORM_SIZES)
def test_rms_norm_int8(T, d, dt):
    g = rng(T * 5 + d)
    x, r, w = norm_case(T, d, dt, g, residual=(T + d) % 2 > 0, weight=d % 3 > 0)
    xd, _ = padded(x, d % 3, T % 4)
    rd = None if r is None else padded(r, T % 2, d % 3)[0]
    wd = None if w is None else w.cuda()
    h = H.stream(x, r)
    q, scale, hd = sk.rms_norm_int8(xd, wd, rd, eps=EPS)
    want = H.eight(h, w, EPS)
    assert torch.equal(hd.cpu(), h) and torch.equal(q.cpu(), want[0])
    H.check(scale, want[1:], "scale")
    assert q.stride(0) % 16 == 0 or T == 1
    qv, qbuf = padded(torch.zeros(T, d, dtype=torch.int8), 5, 3, fill=7)
    got = sk.rms_norm_int8(xd, wd, rd, eps=EPS, out=(qv, torch.empty_like(scale), None))
    assert got[2] is None and torch.equal(qv, q) and gaps_kept(qv, qbuf, 7)
    assert torch.equal(got[1], scale)
    q, scale = sk.quantize_int8(xd)
    want = H.eight(x, None, None)
    assert torch.equal(q.cpu(), want[0])
    H.check(scale, want[1:], "scale without a norm")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,d", NORM_SIZES)
def test_rms_norm_backward(T, d, dt):
    g = rng(T * 7 + d)
    h, dh, w = norm_case(T, d, dt, g, residual=(T + d) % 3 > 0, weight=d % 4 > 0)
    dy = torch.randn(T, d, generator=g).to(h.dtype)
    hd, dyd = padded(h, T % 3, d % 5)[0], padded(dy, d % 3, T % 2)[0]
    dhd = None if dh is None else padded(dh, 1, 0)[0]
    wd = None if w is None else w.cuda()
    dx, dw = sk.rms_norm_backward(dyd, hd, wd, dh=dhd, eps=EPS)
    wx, ww = H.norm_backward(dy, h, w, dh, EPS, workers=min(T, 256))
    H.check(dx, wx, "dx")
    assert (dw is None) == (w is None)
    if dw is not None:
        H.check(dw, ww, "dweight")
    # over each of its inputs, and dweight without a weight
    first = dx.clone()
    dw2 = torch.empty(d, device="cuda")
    for k in range(3 if dhd is not None else 2):
        a, b, c = dyd.clone(), hd.clone(), None if dhd is None else dhd.clone()
        over = (a, b, c)[k]
        got, _ = sk.rms_norm_backward(a, b, wd, dh=c, eps=EPS, out=(over, dw2))
        assert torch.equal(got, first) and got.data_ptr() == over.data_ptr()
        H.check(dw2, ww, "dweight")


@pytest.mark.parametrize("dt", TYPES)
def test_norm_of_extreme_rows(dt):
    """The largest and smallest finite values, whose squares leave fp32; infinities and NaN."""
    dtype = TYPES[dt]
    info = torch.finfo(dtype)
    d = 515
    x = torch.randn(8, d, generator=rng(1))
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = info.max / 8
    x[3] = 0
    x[4, 100] = 2.0 ** 100
    x[5, 7] = math.inf
    x[6, 514] = math.nan
    x = x.to(dtype)
    w = torch.ones(d, dtype=dtype)
    xd, wd = x.cuda(), w.cuda()
    for eps in (1e-6, 1e-30):
        y, _ = sk.rms_norm(xd, wd, eps=eps)
        keep = [0, 1, 2, 3, 4, 7]
        ref, tol = H.norm(x, w, eps, dtype)
        H.check(y[keep], (ref[keep], tol[keep]), "y")
        assert y[5].isnan().sum() == 1 and y[6].isnan().all()
        q, scale, _ = sk.rms_norm_int8(xd, wd, eps=eps)
        want = H.eight(x, w, eps)
        assert torch.equal(q.cpu()[keep], want[0][keep])
        H.check(scale, want[1:], "scale")
        assert (q[5:7] == 0).all()
        dx, _ = sk.rms_norm_backward(torch.ones_like(xd), xd, wd, eps=eps)
        assert dx[5:7].isnan().any(1).all()
        ref, tol = H.norm_backward(torch.ones_like(x), x, w, None, eps)[0]
        # a factor cubed has to stay within fp32: rows of ordinary size
        H.check(dx[[3, 7]], (ref[[3, 7]], tol[[3, 7]]), "dx")
    q, scale = sk.quantize_int8(xd)
    want = H.eight(x, None, None)
    assert torch.equal(q.cpu(), want[0])
    H.check(scale, want[1:], "scale without a norm")


@pytest.mark.parametrize("dt", TYPES)
def test_eight_bits_at_ties(dt):
    """Values that lie in the middle of two steps, to the last bit: a = 254 makes 127 p / a = p / 2,
    a = 127 p itself."""
    dtype = TYPES[dt]
    for a in (254.0, 127.0):
        row = torch.arange(-254, 255).float() / (1 if a == 254 else 2)
        x = torch.stack([row, -row, row * 2 ** -20, row * 2.0 ** 60]).to(dtype)
        q, _ = sk.quantize_int8(x.cuda())
        assert torch.equal(q.cpu(), H.eight(x, None, None)[0])


# --- the product

# tokens, K, channels
PRODUCTS = [(1, 1, 1), (1, 16, 5), (3, 15, 17), (16, 64, 16), (2, 4096, 300), (17, 100, 33), (32, 257, 64),
            (33, 1000, 31), (64, 272, 130), (65, 64, 128), (70, 1, 129), (130, 63, 200), (100, 65, 7),
            (128, 192, 256), (129, 255, 257), (200, 1500, 500), (65, 5000, 40), (300, 128, 4100),
            (500, 333, 9000), (4097, 200, 4200), (2, 131071, 20), (66, 131071, 20), (5, 200, 8200),
            (16, 4001, 16000), (33, 8000, 90), (64, 777, 33000), (3, 40, 32768), (3000, 2049, 4500),
            (257, 2311, 49152), (256, 2048, 49153),
            (250, 1999, 25000), (1023, 17, 20001)]


def eight_rows(rows, K, g, pad=0):
    """int8 rows at multiples of 16 bytes, the bytes between them not 0; largest values among them."""
    ld = (K + 15) // 16 * 16 + 16 * pad
    buf = torch.randint(-128, 128, (rows, ld), generator=g, dtype=torch.int16).to(torch.int8)
    buf[rows // 2, :K] = -128
    scale = torch.rand(rows, generator=g) * 0.01 + 1e-4
    return buf.cuda()[:, :K], scale.cuda()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,K,N", PRODUCTS)
def test_int8_linear(T, K, N, dt):
    g = rng(T + K + N)
    x, xs = eight_rows(T, K, g, pad=T % 2)
    w, ws = eight_rows(N, K, g, pad=N % 3)
    bias = torch.randn(N, generator=g).cuda() if (T + N) % 2 else None
    got = sk.int8_linear(x, xs, w, ws, bias=bias, dtype=TYPES[dt])
    want = H.linear(x, xs, w, ws, bias, TYPES[dt])
    H.check(got, want, "product")
    out, buf = padded(torch.zeros(T, N, dtype=TYPES[dt]), T % 4, N % 3)
    assert torch.equal(sk.int8_linear(x, xs, w, ws, bias=bias, out=out), got) and gaps_kept(out, buf)
    # other layouts are copied
    loose = torch.empty(K, T, dtype=torch.int8, device="cuda").t().copy_(x)
    tight = w.reshape(-1).view(N, K)
    assert torch.equal(sk.int8_linear(loose, xs, tight, ws, bias=bias, dtype=TYPES[dt]), got)


def test_sums_at_the_limit_are_exact():
    """131071 products of -128 and -128, the largest sum there is, in both kernels; alternating signs
    cancel to the last one."""
    K = 131071
    for T in (3, 70):
        x = torch.full((T, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
        w = x.clone()[:2] if T > 2 else x
        w = torch.full((2, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
        w[1, 1::2] = 127
        one = torch.ones(T, device="cuda")
        got = sk.int8_linear(x, one, w, one[:2], dtype=torch.float32).cpu().double()
        s = torch.tensor([128.0 * 128 * K, 128.0 * (128 * ((K + 1) // 2) - 127 * (K // 2))])
        assert torch.equal(got, s.float().double().expand(T, 2))


def test_scales_of_nan_and_zero():
    g = rng(5)
    for T in (4, 80):
        x, xs = eight_rows(T, 128, g)
        w, ws = eight_rows(150, 128, g)
        xs[1], ws[3], xs[2] = math.nan, 0.0, math.inf
        got = sk.int8_linear(x, xs, w, ws, dtype=torch.float32)
        assert got[1].isnan().all() and (got[0, 3] == 0) and got[2, 3].isnan()
        H.check(got[3:], H.linear(x[3:], xs[3:], w, ws, None, torch.float32), "the other rows")


# --- scores

SIZES = [(1, 1), (1, 2), (3, 7), (2, 64), (5, 129), (4, 1000), (300, 33), (9, 2049), (2, 4097),
         (3, 8191), (1, 16385), (600, 515), (2, 32000), (3, 50001), (1, 65537), (2, 131077),
         (1, 262151), (130, 65537), (129, 70001), (130, 125003), (131, 140007)]


def logits(T, V, dt, g, pad=0, shift=0):
    z = torch.randn(T, V, generator=g) * 2
    y = torch.randint(0, V, (T,), generator=g)
    z[torch.arange(T), y] += 4 + 3 * torch.randn(T, generator=g)
    y = torch.where(torch.rand(T, generator=g) < 0.15, -1, y).int()
    z = z.to(TYPES[dt])
    if T > 2 and V > 3:     # what masks do
        z[0] = -math.inf
        z[1] = torch.finfo(z.dtype).min
        z[2, ::2] = -math.inf
        y[:2] = 1
        y[2] = 3
    return padded(z, pad, shift)[0], y.cuda()


def check_scores(got, S, labels, top):
    logp, lse, ent, index, best = got
    if labels is None:
        assert logp is None
    else:
        H.check(logp, S.logp, "logp")
    H.check(lse, S.lse, "lse")
    H.check(ent, S.entropy, "entropy")
    if top:
        assert torch.equal(index.cpu(), S.index)
        H.check(best, S.best, "best")
    else:
        assert index is None and best is None


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
def test_token_scores(T, V, dt):
    g = rng(T * 17 + V)
    z, y = logits(T, V, dt, g, pad=T % 3, shift=V % 5)
    scale = 0.8
    for top in (0, (1, 5, 64, 128)[(T + V) % 4], 20):
        labels = None if (top + T) % 3 == 0 else y
        S = H.Scores(z, labels, scale, top)
        check_scores(sk.token_scores(z, labels, top=top, scale=scale), S, labels, top)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
def test_token_scores_backward(T, V, dt):
    g = rng(T * 19 + V)
    z, y = logits(T, V, dt, g, pad=V % 3, shift=T % 5)
    gl, ge = torch.randn(T, generator=g), torch.randn(T, generator=g)
    if T > 4:
        gl[3] = 0.0
        ge[3:5] = 0.0
    S = H.Scores(z, y, 1.2)
    cases = [(y, gl.cuda(), ge.cuda()), (y, gl.cuda(), None), (None, None, ge.cuda())]
    for labels, a, b in cases[:1] if V > 65000 and T > 2 else cases:
        d = sk.token_scores_backward(z, labels, a, b, scale=1.2)
        F = S if labels is not None else H.Scores(z, None, 1.2)
        H.check(d, F.backward(labels, a, b), "dlogits")
    over = z.clone()
    first = sk.token_scores_backward(over.clone(), y, gl.cuda(), ge.cuda(), scale=1.2)
    assert torch.equal(sk.token_scores_backward(over, y, gl.cuda(), ge.cuda(), scale=1.2, out=over), first)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V", [(3, 100), (4, 3000), (5, 33000), (3, 150001), (131, 140007)])
def test_alternatives_of_ties_and_crowds(T, V, dt):
    """Rows of one value, of few values, with the large ones side by side (in one thread's chunks),
    with fewer finite values than places, and of zeros of both signs."""
    g = rng(T + V)
    z = torch.randint(-2, 3, (T, V), generator=g).float()
    z[0] = 1.5
    z[1, V // 3:V // 3 + 90] = 50 + torch.arange(min(90, V - V // 3)).float()
    z[2, 3:] = -math.inf
    if T > 3:
        z[3] = torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)
    if T > 4:
        z[4] = torch.arange(V).float() / 8
        z[4, ::64] += 1e5
    z = z.to(TYPES[dt]).cuda()
    # the lowest finite value but for a few larger ones, the last of them behind all chunks
    z[-1] = torch.finfo(z.dtype).min
    z[-1, V - 1] = z[-1, V // 2] = 3.0
    for top in (1, 40, 128):
        got = sk.token_scores(z, None, top=top)
        keep = list(range(min(T, 5))) + [T - 1]
        index, best = H.alternatives(z[keep], [True] * len(keep), got[1][keep].cpu().double(), 1.0, top)
        assert torch.equal(got[3][keep].cpu(), index)
        tol = (2 * H.U + L.U) * (best.abs().nan_to_num(posinf=0.0) + got[1][keep].cpu().double().abs()[:, None])
        H.check(got[4][keep], (best, tol + H.TINY), "best")


def test_ties_of_the_longest_rows():
    """Equal values throughout rows that end at the last index there is, where what stands for none
    behind the row's end has an index beyond it."""
    for V in ((1 << 24) - 5, 1 << 24):
        z = torch.zeros(2, V, device="cuda")
        z[1, V - 3:] = 1.0
        _, lse, ent, index, best = sk.token_scores(z, top=40)
        assert index[0].tolist() == list(range(40))
        assert index[1].tolist() == [V - 3, V - 2, V - 1] + list(range(37))
        # S = V, exact sums of ones; lse and entropy are log V
        H.check(lse[:1], (torch.tensor([math.log(V)]).double(), 2 * H.U * math.log(V)), "lse")
        H.check(ent[:1], (torch.tensor([math.log(V)]).double(), 2 * H.U * math.log(V)), "entropy")
        H.check(best[0], (torch.full((40,), -math.log(V)).double(), 2 * H.U * math.log(V)), "best")


@pytest.mark.parametrize("T,V", [(5, 300), (5, 9000), (6, 70001), (200, 500)])
def test_nan_and_infinity_stay_in_their_row(T, V):
    g = rng(V)
    z, y = logits(T, V, "f32", g)
    y[:] = 2
    grad = torch.ones(T, device="cuda")
    want = sk.token_scores(z, y, top=6)
    dwant = sk.token_scores_backward(z, y, grad, grad)
    z[3, 11], z[4, 17], z[4, 40], z[4, 30] = math.nan, math.inf, math.inf, math.nan
    got = sk.token_scores(z, y, top=6)
    d = sk.token_scores_backward(z, y, grad, grad)
    keep = [t for t in range(T) if t not in (3, 4)]
    for a, b in zip((*got, d), (*want, dwant)):
        assert torch.equal(a[keep], b[keep])
    for a in (got[0], got[1], got[2], got[4], d):
        assert a[3:5].isnan().all()
    assert got[3][3, 0] == 11 and got[3][4, :3].tolist() == [30, 17, 40]
    order = H.alternatives(z[3:5], [True, True], got[1][3:5].cpu().double(), 1.0, 6)[0]
    assert torch.equal(got[3][3:5].cpu(), order)


def test_labels_out_of_range():
    for T, V in ((4, 300), (4, 70000)):
        z, y = logits(T, V, "f32", rng(V))
        z[:3] = z[3]
        y[:] = torch.tensor([V, 2 ** 31 - 1, 5, -2 ** 31], dtype=torch.int32)
        logp, lse, ent, index, best = sk.token_scores(z, y, top=3)
        assert logp[:2].isnan().all() and logp[2:].isfinite().all() and lse.isfinite().all()
        assert torch.equal(index[0], index[2]) and ent[0] == ent[2] and ent[3] == 0
        assert index[3].tolist() == [-1] * 3 and (best[3] == -math.inf).all()
        one = torch.ones(4, device="cuda")
        d = sk.token_scores_backward(z, y, one, one)
        assert d[:2].isnan().all() and d[2].isfinite().all() and (d[3] == 0).all()
        d = sk.token_scores_backward(z, y, 0 * one, one)      # no gradient of logp: the entropy's
        assert torch.equal(d[0], d[2])


def test_entropy_keeps_its_precision_near_zero():
    """One token with nearly all of the probability: H = q d of the other one and its logarithm's
    series, here (d + 1) e^-d to the second order in e^-d."""
    for V in (900, 20001, 70001):
        z = torch.full((4, V), -math.inf)
        z[:, V // 2] = 3.0
        for t, d in enumerate((10.0, 20.0, 30.0, 60.0)):
            z[t, V // 3] = 3.0 - d
        ent = sk.token_scores(z.cuda())[2].cpu().double()
        for t, d in enumerate((10.0, 20.0, 30.0, 60.0)):
            e = math.exp(-d)
            want = math.log1p(e) + d * e / (1 + e)
            # the exponential (2^-23, its exponent's three roundings), d's and the output's
            assert abs(ent[t] / want - 1) < H.U * (2 + 3 * d + 6), (V, d)


def test_gradient_coefficients_beyond_fp32():
    """As grad scale / (1 + R) leaves fp32, what has no probability still has gradient 0."""
    z = torch.full((2, 900), -math.inf)
    z[:, 3] = z[:, 700] = 0.0
    y = torch.full((2,), 3, dtype=torch.int32).cuda()
    G = torch.tensor([3e38, -2.5e38])
    d = sk.token_scores_backward((z / 2).cuda(), y, G.cuda(), None, scale=2.0).cpu().double()
    want = torch.zeros(2, 900, dtype=torch.float64)
    want[:, 3], want[:, 700] = G.double(), -G.double()
    assert torch.equal(d[:, [0, 5, 899]], want[:, [0, 5, 899]])
    assert ((d - want).abs() <= 8 * H.U * want.abs()).all()


@pytest.mark.parametrize("dt", TYPES)
def test_gradients_against_differences(dt):
    """Directional differences of the kernels' own outputs.  With step h = 2^-6 and |direction| <= 1
    the third derivatives of logp and entropy (cumulants of bounded variables times distances of at
    most 16) are below 512, the truncation below h^2 512 / 6 = 0.021 a unit of weight; the outputs'
    own error, 1e-5, is divided by h.  bf16 logits are exact on a grid of 2^-6 below 2."""
    g = rng(8)
    T, V, h = 5, 700, 2.0 ** -6
    z = (torch.randint(-64, 65, (T, V), generator=g).float() / 64).to(TYPES[dt])
    dir_ = torch.randint(-1, 2, (T, V), generator=g).float()
    y = torch.randint(0, V, (T,), generator=g).int().cuda()
    wl, we = torch.rand(T, generator=g), torch.rand(T, generator=g)
    d = sk.token_scores_backward(z.cuda(), y, wl.cuda(), we.cuda()).float().cpu()

    def total(s):
        o = sk.token_scores((z.float() + s * dir_).to(z.dtype).cuda(), y)
        return (wl * o[0].cpu() + we * o[2].cpu()).double().sum()
    diff = (total(h) - total(-h)) / (2 * h)
    # entries of the gradient: a rounding to the type each, of values that sum to at most 2 T
    slack = (wl + we).sum() * 0.021 + T * 2e-5 / h + H.HALF[z.dtype] * d.abs().sum()
    assert abs(diff - (d * dir_).double().sum()) < slack
    x = (torch.randn(6, 64, generator=g)).to(TYPES[dt])
    w = torch.ones(64, dtype=x.dtype)
    dy = torch.randn(6, 64, generator=g).to(x.dtype)
    dx, dw = sk.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda())
    move = torch.randn(64, generator=g)
    y0 = H.norm(x, None, 1e-6, torch.float64)[0]
    assert abs((dw.cpu().double() * move).sum() - (y0 * move * dy.double()).sum()) < 1e-4


# --- the calls around them

def score_call(T, V, dt="f32", seed=3, top=9):
    z, y = logits(T, V, dt, rng(seed))
    z = z.contiguous()

    def call(out=None, workspace=None):
        return sk.token_scores(z, y, top=top, out=out, workspace=workspace)
    return z, call, call(), sk.head_workspace_bytes(2, T, V, top, dt == "bf16")


def score_grad_call(T, V, dt="f32", seed=4):
    z, y = logits(T, V, dt, rng(seed))
    z = z.contiguous()
    a, b = torch.randn(2, T, generator=rng(1)).cuda()

    def call(out=None, workspace=None):
        return (sk.token_scores_backward(z, y, a, b, out=None if out is None else out[0],
                                         workspace=workspace),)
    return z, call, call(), sk.head_workspace_bytes(3, T, V, 0, dt == "bf16")


def norm_grad_call(T, d, dt="f32", seed=5):
    h, dh, w = norm_case(T, d, dt, rng(seed))
    h, dh, w = h.cuda(), dh.cuda(), w.cuda()
    dy = torch.randn(T, d, generator=rng(2)).to(h.dtype).cuda()

    def call(out=None, workspace=None):
        return sk.rms_norm_backward(dy, h, w, dh=dh, out=out, workspace=workspace)
    return h, call, call(), sk.head_workspace_bytes(0, T, d, 0, dt == "bf16")


def norm_call(T, d, dt="f32", seed=6):
    x, r, w = norm_case(T, d, dt, rng(seed))
    x, r, w = x.cuda(), r.cuda(), w.cuda()

    def call(out=None, workspace=None):
        a = sk.rms_norm(x, w, r, out=None if out is None else out[:2])
        b = sk.rms_norm_int8(x, w, r, out=None if out is None else out[2:5])
        return (*a, *b)
    return x, call, call(), 0


def product_call(T, K, N, dt="f32", seed=7):
    x, xs = eight_rows(T, K, rng(seed))
    w, ws = eight_rows(N, K, rng(seed + 1))

    def call(out=None, workspace=None):
        return (sk.int8_linear(x, xs, w, ws, dtype=TYPES[dt], out=None if out is None else out[0],
                               workspace=workspace),)
    return xs, call, call(), sk.head_workspace_bytes(1, T, N, K, dt == "bf16")


CALLS = [(score_call, (40, 1000)), (score_call, (6, 70001, "bf16")), (score_call, (140, 70001)),
         (score_grad_call, (40, 1000, "bf16")), (score_grad_call, (6, 70001)), (norm_grad_call, (700, 500)),
         (norm_grad_call, (50, 9000, "bf16")), (norm_call, (40, 1000)), (norm_call, (9, 9001, "bf16")),
         (product_call, (5, 300, 1000)), (product_call, (200, 3000, 150, "bf16")),
         (product_call, (4097, 256, 4096))]


@pytest.mark.parametrize("make,size", CALLS)
def test_graph_replays(make, size):
    z, call, out, _ = make(*size)
    first = z.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    outs = tuple(torch.empty_strided(o.shape, o.stride(), dtype=o.dtype, device=o.device) for o in out)
    with torch.cuda.graph(graph, stream=side):
        call(outs)
    for turn in range(4):
        z.copy_((first.float() * (1 + turn)).to(z.dtype))
        eager = call()
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, eager)):
            assert torch.equal(a, b) or torch.equal(a.isnan(), b.isnan()), (turn, i)
            assert torch.equal(a.nan_to_num(), b.nan_to_num()), (turn, i)


@pytest.mark.parametrize("make,size", CALLS)
def test_two_streams_at_once(make, size):
    _, call, _, _ = make(*size)
    want = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(call())
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, want):
            assert torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("make,size", CALLS)
def test_workspace_is_checked_and_not_overrun(make, size):
    _, call, out, need = make(*size)
    if not need:
        return
    with pytest.raises(ValueError):
        call(out, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        call(out, workspace=torch.empty(need, dtype=torch.uint8))
    big = torch.full((need + 4096 + 3,), 0xA5, dtype=torch.uint8, device="cuda")
    room = big[3:3 + need]
    got = call(workspace=room)
    for a, b in zip(got, out):
        assert torch.equal(a.nan_to_num(), b.nan_to_num())
    assert (big[:3] == 0xA5).all() and (big[3 + need:] == 0xA5).all()


def test_overlaps_are_refused():
    x = torch.randn(64, 256, device="cuda")
    for call in (lambda: sk.rms_norm(x[:32], out=(x[1:33], None)),
                 lambda: sk.rms_norm(x[:32], None, x[32:], out=(x[:32], x[:32])),
                 lambda: sk.rms_norm_backward(x[:32], x[32:], out=(x[8:40], None)),
                 lambda: sk.token_scores_backward(x[:32], None, None, x[40, :32], out=x[1:33]),
                 lambda: sk.token_scores(x, out=(None, x[0, :64], None, None, None))):
        with pytest.raises(sk.SinkhornError) as e:
            call()
        assert e.value.status == sk.SK_ERR_INVALID_ARG


def test_no_rows():
    z = torch.zeros(0, 16, device="cuda")
    none = z[:, 0].contiguous()
    assert sk.rms_norm(z)[0].shape == (0, 16)
    q, scale, _ = sk.rms_norm_int8(z)
    assert q.shape == (0, 16) and scale.shape == (0,)
    dx, dw = sk.rms_norm_backward(z, z, torch.ones(16, device="cuda"))
    assert dx.shape == (0, 16) and (dw == 0).all()
    w, ws = sk.quantize_int8(torch.ones(5, 16, device="cuda"))
    assert sk.int8_linear(q, scale, w, ws).shape == (0, 5)
    out = sk.token_scores(z, none.int(), top=3)
    assert [tuple(o.shape) for o in out] == [(0,), (0,), (0,), (0, 3), (0, 3)]
    assert sk.token_scores_backward(z, none.int(), none, none).shape == (0, 16)


def test_rows_beyond_32_bit_offsets():
    """The last of rows that lie 2^33 bytes into their matrices."""
    T, d, V = 131073, 32768, 70001
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    g = rng(9)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(3, d, generator=g).bfloat16()
    x[-3:] = tail.cuda()
    q, scale = sk.quantize_int8(x)
    assert torch.equal(q[-3:].cpu(), H.eight(tail, None, None)[0])
    y, _ = sk.rms_norm(x)
    H.check(y[-3:], H.norm(tail, None, 1e-6, torch.bfloat16), "y")
    del y
    w, ws = eight_rows(40, d, g)
    got = sk.int8_linear(q, scale, w, ws, dtype=torch.float32)
    H.check(got[-3:], H.linear(q[-3:], scale[-3:], w, ws, None, torch.float32), "product")
    del q
    # a product whose result is what lies that far
    N = 1 << 24
    few, fs = eight_rows(66, 16, g)
    many, ms = eight_rows(N, 16, g)
    out = sk.int8_linear(few, fs, many, ms)
    H.check(out[-2:, -50:], H.linear(few[-2:], fs[-2:], many[-50:], ms[-50:], None, torch.bfloat16),
            "far results")
    del many, out
    z = x.view(-1)[: T * d // V * V].view(-1, V)
    rows = z.shape[0]
    z[-2:] = torch.randn(2, V, generator=g).bfloat16().cuda()
    y = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    y[-2:] = torch.tensor([5, V - 1], dtype=torch.int32)
    got = sk.token_scores(z, y, top=7)
    S = H.Scores(z[-2:], y[-2:], 1.0, 7)
    check_scores([o[-2:] for o in got], S, y[-2:], 7)


def test_on_another_device_argument_checks():
    x = torch.randn(4, 32, device="cuda")
    with pytest.raises(ValueError):
        sk.rms_norm(x, torch.ones(32))
    with pytest.raises(TypeError):
        sk.rms_norm(x, torch.ones(32, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        sk.rms_norm(x, None, x[:3])
    with pytest.raises(ValueError):
        sk.token_scores(x, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(sk.SinkhornError):
        sk.token_scores(x, top=129)
    with pytest.raises(sk.SinkhornError):
        sk.token_scores_backward(x, None, torch.ones(4, device="cuda"), None)


# --- together, as they are used

@pytest.mark.parametrize("dt", TYPES)
def test_a_frozen_models_output_end(dt):
    """Hidden states to logits in 8 bits to scores, and the losses that take them: the teacher's
    top tokens for distillation, its log-probabilities for the policy loss's old and reference."""
    g = rng(12)
    T, d, V, K = 150, 200, 1500, 12
    x, r, w = norm_case(T, d, dt, g)
    head = (torch.randn(V, d, generator=g) * 0.3).to(TYPES[dt]).cuda()
    w8, ws = sk.quantize_int8(head)
    q, scale, h = sk.rms_norm_int8(x.cuda(), w.cuda(), r.cuda())
    logits_ = sk.int8_linear(q, scale, w8, ws, dtype=torch.float32)
    want = H.eight(H.stream(x, r), w, 1e-6)
    assert torch.equal(q.cpu(), want[0])
    H.check(logits_, H.linear(q, scale, w8, ws, None, torch.float32), "logits")
    # the 8-bit logits are near those of the layer itself: half a step of 127 in either factor of
    # each product, a / 254 and b / 254 for the largest |a| and |b| of their rows
    y = H.norm(H.stream(x, r), w, 1e-6, torch.float64)[0]
    full = y @ head.cpu().double().t()
    a, b = y.abs().amax(1)[:, None] / 254, head.cpu().double().abs().amax(1)[None] / 254
    bound = a * head.cpu().double().abs().sum(1)[None] + b * y.abs().sum(1)[:, None] + d * a * b
    assert ((logits_.cpu().double() - full).abs() <= bound * 1.001).all()
    labels = torch.randint(0, V, (T,), generator=g).int().cuda()
    labels[::9] = -1
    old, lse, ent, index, best = sk.token_scores(logits_, labels, top=K)
    check_scores((old, lse, ent, index, best), H.Scores(logits_, labels, 1.0, K), labels, K)
    # the same log-probabilities as the losses', and their gradient without the entropy's
    assert torch.allclose(old, sk.token_logprobs(logits_, labels)[0], rtol=0, atol=1e-6)
    student = (logits_ + 0.3 * torch.randn(T, V, generator=g).cuda()).to(TYPES[dt])
    loss, _ = sk.distill_loss(student, index, best, teacher_lse=torch.zeros_like(lse))
    (value, tol), _ = L.distill(student, index, best, teacher_lse=torch.zeros(T))
    H.check(loss, (value, tol), "distillation")
    assert (loss[labels < 0] == 0).all()        # rows without entries
    off = torch.tensor([0, 70, T]).cuda()
    _, kl, logp, dz = sk.policy_loss(student, labels, off, old, torch.ones(2, device="cuda"), ref=old, kl=0.1)
    same = sk.policy_loss(logits_, labels, off, old, torch.ones(2, device="cuda"), ref=old, kl=0.1)
    assert same[1].abs().max() < 1e-9 and (kl > 0).all()
    # an entropy bonus beside the policy's gradient
    bonus = sk.token_scores_backward(student, labels, None, torch.full((T,), -0.01, device="cuda"))
    assert bonus.shape == dz.shape and bonus.isfinite().all()
