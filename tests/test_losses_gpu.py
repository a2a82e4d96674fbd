"""The losses over logits on the GPU against their formulas in float64 (losses_formulas.py, where
the tolerances are derived)."""
import math

import pytest
import torch

import losses_formulas as F
import sinkhorn_point_cloud_amd as sk

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# rows x values: one of each, odd lengths, row starts at every alignment, rows that one wave, one
# work-group or several hold, lengths beside the limits of each launch shape
SIZES = [(1, 1), (1, 2), (3, 7), (2, 64), (5, 129), (4, 1000), (300, 33), (9, 2049), (2, 4097),
         (3, 8191), (1, 16385), (600, 515), (2, 32000), (3, 50001), (1, 65537), (2, 131077),
         (1, 262151)]


# more rows than are split, as long as registers, registers and LDS, and neither hold (the last
# multiple of 16 bytes, one value more or less, and beyond)
SIZES += [(130, 65537), (129, 70001), (130, 125003), (131, 140007)]


@pytest.fixture(autouse=True)
def _say(request):
    print(request.node.name, flush=True)
    yield


def rng(seed):
    return torch.Generator().manual_seed(seed)


def make(T, V, dtype, g, pad=0, shift=0):
    """Logits [T, V] on the GPU, rows V + pad apart, the first `shift` elements into a buffer; and
    labels, some of them not scored, their logits raised."""
    z = torch.randn(T, V, generator=g) * 2
    y = torch.randint(0, V, (T,), generator=g)
    z[torch.arange(T), y] += 4 + 3 * torch.randn(T, generator=g)
    y = torch.where(torch.rand(T, generator=g) < 0.15, -1, y)
    buf = torch.full((T * (V + pad) + shift,), 7.0, dtype=dtype)
    view = buf[shift:].view(T, V + pad)[:, :V]
    view.copy_(z.to(dtype))
    dev = buf.cuda()
    return dev[shift:].view(T, V + pad)[:, :V], y.int().cuda()


def odd_rows(z, y):
    """What masks do: a row of nothing, a row of the lowest finite value, a masked label, masked
    columns."""
    T, V = z.shape
    if T > 2 and V > 3:
        z[0] = -math.inf
        z[1] = torch.finfo(z.dtype).min
        z[2, ::2] = -math.inf
        y[:2] = 1
        y[2] = 3
    return z, y


def cut(T, n, g, first=0, last=None):
    last = T if last is None else last
    inner = torch.sort(torch.randint(first, last + 1, (n - 1,), generator=g)).values
    return torch.cat([torch.tensor([first]), inner, torch.tensor([last])]).cuda()


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
def test_token_logprobs(T, V, dt):
    g = rng(T * 7 + V)
    z, y = make(T, V, TYPES[dt], g, pad=T % 3, shift=V % 5)
    odd_rows(z, y)
    scale = 0.8
    logp, lse = sk.token_logprobs(z, y, scale=scale)
    R = F.Rows(z, scale)
    F.check(logp, R.logp(y), "logp")
    want = torch.where(y.cpu() >= 0, R.lse, 0.0)
    F.check(lse, (want, F.eps_sum(V) + 2 * F.U * torch.where(want.isfinite(), want.abs(), 0.0)),
            "lse")
    grad = torch.randn(T, generator=g).cuda()
    if T > 4:
        grad[3] = 0.0
    d = sk.token_logprobs_backward(z, y, grad, scale=scale)
    coef = grad.cpu().double()
    F.check(d, R.label_grad(y, coef, torch.zeros(T, dtype=torch.float64)), "dlogits")
    only = sk.losses.load_library()     # either output alone
    alone = torch.empty_like(lse)
    ws = torch.empty(sk.losses_workspace_bytes(0, T, V, 0, dt == "bf16"), dtype=torch.uint8,
                     device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    ld = max(V, z.stride(0))
    assert only.sinkhorn_token_logprobs(z.data_ptr(), dt == "bf16", ld, y.data_ptr(), T, V, scale,
                                        None, alone.data_ptr(), ws.data_ptr(), ws.numel(), st) == 0
    assert torch.equal(alone, lse)


POLICY = [dict(), dict(mean=False, kl=0.1), dict(ref=True, kl=0.07, clip=(0.1, 0.3)),
          dict(ref=True, kl=0.2, weights=True, scale=1.3, per_seq=True)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
def test_policy_loss(T, V, dt):
    g = rng(T * 11 + V)
    z, y = make(T, V, TYPES[dt], g, pad=(V + 1) % 3, shift=V % 3)
    odd_rows(z, y)
    n = min(4, T)
    off = cut(T, n, g, last=T - T // 10)
    kw = dict(POLICY[(T + V) % 4])
    per_seq, scale = kw.pop("per_seq", False), kw.get("scale", 1.0)
    lp = F.Rows(z, scale).logp(y)[0]
    lp = torch.where(lp.isfinite(), lp, -20.0)
    old = (lp + 0.25 * torch.randn(T, generator=g).double()).float().cuda()
    ref = (lp + 0.3 * torch.randn(T, generator=g).double()).float().cuda() if kw.pop("ref", 0) \
        else None
    if kw.pop("weights", 0):
        kw["weights"] = torch.rand(n, generator=g).cuda()
    adv = torch.randn(n if per_seq else T, generator=g).cuda()
    if ref is not None and T > 2 and V > 3:
        y[2] = -1       # a masked label has an infinite KL: its own test
    got = sk.policy_loss(z, y, off, old, adv, ref=ref, **kw)
    want = F.policy(z, y, off, old, adv, ref=ref, **kw)
    border = want[4]
    assert border[torch.isfinite(border)].min() > 1e-5      # no decision left to the last bits
    inside = torch.arange(T) < int(off[-1])
    lpv, lpt = want[2]
    F.check(got[2], (torch.where(inside, lpv, 0.0), lpt), "logp")
    for k, name in ((0, "loss"), (1, "kl"), (3, "dlogits")):
        F.check(got[k], want[k], name)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
def test_preference_loss(T, V, dt):
    g = rng(T * 13 + V)
    z, y = make(T, V, TYPES[dt], g, pad=V % 4, shift=T % 4)
    z, y = odd_rows(z, y)
    if T > 2 and V > 3:
        y[2] = 4 if V > 4 else -1          # a masked label's sum is infinite: its own test
        z[2, 4:5] = 1.0
    off = cut(T, 2 * min(3, (T + 1) // 2), g, last=T - T // 10)
    P = (off.numel() - 1) // 2
    kw = [dict(), dict(kind="square", beta=0.5, mean=True), dict(beta=0.3, smoothing=0.2),
          dict(mean=True, beta=0.4, scale=0.7)][(T + V) % 4]
    if (T + V) % 3 == 0:
        kw = dict(kw, weights=torch.rand(P, generator=g).cuda())
    lp = F.Rows(z, kw.get("scale", 1.0)).logp(y)[0]
    ref = (lp + 0.3 * torch.randn(T, generator=g).double()).float().cuda() if V % 2 else None
    got = sk.preference_loss(z, y, off, ref, **kw)
    want = F.preference(z, y, off, ref, **kw)
    inside = torch.arange(T) < int(off[-1])
    F.check(got[2], (torch.where(inside, want[2][0], 0.0), want[2][1]), "logp")
    for k, name in ((0, "loss"), (1, "reward"), (3, "dlogits")):
        F.check(got[k], want[k], name)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V", SIZES)
def test_distill_loss(T, V, dt):
    g = rng(T * 17 + V)
    z, y = make(T, V, TYPES[dt], g, pad=V % 2, shift=(T + 1) % 5)
    if T > 2 and V > 3:
        z[0] = -math.inf
        z[1] = torch.finfo(z.dtype).min
    K = min([1, 3, 20, 64, 65, 200, 1024][(T + V) % 7], 2 * V)
    idx = torch.randint(0, V, (T, K), generator=g)
    idx[:, 0] = V - 1                       # the last value, and where K > V tokens stand twice
    if K > 2:
        idx[0, 1] = idx[0, 2]
        idx[-1, 1] = -1
    u = z.float().cpu().gather(1, idx.clamp(min=0)) + 0.5 * torch.randn(T, K, generator=g)
    u = torch.where(u.isfinite() & (u > -1e30), u, torch.randn(T, K, generator=g))
    if T > 3 and K > 1:
        u[3, :] = -math.inf
        u[2, 1] = -math.inf
    tau = [1.0, 2.0, 0.7][(T + V) % 3]
    lse = torch.logsumexp(u.double() / tau, 1).float() + 0.1 if V % 2 else None
    if lse is not None:
        lse = torch.where(lse.isfinite(), lse, 1.0).cuda()
    w = None
    if T % 2 == 0:
        w = torch.rand(T, generator=g)
        w[-1] = 0.0
        w = w.cuda()
    args = (z, idx.int().cuda(), u.cuda())
    got = sk.distill_loss(*args, teacher_lse=lse, temperature=tau, weights=w)
    want = F.distill(*args, teacher_lse=lse, temperature=tau, weights=w)
    F.check(got[0], want[0], "loss")
    F.check(got[1], want[1], "dlogits")
    assert torch.equal(sk.distill_loss(*args, teacher_lse=lse, temperature=tau, weights=w,
                                       grad=False)[0], got[0])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,E,K,G", [
    (1, 1, 1, 0), (1, 8, 2, 0), (7, 5, 1, 3), (64, 8, 2, 1), (1000, 16, 2, 5), (333, 31, 4, 0),
    (513, 64, 6, 9), (100, 65, 8, 2), (777, 160, 8, 70), (2000, 256, 8, 3), (90, 257, 1, 4),
    (65, 512, 64, 2), (40, 1000, 3, 1), (33, 1024, 8, 0), (5000, 4, 4, 200), (20000, 8, 2, 2)])
def test_balance_loss(T, E, K, G, dt):
    g = rng(T + E)
    z, _ = make(T, E, TYPES[dt], g, pad=T % 3, shift=E % 3)
    idx = z.float().cpu().topk(min(K, E), dim=1).indices
    if K > E:
        idx = torch.cat([idx, idx[:, :K - E]], 1)
    if T > 5:
        idx[1] = -1
        idx[2, 0] = -1
        z[3] = -math.inf
        z[4] = torch.finfo(z.dtype).min
        z[5, :1] = -math.inf
    off = None
    if G:
        off = cut(T, G, g, first=min(1, T - 1), last=T - T // 8)
    a = (z, idx.int().cuda(), off)
    got = sk.balance_loss(*a, balance=0.3, z=0.02)
    want = F.balance(*a, balance=0.3, z=0.02)
    assert torch.equal(got[2].cpu(), want[2])
    for k, name in ((0, "loss"), (1, "zloss"), (3, "dlogits")):
        F.check(got[k], want[k], name)
    again = sk.balance_loss(*a, balance=0.3, z=0.02, grad=False)
    assert again[3] is None and all(torch.equal(x, y) for x, y in zip(got[:3], again[:3]))


def test_distill_of_a_long_list_on_a_long_row():
    # a list that leaves no room for a row in LDS
    g = rng(21)
    T, V, K = 129, 80003, 1024
    z, _ = make(T, V, torch.float32, g)
    idx = torch.randint(0, V, (T, K), generator=g)
    idx[:, 700] = idx[:, 3]
    u = torch.randn(T, K, generator=g)
    args = (z, idx.int().cuda(), u.cuda())
    got, want = sk.distill_loss(*args), F.distill(*args)
    F.check(got[0], want[0], "loss")
    F.check(got[1], want[1], "dlogits")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V", [(9, 900), (9, 40000), (9, 90001), (133, 70001)])
def test_one_value_has_nearly_all_of_the_probability(T, V, dt):
    """log q and 1 - q near 0 to their own size.  The rest of the sum, without the largest term, is
    off relative by the terms' own errors (arguments up to 40: 3 ln 2 2^-24 * 40, and 2^-23) and
    its additions, as eps_S; the logarithm and the last roundings add 4 units."""
    g = rng(T + V)
    z = (torch.randn(T, V, generator=g)).to(TYPES[dt])
    y = torch.randint(0, V, (T,), generator=g)
    y[0], y[1], y[2] = 0, V - 1, 5
    z[torch.arange(T), y] = torch.linspace(12, 27, T).to(TYPES[dt])
    z, y = z.cuda(), y.int().cuda()
    R = F.Rows(z)
    x = R.z.clone()
    x[torch.arange(T), y.cpu().long()] = -math.inf
    rest = torch.exp(x - R.M[:, None]).sum(1)
    logp = -torch.log1p(rest)
    rel = F.U * (2 + 2.1 * 40 + V / 512 + 100 + 4)
    got, _ = sk.token_logprobs(z, y)
    F.check(got, (logp, rel * logp.abs()), "logp")
    far = rest / (1 + rest)               # 1 - q at the label
    want = -R.q
    want[torch.arange(T), y.cpu().long()] = far
    # bf16: the rounding of each value, fp32: within eps_S and the argument's error, relative
    tol = (rel + F.HALF[z.dtype]) * 1.01 * want.abs()
    F.check(sk.token_logprobs_backward(z, y, torch.ones(T).cuda()), (want, tol), "dlogits")
    off = torch.tensor([0, T]).cuda()
    loss, reward, lp, d = sk.preference_loss(z, y, torch.tensor([0, T, T]).cuda(), kind="square",
                                             beta=1.0)
    slope = 2 * (logp.sum() - 0.5)
    F.check(d, (want * slope, tol * slope.abs() + rel * (want * slope).abs()), "pairs")
    _, _, _, d = sk.policy_loss(z, y, off, got, torch.ones(T).cuda(), mean=False)
    F.check(d, (-want, tol + 4 * rel * want.abs()), "policy")
    u = torch.zeros(T, 1).cuda()
    loss, d = sk.distill_loss(z, y[:, None], u)
    F.check(loss, (-logp, rel * logp.abs()), "loss")
    F.check(d, (-want, tol), "distill")


def test_one_token_many_times():
    # every entry the same token, and pairs of them on either side of a wave's 64 entries
    g = rng(22)
    for V, K in ((300, 200), (9000, 130), (40, 64)):
        z, _ = make(5, V, torch.float32, g)
        idx = torch.full((5, K), 7)
        idx[1] = torch.arange(K) % (K // 2) % V
        idx[2] = torch.arange(K) // 2 % V
        idx[3, ::3] = -1
        u = torch.randn(5, K, generator=g)
        args = (z, idx.int().cuda(), u.cuda())
        got, want = sk.distill_loss(*args), F.distill(*args)
        F.check(got[0], want[0], "loss")
        F.check(got[1], want[1], "dlogits")
        for _ in range(3):
            assert torch.equal(sk.distill_loss(*args)[1], got[1])


# ------------------------------------------------------------------ every operator

def _setup(name, T=37, V=900, dt="bf16", seed=5):
    """(call(out) -> outputs, fresh outputs, logits, per-row outputs' positions)."""
    g = rng(seed)
    z, y = make(T, V, TYPES[dt], g)
    off = torch.tensor([3, 10, 10, 21, 30]).cuda()
    new = lambda *s, dtype=torch.float32: torch.full(s, 7, dtype=dtype, device="cuda")  # noqa: E731
    lp = F.Rows(z).logp(y)[0]
    old = (lp + 0.2 * torch.randn(T, generator=g).double()).float().cuda()
    d = new(T, V, dtype=z.dtype)
    if name == "policy":
        adv = torch.randn(T, generator=g).cuda()
        return (lambda out, z=z, **k: sk.policy_loss(z, y, off, old, adv, ref=old, kl=0.1, out=out,
                                                     **k), (new(4), new(4), new(T), d), z, (2, 3))
    if name == "preference":
        return (lambda out, z=z, **k: sk.preference_loss(z, y, off, old, out=out, **k),
                (new(2), new(4), new(T), d), z, (2, 3))
    if name == "distill":
        idx = torch.randint(0, V, (T, 9), generator=g).int().cuda()
        u = torch.randn(T, 9, generator=g).cuda()
        return (lambda out, z=z, **k: sk.distill_loss(z, idx, u, out=out, **k), (new(T), d), z, ())
    if name == "balance":
        idx = torch.randint(0, V, (T, 4), generator=g).int().cuda()
        return (lambda out, z=z, **k: sk.balance_loss(z, idx, off, z=0.1, out=out, **k),
                (new(4), new(4), new(4, V, dtype=torch.int32), d), z, (3,))
    grad = torch.randn(T, generator=g).cuda()

    def both(out, z=z, **k):
        logp, lse = sk.token_logprobs(z, y, out=None if out is None else out[:2], **k)
        return logp, lse, sk.token_logprobs_backward(z, y, grad,
                                                     out=None if out is None else out[2], **k)
    return both, (new(T), new(T), d), z, ()


NAMES = ("logp", "policy", "preference", "distill", "balance")
SHAPES = [(37, 900, "bf16"), (37, 1001, "f32")]
LARGE = [(40, 70009, "bf16"), (31, 20001, "f32"), (130, 70001, "f32"), (31, 40001, "f32")]


def sizes_for(name):
    return SHAPES if name == "balance" else SHAPES + LARGE


EACH = [(n, s) for n in NAMES for s in sizes_for(n)]


@pytest.mark.parametrize("name,size", EACH)
def test_callers_buffers_and_rows_outside(name, size):
    call, out, z, rows = _setup(name, *size)
    fresh = call(None)
    got = call(out)
    for a, b in zip(got, out):
        assert a is b
    for i, (a, b) in enumerate(zip(fresh, out)):
        if i in rows:       # rows 0..2 and from 30 on belong to no sequence
            assert (a[:3] == 0).all() and (a[30:] == 0).all()
            assert (b[:3] == 7).all() and (b[30:] == 7).all()
            a, b = a[3:30], b[3:30]
        assert torch.equal(a, b), i


@pytest.mark.parametrize("name,size", EACH)
def test_gradient_over_the_logits(name, size):
    call, out, z, _ = _setup(name, *size)
    call(out)
    mine = z.clone()
    outs = [o.clone().fill_(7) for o in out]
    outs[-1] = mine
    rows_left = z.clone()
    call(tuple(outs), z=mine)
    if name in ("policy", "preference", "balance"):
        assert torch.equal(mine[:3], rows_left[:3]) and torch.equal(mine[30:], rows_left[30:])
        assert torch.equal(mine[3:30], out[-1][3:30])
    else:
        assert torch.equal(mine, out[-1])
    for a, b in zip(outs[:-1], out[:-1]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name,size", EACH)
def test_gradient_at_another_alignment(name, size):
    call, out, z, _ = _setup(name, *size)
    call(out)
    T, V = z.shape
    for pad, shift in ((3, 1), (0, 3), (8, 0)):
        buf = torch.full((T * (V + pad) + shift,), 7, dtype=z.dtype, device="cuda")
        d = buf[shift:].view(T, V + pad)[:, :V]
        call((*[o.clone() for o in out[:-1]], d))
        assert torch.equal(d, out[-1])
        if pad:
            assert (buf[shift:].view(T, V + pad)[:, V:] == 7).all()
        assert (buf[:shift] == 7).all()


@pytest.mark.parametrize("name,size", EACH)
def test_strided_logits(name, size):
    call, _, z, _ = _setup(name, *size)
    want = call(None)
    T, V = z.shape
    # 128 bytes more: the rows start at the same alignment, and the sums group alike
    wide = torch.full((T, V + 128 // z.element_size()), math.nan, dtype=z.dtype, device="cuda")
    wide[:, :V] = z
    columns = z.t().contiguous().t()
    for other in (wide[:, :V], columns):
        for a, b in zip(call(None, z=other), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name,size", EACH)
def test_graph_replays(name, size):
    call, out, z, _ = _setup(name, *size)
    first = z.clone()
    call(out)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    outs = tuple(o.clone() for o in out)
    with torch.cuda.graph(graph, stream=side):
        call(outs)
    g = rng(9)
    for turn in range(4):
        z.copy_((first.float() + turn * torch.randn(z.shape, generator=g).cuda()).to(z.dtype))
        eager = call(tuple(o.clone() for o in outs))
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, eager)):
            if a.shape[0] == z.shape[0] and name in ("policy", "preference", "balance"):
                a, b = a[3:30], b[3:30]
            assert torch.equal(a, b), (turn, i)


@pytest.mark.parametrize("name,size", EACH)
def test_two_streams_at_once(name, size):
    call, _, z, _ = _setup(name, *size)
    want = [call(None), call(None, z=(z.float() * 0.5).to(z.dtype))]
    half = (z.float() * 0.5).to(z.dtype)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(None, z=(z, half)[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for a, b in zip(r, want[i]):
                assert torch.equal(a, b)


@pytest.mark.parametrize("name,size", EACH)
def test_nan_and_infinity_stay_in_their_row(name, size):
    call, _, z, _ = _setup(name, *size)
    want = call(None)[-1]
    z[12, 5] = math.nan
    z[14, 7] = math.inf
    got = call(None)[-1]
    keep = torch.ones(z.shape[0], dtype=torch.bool)
    if name == "preference":    # its sequence's sum is NaN, and with it the pair's rows
        keep[10:30] = False
    else:
        keep[12] = keep[14] = False
    y_used = got[12].isnan().all() or (got[12] == 0).all()
    assert y_used and (got[14].isnan().any() or (got[14] == 0).all())
    assert torch.equal(got[keep.cuda()], want[keep.cuda()])


@pytest.mark.parametrize("name", NAMES)
def test_workspace_is_checked(name):
    call, out, z, _ = _setup(name)
    with pytest.raises(ValueError):
        call(out, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        call(out, workspace=torch.empty(1 << 22, dtype=torch.uint8))
    big = torch.empty((1 << 22) + 3, dtype=torch.uint8, device="cuda")[3:]
    call(out, workspace=big)


@pytest.mark.parametrize("name", NAMES)
def test_overlapping_gradient_is_refused(name):
    call, out, z, _ = _setup(name)
    T, V = z.shape
    buf = torch.zeros(2 * T, V, dtype=z.dtype, device="cuda")
    src = buf[:T]
    src.copy_(z)
    with pytest.raises(sk.SinkhornError) as e:
        call((*out[:-1], buf[1:T + 1]), z=src)
    assert e.value.status == sk.SK_ERR_INVALID_ARG
    # columns of one buffer side by side do not overlap
    side = torch.zeros(T, 2 * V, dtype=z.dtype, device="cuda")
    side[:, :V] = z
    call((*out[:-1], side[:, V:]), z=side[:, :V])
    ref = call(None)
    rows = slice(3, 30)
    assert torch.equal(side[rows, V:], ref[-1][rows])


@pytest.mark.parametrize("name", NAMES)
def test_no_rows(name):
    dev = "cuda"
    z = torch.zeros(0, 16, device=dev)
    y = torch.zeros(0, dtype=torch.int32, device=dev)
    x = torch.zeros(0, device=dev)
    off = torch.zeros(5, dtype=torch.int64, device=dev)
    if name == "logp":
        logp, lse = sk.token_logprobs(z, y)
        assert logp.shape == (0,) and sk.token_logprobs_backward(z, y, x).shape == (0, 16)
    elif name == "policy":
        got = sk.policy_loss(z, y, off, x, x)
        assert (got[0] == 0).all() and (got[1] == 0).all() and got[3].shape == (0, 16)
    elif name == "preference":
        got = sk.preference_loss(z, y, off)
        # an empty pair has the log-ratio 0: log 2, rounded once
        assert (got[0] - math.log(2)).abs().max() <= 2.0 ** -24 and (got[1] == 0).all()
    elif name == "distill":
        got = sk.distill_loss(z, y.view(0, 1).expand(0, 4), x.view(0, 1).expand(0, 4))
        assert got[0].shape == (0,) and got[1].shape == (0, 16)
    else:
        got = sk.balance_loss(z, y.view(0, 1).expand(0, 2), off)
        assert (got[0] == 0).all() and (got[2] == 0).all() and got[2].shape == (4, 16)


def test_labels_and_indices_out_of_range():
    g = rng(3)
    for T, V in ((6, 300), (6, 70000)):
        z, y = make(T, V, torch.float32, g)
        y[:] = 5
        y[2] = V
        y[4] = 2 ** 31 - 1
        logp, lse = sk.token_logprobs(z, y)
        assert logp[[2, 4]].isnan().all() and logp[[0, 1, 3, 5]].isfinite().all()
        d = sk.token_logprobs_backward(z, y, torch.ones(T, device="cuda"))
        assert d[[2, 4]].isnan().all() and d[[0, 1, 3, 5]].isfinite().all()
        off = torch.tensor([0, 2, 4, 6]).cuda()
        loss, _, _, d = sk.policy_loss(z, y, off, logp.nan_to_num(), torch.ones(T, device="cuda"))
        assert loss[0].isfinite() and loss[1:].isnan().all() and d[[2, 4]].isnan().all()
        assert d[[0, 1, 3, 5]].isfinite().all()
        idx = torch.zeros(T, 3, dtype=torch.int32, device="cuda")
        idx[1, 2], idx[3, 0] = V, 2 ** 31 - 1
        loss, d = sk.distill_loss(z, idx, torch.zeros(T, 3, device="cuda"))
        assert loss[[1, 3]].isnan().all() and d[[1, 3]].isnan().all()
        assert loss[[0, 2]].isfinite().all() and d[[0, 2]].isfinite().all()
    z = torch.randn(8, 10, generator=g).cuda()
    idx = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    idx[6, 1] = 10
    loss, _, counts, d = sk.balance_loss(z, idx, torch.tensor([0, 4, 8]).cuda())
    assert loss[0].isfinite() and loss[1].isnan()
    assert counts.cpu().tolist() == [[8] + [0] * 9, [7] + [0] * 9]
    assert d[:4].isfinite().all() and d[4:].isnan().all()


def test_offsets_out_of_order_stay_in_bounds():
    # not a call the documentation allows; nothing may be read or written out of range
    g = rng(4)
    z, y = make(40, 200, torch.float32, g)
    x = torch.zeros(40, device="cuda")
    for off in ([0, 30, 10, 40, 5], [-7, 3, 900, 2 ** 40, 10], [40, 30, 20, 10, 0]):
        o = torch.tensor(off).cuda()
        sk.policy_loss(z, y, o, x, x)
        sk.preference_loss(z, y, o)
        sk.balance_loss(z, y.abs()[:, None], o)
    torch.cuda.synchronize()


def test_masked_label_takes_the_formula():
    # probability 0: log-probability -inf, ratio 0, infinite KL where there is a reference
    g = rng(6)
    z, y = make(6, 500, torch.float32, g)
    y[:] = 3
    z[2, 3] = -math.inf
    logp, lse = sk.token_logprobs(z, y)
    assert logp[2] == -math.inf and lse.isfinite().all()
    F.check(sk.token_logprobs_backward(z, y, torch.ones(6).cuda()),
            F.Rows(z).label_grad(y, torch.ones(6).double(), torch.full((6,), 4e-6).double()), "grad")
    off = torch.tensor([0, 6]).cuda()
    old = logp.clamp(min=-20)
    loss, kl, _, d = sk.policy_loss(z, y, off, old, torch.ones(6).cuda())
    F.check(loss, F.policy(z, y, off, old, torch.ones(6))[0], "loss")
    assert (d[2] == 0).all() and kl == 0
    assert sk.policy_loss(z, y, off, old, torch.ones(6).cuda(), ref=old, kl=0.1)[1] == math.inf
    # with coefficient 0 the infinite KL is reported and enters nothing
    loss0, kl0, _, d0 = sk.policy_loss(z, y, off, old, torch.ones(6).cuda(), ref=old, kl=0.0)
    assert kl0 == math.inf and torch.equal(loss0, loss) and torch.equal(d0, d)
    # an impossible token: of the other sequence, the loss is 0 and nothing is left to learn; of the
    # preferred one, it is infinite
    pair = torch.tensor([0, 2, 4]).cuda()
    loss, reward, _, d = sk.preference_loss(z, y, pair)
    assert loss == 0 and reward[1] == -math.inf and (d == 0).all()
    loss, reward, _, d = sk.preference_loss(z, y, torch.tensor([1, 4, 6]).cuda())
    assert loss == math.inf and reward[0] == -math.inf and d.isfinite().all()
    # distillation towards it: infinite loss, finite gradient
    idx = torch.tensor([[3, 4]] * 6, dtype=torch.int32).cuda()
    u = torch.zeros(6, 2).cuda()
    loss, d = sk.distill_loss(z, idx, u)
    assert loss[2] == math.inf and d.isfinite().all() and d[2, 3].item() == -0.5
    u[1, 0], u[4, 1] = math.inf, math.nan
    loss, d = sk.distill_loss(z, idx, u)
    assert loss[[1, 4]].isnan().all() and d[[1, 4]].isnan().all() and d[[0, 2, 3, 5]].isfinite().all()


def test_ratio_at_a_border_is_not_clipped():
    # two equal logits: logp = log(1/2) and old = log(1/2) - log(1 + clip) are not exact in fp32,
    # clip = 0 with old = logp's own fp64 value is: r is 1 to within the last bits on either side
    z = torch.zeros(2, 2).cuda()
    y = torch.zeros(2, dtype=torch.int32).cuda()
    off = torch.tensor([0, 2]).cuda()
    old = torch.full((2,), -math.inf).cuda()         # ratio +inf
    _, _, _, d = sk.policy_loss(z, y, off, old, torch.tensor([1.0, 1.0]).cuda())
    assert (d == 0).all()                            # clipped from above
    _, _, _, d = sk.policy_loss(z, y, off, torch.zeros(2).cuda(), torch.tensor([1.0, -1.0]).cuda(),
                                clip=(0.5, 0.0), mean=False)
    # r = 1/2 is the lower border exactly for the second row: kept, gradient -r A (1 - q)
    assert d[0, 0].item() == -0.25 and d[1, 0].item() == 0.25


@pytest.mark.parametrize("dt", TYPES)
def test_against_differences(dt):
    """Directional derivatives of the kernels' own losses.  With h = 2^-6 and |direction| <= 1 the
    third derivative of each is below 16 times the sum of the weights (cumulants of a bounded
    variable), so the truncation is below h^2 * 16 / 6 = 7e-4 a unit of weight; the losses' own
    errors, eps_S a row, enter divided by h: 3e-4.  bf16 logits move by their own roundings, so
    there the direction is what the logits really moved by."""
    g = rng(8)
    T, V = 24, 700
    z, y = make(T, V, TYPES[dt], g)
    y[:] = y.clamp(min=0)
    off = torch.tensor([0, 6, 12, 18, 24]).cuda()
    lp = F.Rows(z).logp(y)[0]
    old = (lp + 0.05).float().cuda()
    idx = torch.randint(0, V, (T, 6), generator=g).int().cuda()
    u = torch.randn(T, 6, generator=g).cuda()
    runs = {
        "policy": lambda x: sk.policy_loss(x, y, off, old, torch.ones(T).cuda(), ref=old, kl=0.1),
        "preference": lambda x: sk.preference_loss(x, y, off, old, mean=True),
        "distill": lambda x: sk.distill_loss(x, idx, u),
    }
    h = 2.0 ** -6
    up = (z.float() + h * (2 * torch.rand(T, V, generator=g) - 1).cuda()).to(z.dtype)
    down = (2 * z.float() - up.float()).to(z.dtype)
    move = (up.double() - down.double())
    mid = ((up.double() + down.double()) / 2)
    assert (mid - z.double()).abs().max() <= 2.0 ** -8 * z.float().abs().max()
    weight = {"policy": 4.0, "preference": 2.0, "distill": 24.0}
    for name, run in runs.items():
        diff = (run(up)[0].double() - run(down)[0].double()).sum().item()
        along = (run(z)[-1].double() * move).sum().item()
        size = move.abs().max().item() / 2
        # bf16: the gradient's own rounding, 2^-8 of sum |g| |move|, and the middle point's offset
        slack = weight[name] * (size ** 3 * 16 / 3 + 2 * F.eps_sum(V) * 4 + 1e-6)
        if dt == "bf16":
            slack += 2.0 ** -8 * (run(z)[-1].double() * move).abs().sum().item()
            slack += weight[name] * 4 * (mid - z.double()).abs().max().item() * size
        assert abs(diff - along) <= slack, (name, diff, along, slack)


def test_a_training_step_of_them_together():
    """Scored by two models, a policy step, a preference step and a distillation step on the same
    logits, with the router's balance loss beside them: the pieces fit each other."""
    g = rng(10)
    T, V, E = 48, 1200, 16
    z, y = make(T, V, torch.bfloat16, g)
    ref_z = (z.float() + 0.3 * torch.randn(T, V, generator=g).cuda()).bfloat16()
    off = torch.tensor([0, 10, 22, 30, 44]).cuda()
    old, lse = sk.token_logprobs(z, y)
    ref, _ = sk.token_logprobs(ref_z, y)
    adv = torch.randn(4, generator=g).cuda()
    loss, kl, logp, d = sk.policy_loss(z, y, off, old, adv, ref=ref, kl=0.05)
    want = F.policy(z, y, off, old, adv, ref=ref, kl=0.05)
    rows = want[2][0][:44], want[2][1][:44]
    F.check(logp[:44], rows, "logp")
    F.check(old[:44], rows, "old")
    F.check(loss, want[0], "policy")
    # on the behaviour policy itself every ratio is 1: without the KL term the gradient is that of -A logp / n
    share = torch.zeros(T, device="cuda")
    for i, (a, b) in enumerate(F.ranges(off, T)):
        share[a:b] = adv[i] / (y[a:b] >= 0).sum().clamp(min=1)
    plain = sk.token_logprobs_backward(z, y, -share)
    nokl = sk.policy_loss(z, y, off, old, adv)[3]
    assert (plain[:44].float() - nokl[:44].float()).abs().max() <= \
        2.0 ** -7 * nokl.float().abs().max()         # two roundings to bf16
    ploss, reward, plogp, pd = sk.preference_loss(z, y, off, ref, beta=0.2)
    F.check(ploss, F.preference(z, y, off, ref, beta=0.2)[0], "preference")
    F.check(plogp[:44], rows, "logp of the pairs")
    top = ref_z.float().topk(8, dim=1)
    tl = torch.logsumexp(ref_z.float(), 1)
    dl, dd = sk.distill_loss(z, top.indices.int(), top.values.contiguous(), teacher_lse=tl)
    F.check(dl, F.distill(z, top.indices.int(), top.values, teacher_lse=tl)[0], "distill")
    router = torch.randn(T, E, generator=g).cuda()
    idx = router.topk(2, dim=1).indices.int()
    bl, zl, counts, bd = sk.balance_loss(router, idx, off, balance=0.01, z=0.001)
    assert counts.sum().item() == 88 and bl.isfinite().all()
    total = loss.sum() + ploss.sum() + dl.sum() + 0.01 * bl.sum() + 0.001 * zl.sum()
    assert total.isfinite() and all(x.float().isfinite().all() for x in (d, pd, dd, bd))


def test_long_rows_pass_32_bits():
    """Row starts beyond 2^31 elements: the last rows of a tall matrix equal the same rows alone."""
    T, V = 36000, 65536
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 20 GB")
    z = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(4, V, generator=rng(11)).bfloat16().cuda()
    z[-4:] = tail
    y = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    y[-4:] = torch.tensor([0, 1, V - 1, 77], dtype=torch.int32)
    logp, lse = sk.token_logprobs(z, y)
    want = sk.token_logprobs(tail, y[-4:])
    tol = 2 * F.eps_sum(V)
    assert (logp[-4:] - want[0]).abs().max() <= tol and (lse[-4:] - want[1]).abs().max() <= tol
    grad = torch.ones(T, device="cuda")
    d = sk.token_logprobs_backward(z, y, grad, out=z)
    ref, t = F.Rows(tail).label_grad(y[-4:], torch.ones(4).double(), torch.full((4,), 4 * tol).double())
    F.check(d[-4:], (ref, t), "dlogits")
    assert (d[:-4].view(torch.int16) == 0).all()


@pytest.mark.parametrize("T,V", [((1 << 20) * 3 + 7, 3), (2, 1 << 24)])
def test_many_rows_and_the_longest(T, V):
    # more work-groups than one dimension of a launch is given, and the largest row
    g = rng(31)
    z = torch.randn(T, V, generator=g)
    y = torch.randint(-1, V, (T,), generator=g).int()
    y[-1] = V - 1
    zd, yd = z.cuda(), y.cuda()
    R = F.Rows(z)
    logp, _ = sk.token_logprobs(zd, yd)
    F.check(logp, R.logp(y), "logp")
    w = torch.randn(T, generator=g)
    d = sk.token_logprobs_backward(zd, yd, w.cuda())
    F.check(d, R.label_grad(y, w.double(), torch.zeros(T).double()), "dlogits")
    idx = torch.randint(0, V, (T, 2), generator=g).int()
    u = torch.randn(T, 2, generator=g)
    loss, dd = sk.distill_loss(zd, idx.cuda(), u.cuda())
    rows = torch.tensor([0, 1, T // 2, T - 1])
    want = F.distill(z[rows], idx[rows], u[rows])
    F.check(loss[rows.cuda()], want[0], "loss")
    F.check(dd[rows.cuda()], want[1], "distill")


def test_many_routed_rows():
    g = rng(32)
    T, E, K = (1 << 21) + 3, 4, 2
    z = torch.randn(T, E, generator=g)
    idx = z.topk(K, dim=1).indices.int()
    off = torch.tensor([0, 5, T // 3, T // 3, T])
    loss, zloss, counts, d = sk.balance_loss(z.cuda(), idx.cuda(), off.cuda(), balance=2.0, z=0.5)
    q, lse = torch.softmax(z.double(), 1), torch.logsumexp(z.double(), 1)
    for i, (a, b) in enumerate(F.ranges(off, T)):
        n = b - a
        hot = torch.bincount(idx[a:b].reshape(-1).long(), minlength=E)
        assert torch.equal(counts[i].cpu().long(), hot)
        if not n:
            assert loss[i] == 0 and zloss[i] == 0
            continue
        f = hot.double() * E / (K * n)
        dot = (q[a:b] * f).sum(1)
        # per row: the softmax's eps_S, f's rounding; the sum over rows is fp64
        assert abs(loss[i].item() - dot.mean().item()) <= (F.eps_sum(E) + 8 * F.U) * f.max().item()
        want = q[a:b] * (2.0 * (f - dot[:, None]) + lse[a:b, None]) / n
        size = (2 * (f.max() + dot[:, None]) + lse[a:b, None].abs()) * q[a:b] / n
        assert ((d[a:b].cpu().double() - want).abs() <= 2 * (F.eps_sum(E) + 16 * F.U) * size).all()
        assert abs(zloss[i].item() - (lse[a:b] ** 2).mean().item()) <= \
            (2 * F.eps_sum(E) + 8 * F.U) * ((lse[a:b].abs() + 1) ** 2).mean().item()


@pytest.mark.parametrize("T,V,n", [(2500, 70, 5), (90, 300, 130), (3001, 33, 2), (2049, 257, 64),
                                   (2048, 130, 64), (700, 9, 65)])
@pytest.mark.parametrize("mean", [True, False])
def test_many_sequences_and_long_ones(T, V, n, mean):
    """More sequences than lanes and more rows than a row's own work-group looks through, and
    the last sizes that it does."""
    g = rng(T + V + n)
    z, y = make(T, V, torch.float32, g)
    off = cut(T, n, g, first=3, last=T - 7)
    lp = F.Rows(z).logp(y)[0]
    old = (lp + 0.25 * torch.randn(T, generator=g).double()).float().cuda()
    ref = (lp + 0.3 * torch.randn(T, generator=g).double()).float().cuda()
    w = torch.rand(n, generator=g).cuda()
    adv = torch.randn(n, generator=g).cuda()
    inside = (torch.arange(T) >= 3) & (torch.arange(T) < T - 7)
    kw = dict(ref=ref, kl=0.1, weights=w, mean=mean)
    got, want = sk.policy_loss(z, y, off, old, adv, **kw), F.policy(z, y, off, old, adv, **kw)
    assert want[4][torch.isfinite(want[4])].min() > 1e-6
    F.check(got[2], (torch.where(inside, want[2][0], 0.0), want[2][1]), "logp")
    for k, name in ((0, "loss"), (1, "kl"), (3, "dlogits")):
        F.check(got[k], want[k], name)
    none = sk.policy_loss(z, y, off, old, adv, grad=False, **kw)
    assert none[3] is None and all(torch.equal(a, b) for a, b in zip(none[:3], got[:3]))
    if n % 2:
        off = off[:-1]
        n -= 1
    inside = (torch.arange(T) >= 3) & (torch.arange(T) < int(off[-1]))
    kw = dict(beta=0.2, smoothing=0.05, weights=w[:n // 2], mean=mean)
    got, want = sk.preference_loss(z, y, off, ref, **kw), F.preference(z, y, off, ref, **kw)
    F.check(got[2], (torch.where(inside, want[2][0], 0.0), want[2][1]), "logp of pairs")
    for k, name in ((0, "loss"), (1, "reward"), (3, "dlogits")):
        F.check(got[k], want[k], name)
    none = sk.preference_loss(z, y, off, ref, grad=False, **kw)
    assert none[3] is None and all(torch.equal(a, b) for a, b in zip(none[:3], got[:3]))
    over = z.clone()
    again = sk.preference_loss(over, y, off, ref, out=(*[o.clone() for o in got[:3]], over), **kw)
    assert torch.equal(again[3][inside.cuda()], got[3][inside.cuda()])
    assert torch.equal(over[~inside.cuda()], z[~inside.cuda()])
    over = z.clone()
    off2 = cut(T, n, g)
    new = sk.policy_loss(z, y, off2, old, adv[:n], mean=mean)
    sk.policy_loss(over, y, off2, old, adv[:n], mean=mean, out=(*[o.clone() for o in new[:3]], over))
    assert torch.equal(over, new[3])


def test_a_ratio_beyond_fp32():
    """e^200 is an ordinary number in 64 bits: times an advantage of 0 it is 0, times a small one
    a number.  The log-probability is off by eps_S, the exponential and two roundings by 2^-23."""
    g = rng(61)
    T, V = 6, 900
    z, y = make(T, V, torch.float32, g)
    y = y.abs() % V
    off = torch.tensor([0, 2, 4, 6]).cuda()
    lp = F.Rows(z).logp(y)[0]
    old = (lp - torch.tensor([200.0, 200.0, 120.0, 120.0, -200.0, -200.0])).float().cuda()
    adv = torch.tensor([0.0, -1e-30, 0.0]).cuda()
    loss, kl, logp, d = sk.policy_loss(z, y, off, old, adv)
    r = torch.exp(lp - old.cpu().double())
    want = (r[2] + r[3]) / 2 * float(torch.tensor(1e-30).double())
    assert loss[0] == 0 and loss[2] == 0 and kl.abs().sum() == 0
    assert abs(float(loss[1]) / float(want) - 1) < F.eps_sum(V) + 4 * F.U * 2 + F.U * 40
    assert torch.equal(d[:2], torch.zeros_like(d[:2])) and torch.equal(d[4:], torch.zeros_like(d[4:]))
    assert torch.isfinite(d).all() and d[2].abs().max() > 0


@pytest.mark.parametrize("T,K", [(3, 7), (5, 300)])
@pytest.mark.parametrize("V", [900, 70001])
def test_lists_padded_with_a_token(T, K, V):
    """Padding by a token that the list may hold, its logits -inf, changes nothing but roundings."""
    g = rng(T + K + V)
    z, _ = make(T, V, torch.float32, g)
    idx = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)]).int()
    u = 3 * torch.randn(T, K, generator=g)
    u[:, K // 2:] = -math.inf
    idx[:, K // 2:] = 5
    idx[0, 0] = 5
    loss, d = sk.distill_loss(z, idx.cuda(), u.cuda(), temperature=1.5)
    (want, tol), grad = F.distill(z, idx, u, temperature=1.5)
    F.check(loss, (want, tol), "loss")
    F.check(d, grad, "dlogits")
    cut_off = sk.distill_loss(z, idx[:, :K // 2].cuda(), u[:, :K // 2].cuda(), temperature=1.5)
    F.check(cut_off[0], (want, tol), "loss of the list without padding")
    F.check(cut_off[1], grad, "dlogits of the list without padding")


@pytest.mark.parametrize("T,E", [(40, 8), (3000, 40)])
def test_rows_sent_to_no_expert_there_is(T, E):
    """A row whose one index lies beyond E has an index: it counts in n, and its group has no
    balance loss."""
    g = rng(T + E)
    z, _ = make(T, E, torch.float32, g)
    idx = torch.randint(0, E, (T, 1), generator=g).int()
    half = T // 2
    idx[half:] = E
    off = torch.tensor([0, half, T]).cuda()
    loss, zloss, counts, d = sk.balance_loss(z, idx.cuda(), off, balance=0.3, z=0.02)
    want = F.balance(z, idx, off.cpu(), balance=0.3, z=0.02)
    assert torch.isnan(loss[1]) and torch.isnan(d[half:]).all() and counts[1].sum() == 0
    for k, name in ((0, "loss"), (1, "zloss")):
        F.check((loss, zloss)[k][:1], (want[k][0][:1], want[k][1][:1]), name)
    F.check(d[:half], (want[3][0][:half], want[3][1][:half]), "dlogits")
    whole = F.balance(z, idx.clamp(max=E - 1), off.cpu(), balance=0.3, z=0.02)
    F.check(zloss, whole[1], "zloss of both")


@pytest.mark.parametrize("T,G", [(300007, 1 << 20), (70001, 4097), (20000, 65), (66000, 64)])
def test_many_groups_of_routed_rows(T, G):
    """Most of 2^20 groups empty, groups of one row and long ones: each group's counts, losses and
    gradients against sums over rows in 64 bits."""
    g = rng(T + G)
    E, K = 8, 2
    z = torch.randn(T, E, generator=g)
    idx = z.topk(K, dim=1).indices.int()
    idx[::7] = -1
    cuts = torch.randint(3, T - 5, (G - 1,), generator=g).sort().values
    cuts[:G // 3] = cuts[G // 3]     # the rows before it are one group
    off = torch.cat([torch.tensor([3]), cuts, torch.tensor([T - 5])])
    loss, zloss, counts, d = sk.balance_loss(z.cuda(), idx.cuda(), off.cuda(), balance=0.3, z=0.02)
    seg = torch.bucketize(torch.arange(T), off[1:], right=True).clamp(max=G - 1)
    inside = (torch.arange(T) >= 3) & (torch.arange(T) < T - 5)
    used = inside & (idx[:, 0] >= 0)
    n = torch.zeros(G, dtype=torch.float64).index_add_(0, seg, used.double())
    hot = torch.zeros(T, E, dtype=torch.float64).scatter_(1, idx.long().clamp(min=0), 1.0)
    hot = torch.where(used[:, None], hot, 0.0)
    want = torch.zeros(G, E, dtype=torch.float64).index_add_(0, seg, hot)
    assert torch.equal(counts.cpu(), want.int())
    R = F.Rows(z)
    over = 1.0 / n.clamp(min=1)
    f = (want * (E / K) * over[:, None])[seg]
    dot = (f * R.q).sum(1)
    sums = lambda v: torch.zeros(G, dtype=torch.float64).index_add_(  # noqa: E731
        0, seg, torch.where(used, v, 0.0)) * over
    # as in F.balance: each f - 1 rounded once, p off by q_tol, the row sums by eps_S
    e = F.eps_sum(E)
    size = (R.q * (f - 1).abs()).sum(1)
    off_by = size * (e + 24 * F.U) + E * F.U * size + (R.q_tol * (f - 1).abs()).sum(1)
    F.check(loss, (sums(dot), sums(off_by) + 4 * F.U * sums(dot)), "loss")
    lt = e + 4 * F.U * (R.lse.abs() + R.M.abs())
    F.check(zloss, (sums(R.lse ** 2), sums(2 * R.lse.abs() * lt + lt * lt)
                    + 4 * F.U * sums(R.lse ** 2)), "zloss")
    inner = 0.3 * (f - dot[:, None]) + 0.04 * R.lse[:, None]
    it = 0.3 * (off_by[:, None] + 6 * F.U * ((f - 1).abs() + size[:, None])) \
        + 0.04 * (lt + 4 * F.U * R.lse.abs())[:, None]
    k = torch.where(used, over[seg], 0.0)[:, None]
    grad = R.q * inner * k
    tol = (R.q * it + (R.q_tol + 6 * F.U * R.q) * (inner.abs() + it)) * k
    F.check(d, (grad, tol + F.U * (grad.abs() + tol) * 1.01 + 1e-38), "dlogits")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V", [(256, 9001), (257, 9001), (258, 17011), (259, 30011), (260, 60013)])
def test_distill_of_more_rows_than_compute_units(T, V, dt):
    """Up to 256 rows take more registers each than longer batches do."""
    test_distill_loss(T, V, dt)
