"""The losses over logits at the edges of their ranges: large KL gaps, coefficients beyond fp32,
weights of 0, sums that cancel, and the calls around them.

Most rows here are `even` ones: the label and one more token have the logit 0 and all others are
masked or far below, so that the sum of a row is 2 without any rounding and the log-probability
-ln 2 to 2^-44.  What is left of an error is then the function under test and the last roundings."""
import math

import pytest
import torch

import losses_formulas as F
import sinkhorn_point_cloud_amd as sk

pytestmark = pytest.mark.gpu
U = F.U
# rows that a wave, a work-group and several hold
WIDTHS = [900, 20001, 70001]


@pytest.fixture(autouse=True)
def _say(request):
    print(request.node.name, flush=True)
    yield


def even(T, V, dtype=torch.float32):
    """(logits [T, V], labels [T]) on the GPU; the label 3, its equal V - 2, one token 40 below at
    column 5, nothing else."""
    z = torch.full((T, V), -math.inf, dtype=dtype)
    z[:, 3] = z[:, V - 2] = 0.0
    z[:, 5] = -40.0
    return z.cuda(), torch.full((T,), 3, dtype=torch.int32).cuda()


def near(got, want, rel, what):
    """Equal where the fp32 value of `want` is 0 or infinite, else within rel of it."""
    want = want.double()
    w32 = want.float()
    got = got.cpu()
    plain = w32.isfinite() & (w32 != 0)
    assert torch.equal(got.float()[~plain], w32[~plain]), (what, got[~plain], w32[~plain])
    off = (got.double() - want)[plain].abs() / want[plain].abs()
    assert off.numel() == 0 or off.max() <= rel, (what, off.max().item() / U, "units of 2^-24")


GAPS = [-1000.0, -30.3, -5.7, -1.1, -0.01, 0.3, 5.3, 20.7, 90.1]


@pytest.mark.parametrize("n", [9, 1])
@pytest.mark.parametrize("V", WIDTHS)
def test_kl_far_from_the_reference(V, n):
    """k = e^d - d - 1 and its slope 1 - e^d for d = ref - logp from -1000 to 90, where e^d lies
    beyond fp32 and the weighted loss does not.  kl, loss: the function within half a unit, a
    term and the output rounded, 3 units.  The gradient: slope, exponential at the label (|logp| <
    1: a series of 11 terms, the last few roundings) and the product, 8 units; 40 below the
    maximum, an exponent of 58 rounded three times, 3 * 58 ln 2 units more."""
    T = len(GAPS)
    z, y = even(T, V)
    lp = torch.full((T,), -math.log(2.0), dtype=torch.float64)
    ref = (lp + torch.tensor(GAPS, dtype=torch.float64)).float()
    gap = ref.double() - lp
    w, coef = 2.0 ** -10, 0.01
    kw = dict(ref=ref.cuda(), kl=coef, mean=False)
    k = torch.exp(gap) - gap - 1
    k[4] = gap[4] ** 2 / 2 * (1 + gap[4] / 3 * (1 + gap[4] / 4 * (1 + gap[4] / 5)))
    slope = -coef * w * torch.expm1(gap)
    if n == 1:      # one sequence of all rows
        off, weights = torch.tensor([0, T]), torch.tensor([w])
    else:
        off, weights = torch.arange(T + 1), torch.full((T,), w)
    adv = torch.zeros(T).cuda()
    loss, kl, logp, d = sk.policy_loss(z, y, off.cuda(), lp.float().cuda(), adv,
                                       weights=weights.cuda(), **kw)
    total = (lambda x: x.sum()[None]) if n == 1 else (lambda x: x)
    near(kl, total(w * k), 3 * U, "kl")
    near(loss, total(coef * w * k), 3 * U, "loss")
    want = torch.zeros(T, V, dtype=torch.float64)
    want[:, 3], want[:, V - 2] = slope / 2, -slope / 2
    far = -slope * math.exp(-40) / 2
    near(d[:, 5], far, (8 + 3 * 58 * math.log(2)) * U, "gradient of the far token")
    d[:, 5] = 0
    near(d, want, 8 * U, "gradient")


@pytest.mark.parametrize("V", WIDTHS)
def test_a_label_that_the_reference_forbids(V):
    """ref = -inf: e^d is 0, the term infinite and its slope that of -d, 1 (8 units as above)."""
    z, y = even(3, V)
    old = torch.full((3,), -math.log(2.0)).cuda()
    ref = old.clone()
    ref[1] = -math.inf
    loss, kl, _, d = sk.policy_loss(z, y, torch.arange(4).cuda(), old, torch.zeros(3).cuda(),
                                    ref=ref, kl=0.25)
    assert kl[1] == math.inf and loss[1] == math.inf and loss[[0, 2]].isfinite().all()
    assert d.isfinite().all()
    near(d[1, [3, V - 2]], torch.tensor([0.125, -0.125], dtype=torch.float64), 8 * U, "gradient")


@pytest.mark.parametrize("V", WIDTHS)
def test_coefficients_beyond_fp32(V):
    """A row's coefficient (here up to 1.2e39) is no output: where it meets a probability of 0 the
    gradient is 0, and 40 below the maximum an ordinary number.  Tolerances as for the KL gaps."""
    far_rel = (8 + 3 * 58 * math.log(2)) * U
    far = math.exp(-40) / 2

    def check(d, G, what):
        """d = G (1[label] - q), or G (q - 1[label]) of -G, per row."""
        want = torch.zeros(d.shape, dtype=torch.float64)
        want[:, 3], want[:, V - 2] = G / 2, -G / 2
        near(d[:, 5], -G * far, far_rel, what + " far")
        d = d.clone()
        d[:, 5] = 0
        near(d, want, 8 * U, what)

    z, y = even(2, V)
    G = torch.tensor([3e38, -2.5e38])
    check(sk.token_logprobs_backward(z, y, G.cuda(), scale=1.0), G.double(), "backward")
    half = z / 2        # twice the gradient, half the logits: the same softmax
    check(sk.token_logprobs_backward(half, y, G.cuda(), scale=2.0), 2 * G.double(), "scaled")
    old = torch.full((2,), -math.log(2.0)).cuda()
    ref = (old.double() + 90.1).float()
    d = sk.policy_loss(z, y, torch.arange(3).cuda(), old, torch.zeros(2).cuda(), ref=ref, kl=1.0)[3]
    gap = ref.cpu().double() + math.log(2.0)
    check(d, -torch.expm1(gap), "KL")
    # temperature 2 over twice the logits: w tau (q - 1[token])
    w = G.abs().cuda()
    d = sk.distill_loss(z * 2, y[:, None], torch.zeros(2, 1).cuda(), temperature=2.0, weights=w)[1]
    check(d, -2 * w.cpu().double(), "distillation")


@pytest.mark.parametrize("n", [4, 80])
@pytest.mark.parametrize("V", WIDTHS)
@pytest.mark.parametrize("mean", [True, False])
def test_a_weight_of_zero_takes_a_sequence_out(V, n, mean):
    """Sequences weighted out because they hold NaN, an impossible label or an infinite KL: their
    losses and gradients are 0, their log-probabilities and rewards are reported, and the others are
    as if alone, to the bit."""
    g = torch.Generator().manual_seed(V + n)
    T = 2 * n
    z = torch.randn(T, V, generator=g)
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    clean = z.clone()
    z[2, 7] = math.nan
    z[3, y[3]] = -math.inf
    z, y, clean = z.cuda(), y.cuda(), clean.cuda()
    off = torch.arange(0, T + 1, 2).cuda()
    w = torch.ones(n)
    w[1] = 0.0
    out = torch.ones(T, dtype=torch.bool)
    out[2:4] = False
    old = sk.token_logprobs(clean, y)[0]
    ref = old + 0.1
    args = (y, off, old, torch.ones(n).cuda())
    kw = dict(ref=ref, kl=0.1, weights=w.cuda(), mean=mean)
    loss, kl, logp, d = sk.policy_loss(z, *args, **kw)
    want = sk.policy_loss(clean, *args, **kw)
    assert loss[1] == 0 and kl[1] == 0 and (d[2:4] == 0).all()
    assert logp[2].isnan() and logp[3] == -math.inf
    for a, b in ((loss, want[0]), (kl, want[1])):
        assert torch.equal(a[w.bool().cuda()], b[w.bool().cuda()])
    for a, b in ((logp, want[2]), (d, want[3])):
        assert torch.equal(a[out.cuda()], b[out.cuda()])
    pw = w[:n // 2].clone()
    pw[:2] = torch.tensor([0.0, 1.0])
    for kind in ("sigmoid", "square"):
        kw = dict(weights=pw.cuda(), mean=mean, kind=kind)
        loss, reward, logp, d = sk.preference_loss(z, y, off, old, **kw)
        want = sk.preference_loss(clean, y, off, old, **kw)
        assert loss[0] == 0 and (d[:4] == 0).all() and reward[1].isnan()
        assert logp[2].isnan() and logp[3] == -math.inf
        assert torch.equal(loss, want[0]) and torch.equal(reward[2:], want[1][2:])
        assert torch.equal(reward[0], want[1][0]) and torch.equal(d, want[3])
        assert torch.equal(logp[out.cuda()], want[2][out.cuda()])


def test_no_gradient_into_a_buffer_that_is_not_asked_for():
    g = torch.Generator().manual_seed(1)
    T, V = 6, 300
    z = torch.randn(T, V, generator=g).cuda()
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    off = torch.tensor([0, 2, 6]).cuda()
    x = torch.randn(T, generator=g).cuda()
    new = lambda *s, dtype=torch.float32: torch.full(s, 7, dtype=dtype, device="cuda")  # noqa: E731
    d = new(T, V)
    calls = [(sk.policy_loss, (z, y, off, x, x), (new(2), new(2), new(T))),
             (sk.preference_loss, (z, y, off), (new(1), new(2), new(T))),
             (sk.distill_loss, (z, y[:, None], x[:, None]), (new(T),)),
             (sk.balance_loss, (z, y[:, None], off),
              (new(2), new(2), new(2, V, dtype=torch.int32)))]
    for call, args, out in calls:
        want = call(*args)
        got = call(*args, out=(*out, d), grad=False)
        assert got[-1] is None and (d == 7).all(), call
        for a, b in zip(got[:-1], want[:-1]):
            assert torch.equal(a, b), call


@pytest.mark.parametrize("V,K", [(40, 1024), (1500, 1024), (30011, 700), (70001, 129)])
def test_lists_full_of_repeated_tokens(V, K):
    """Entries of one token dealt to all lanes in turn, among others without probability: every one
    of them is found, and each call finds the same."""
    g = torch.Generator().manual_seed(V + K)
    T = 9
    z = torch.randn(T, V, generator=g)
    few = torch.randint(0, V, (T, 7), generator=g)
    idx = few.gather(1, torch.randint(0, 7, (T, K), generator=g)).int()
    idx[1] = torch.randint(0, V, (K,), generator=g)
    idx[2, ::5] = -1
    u = torch.randn(T, K, generator=g)
    u[3, ::3] = -math.inf
    args = (z.cuda(), idx.cuda(), u.cuda())
    got, want = sk.distill_loss(*args), F.distill(*args)
    F.check(got[0], want[0], "loss")
    F.check(got[1], want[1], "dlogits")
    for _ in range(3):
        again = sk.distill_loss(*args)
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("T,n,V", [(24, 1, 900), (24, 1, 20001), (24, 1, 70001), (2400, 70, 900),
                                   (3001, 3, 4000)])
def test_a_policy_loss_of_terms_that_cancel(T, n, V):
    """Advantages of +1 and -1 over ratios that differ by 1e-6.  A ratio is off by 3e-10 of itself (its
    exponential) and the log-probability's 2^-44, weights, terms and sums are fp64, and the loss is
    rounded once."""
    g = torch.Generator().manual_seed(T + V)
    z, y = even(T, V)
    half = -1.5 + 1.7 * torch.rand(T // 2 + 1, generator=g)
    old = half.repeat_interleave(2)[:T] + torch.tensor([0.0, 1e-6]).repeat(T // 2 + 1)[:T]
    adv = torch.tensor([1.0, -1.0]).repeat(T // 2 + 1)[:T]
    off = torch.arange(n + 1) * T // n
    w = 0.1 + torch.rand(n, generator=g)
    kw = dict(clip=(0.99, math.inf), weights=w.cuda())
    loss = sk.policy_loss(z, y, off.cuda(), old.cuda(), adv.cuda(), **kw)[0]
    r = torch.exp(-math.log(2.0) - old.double())
    sums = lambda v: torch.stack([v[a:b].mean() for a, b in F.ranges(off, T)]) * w.double()  # noqa: E731
    want = sums(-r * adv.double())
    F.check(loss, (want, sums(r) * (3e-10 + 2.0 ** -40) + U * want.abs()), "loss")


@pytest.mark.parametrize("scale", [1.0, math.log(2.0) * (1 + 2.0 ** -24)])
@pytest.mark.parametrize("T,V,dt", [(1000, 32000, torch.float32), (1000, 32000, torch.bfloat16),
                                    (256, 131072, torch.bfloat16), (128, 70001, torch.float32)])
def test_log_probabilities_to_their_own_precision(T, V, dt, scale):
    """A pair's reward is logp - ref before it is rounded; with ref the fp32 value of logp it shows
    each row's error to 1e-13.  Logits of deviation 2: at scale 1 a row's sum is shared by about
    V e^-4 terms (580 at least) that lie 4.4 nats below its maximum in the mean.

    Roundings, root mean square, relative to the sum: a term's exponential (2^-23 / sqrt 3) and
    argument (two of half a unit at 6.3, 2^-22 / sqrt 3 ln 2 each) over the root of the number of
    terms, 6e-9; a thread's 32 to 128 additions (2^-24 / sqrt 3 each, half of that on the mean of a
    growing sum) over the root of 256 to 1024 threads, 6e-9; sums of 16 lanes, 4 additions each,
    over the root of 64, 6e-9.  Together 1.1e-8; the exponential's mean error, of one sign, is given
    1e-8 more.  So 2.1e-8 is allowed, for the mean error and the deviation alike.

    At the scale that makes c = s log2 e = 1 + 2^-24 the arguments are not rounded at random: d, an
    fp32 number of mantissa m in [1, 2), times c lies m / 2 of its unit beyond d and is always
    rounded outwards, by 1 - m / 2 units: 2^-24 (2 / m - 1) of itself.  The mean of that over the
    row's terms, each by its share of the sum, is of one sign and allowed too.

    One fp32 number for the scale would be off by more: 1.3e-8 of each argument at scale 1, 2^-24 at
    the other, with one sign.  The oracle with that mistake planted must be refused."""
    g = torch.Generator().manual_seed(T + V)
    z = (2 * torch.randn(T, V, generator=g)).to(dt)
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)

    def exact(s):
        x = z.double() - z.double().amax(1, keepdim=True)
        return scale * x.gather(1, y.long()[:, None])[:, 0] - torch.logsumexp(s * x, 1)

    lp = exact(scale)
    ref = lp.float()
    reward = sk.preference_loss(z.cuda(), y.cuda(), torch.arange(T + 1).cuda(), ref.cuda(), beta=1.0,
                                scale=scale, grad=False)[1]
    wrong = reward.cpu().double() - (lp - ref.double())
    allowed = 2.1e-8
    if scale != 1.0:
        x = z.double()
        d = x.amax(1, keepdim=True) - x
        m = 2 * torch.frexp(d).mantissa
        outwards = torch.where(d > 0, 2.0 ** -24 * (2 / m - 1) * d * scale, 0.0)
        allowed += (torch.softmax(x * scale, 1) * outwards).sum(1).mean().item()
    print("allowed", allowed, "mean", wrong.mean().item(), "rms", wrong.square().mean().sqrt().item())
    assert wrong.mean().abs() <= allowed and wrong.square().mean().sqrt() <= allowed
    one_piece = float(torch.tensor(scale / math.log(2.0)).float()) * math.log(2.0)
    planted = (exact(one_piece) - lp).mean().abs()
    assert planted > allowed and (scale != 1.0 or planted > 2 * allowed)


@pytest.mark.parametrize("T,V,n", [(40, 200, 4), (5000, 40, 130), (9000, 260, 300)])
def test_offsets_out_of_order_write_nothing_outside(T, V, n):
    """Not a call the documentation allows: outputs and workspace between guards, which stay."""
    g = torch.Generator().manual_seed(T)
    z = torch.randn(T, V, generator=g).cuda()
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    x = torch.zeros(T).cuda()
    pad = 4096
    kept = []

    def guarded(*shape, dtype=torch.float32):
        size = math.prod(shape)
        buf = torch.full((size + 2 * pad,), 77, dtype=dtype, device="cuda")
        kept.append((buf, size))
        return buf[pad:pad + size].view(shape)

    far = torch.randint(-T, 2 * T, (n + 1,), generator=g)
    far[1], far[-1] = 2 ** 40, -2 ** 62
    for off in (torch.randint(0, T + 1, (n + 1,), generator=g), far, torch.arange(n, -1, -1) * (T // n)):
        off = off.cuda()
        sizes = (sk.losses_workspace_bytes(1, T, V, 0, 0), sk.losses_workspace_bytes(2, T, V, 0, 0),
                 sk.losses_workspace_bytes(4, T, V, n, 0))
        ws = [guarded(s, dtype=torch.uint8) for s in sizes]
        sk.policy_loss(z, y, off, x, x, out=(guarded(n), guarded(n), guarded(T), guarded(T, V)),
                       workspace=ws[0])
        sk.preference_loss(z, y, off, workspace=ws[1],
                           out=(guarded(n // 2), guarded(n), guarded(T), guarded(T, V)))
        sk.balance_loss(z, y[:, None], off, workspace=ws[2],
                        out=(guarded(n), guarded(n), guarded(n, V, dtype=torch.int32), guarded(T, V)))
        torch.cuda.synchronize()
        for buf, size in kept:
            assert (buf[:pad] == 77).all() and (buf[pad + size:] == 77).all()
        kept.clear()


@pytest.mark.parametrize("T,E,K,G", [(40, 4, 2, 2), (500, 8, 2, 0), (3000, 8, 2, 3), (2000, 16, 2, 0),
                                     (1500, 64, 6, 2), (1100, 256, 8, 2)])
def test_balance_loss_within_its_own_additions(T, E, K, G, monkeypatch):
    """The formulas' bound of a row's sum counts 100 additions, for rows of any length.  A router's row
    is 16 lanes' of E / 16 values each, rounded up, and 4 additions between the lanes."""
    monkeypatch.setattr(F, "eps_sum", lambda V: U * (2 + 2.1 * math.log2(V) + -(-V // 16) + 4))
    g = torch.Generator().manual_seed(T + E)
    z = 2 * torch.randn(T, E, generator=g)
    idx = z.topk(K, dim=1).indices.int()
    off = torch.arange(G + 1) * T // G if G else None
    got = sk.balance_loss(z.cuda(), idx.cuda(), off.cuda() if G else None, balance=0.3, z=0.02)
    want = F.balance(z, idx, off, balance=0.3, z=0.02)
    assert torch.equal(got[2].cpu(), want[2])
    for k, name in ((0, "loss"), (1, "zloss"), (3, "dlogits")):
        F.check(got[k], want[k], name)
