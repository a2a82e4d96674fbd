"""The losses over logits, host side: their header, their refusals, and the formulas of the
tests against automatic differentiation and against differences."""
import ctypes
import math
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import sinkhorn_point_cloud_amd as sk

import losses_formulas as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sinkhorn_losses.h")
DUMMY = ctypes.c_void_p(4096)   # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return sk.load_library()


def test_header_library_and_binding_name_the_same_functions(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(sinkhorn_\w+)\s*\(", text))
    assert names == set(sk.LOSS_EXPORTS)
    out = os.popen(f"nm -D --defined-only {sk.library_path()}").read()
    for name in names:
        assert re.search(rf"\bT {name}$", out, flags=re.M), name
    for name in ("token_logprobs", "token_logprobs_backward", "policy_loss", "preference_loss",
                 "distill_loss", "balance_loss"):
        assert name in sk.__all__ and callable(getattr(sk, name))


def test_workspace_bytes(lib):
    ws = sk.losses_workspace_bytes
    for op, k in ((0, 0), (1, 0), (2, 0), (3, 16), (4, 3)):
        assert ws(op, 100, 64, k, 0) > 0
        assert ws(op, 0, 64, k, 1) > 0
        assert ws(op, -1, 64, k, 0) == 0 and ws(op, 100, 0, k, 0) == 0
        assert ws(op, 100, 64, k, 7) == 0 and ws(op, (1 << 24) + 1, 64, k, 0) == 0
    assert ws(5, 1, 1, 1, 0) == 0 and ws(-1, 1, 1, 1, 0) == 0
    assert ws(3, 10, 64, 0, 0) == 0 and ws(3, 10, 64, 1025, 0) == 0
    assert ws(4, 10, 1025, 1, 0) == 0 and ws(4, 10, 64, 0, 0) == 0
    # nothing of the size of the logits
    assert ws(1, 8192, 131072, 0, 1) < 1 << 20
    assert ws(3, 4096, 131072, 64, 1) < 4 << 20


def _call(lib, name, changes):
    """One entry point with arguments that are in order but for `changes`."""
    P = DUMMY
    base = dict(logits=P, dtype=0, ld=64, labels=P, T=10, V=64, scale=1.0, logp=P, lse=P, ws=P,
                ws_bytes=1 << 40, grad=P, dlogits=ctypes.c_void_p(1 << 30), dld=64, offsets=P, n=2,
                old=P, adv=P, ref=None, weights=None, lo=0.2, hi=0.2, kl=0.1, flags=0, loss=P,
                klo=P, kind=0, beta=0.1, eps=0.0, reward=P, index=P, teacher=P, K=4, tlse=None,
                tau=1.0, bal=1.0, z=0.0, zloss=P, counts=P, G=1)
    base.update(changes)
    a = lambda names: [base[n] for n in names.split()]  # noqa: E731
    order = {
        "token_logprobs": "logits dtype ld labels T V scale logp lse ws ws_bytes",
        "token_logprobs_backward": "logits dtype ld labels grad T V scale dlogits dld ws ws_bytes",
        "policy_loss": "logits dtype ld labels T V offsets n old adv ref weights scale lo hi kl "
                       "flags loss klo logp dlogits dld ws ws_bytes",
        "preference_loss": "logits dtype ld labels T V offsets n ref weights scale kind beta eps "
                           "flags loss reward logp dlogits dld ws ws_bytes",
        "distill_loss": "logits dtype ld T V index teacher K tlse weights tau loss dlogits dld ws "
                        "ws_bytes",
        "balance_loss": "logits dtype ld T V index K offsets G bal z flags loss zloss counts "
                        "dlogits dld ws ws_bytes",
    }[name]
    return getattr(lib, "sinkhorn_" + name)(*a(order), None)


ALL = ("token_logprobs", "token_logprobs_backward", "policy_loss", "preference_loss",
       "distill_loss", "balance_loss")
GRADS = ALL[1:]
SPACE = ALL


@pytest.mark.parametrize("name,changes,code", [
    *[(n, c, sk.SK_ERR_INVALID_ARG) for n in ALL for c in (
        dict(logits=None), dict(dtype=2), dict(T=-1), dict(T=(1 << 24) + 1), dict(V=0), dict(ld=63),
        dict(logits=ctypes.c_void_p(4098)))],
    *[(n, c, sk.SK_ERR_INVALID_ARG) for n in GRADS for c in (
        dict(dld=63), dict(dlogits=ctypes.c_void_p((1 << 30) + 2)),
        dict(dlogits=ctypes.c_void_p(4096 + 256)),            # inside the logits
        dict(dlogits=ctypes.c_void_p(4096), dld=65),          # their address, another distance
        dict(dlogits=ctypes.c_void_p(4096 + 4 * 32), ld=96, dld=96))],   # columns that overlap
    *[(n, c, sk.SK_ERR_WORKSPACE) for n in SPACE for c in (dict(ws=None), dict(ws_bytes=8))],
    *[(n, c, sk.SK_ERR_INVALID_ARG) for n in ALL[:4] for c in (
        dict(labels=None), dict(scale=0.0), dict(scale=1e-21), dict(scale=1e21), dict(scale=-1.0),
        dict(scale=math.nan), dict(scale=math.inf), dict(V=(1 << 24) + 1, ld=1 << 25))],
    ("token_logprobs", dict(logp=None, lse=None), sk.SK_ERR_INVALID_ARG),
    ("token_logprobs_backward", dict(grad=None), sk.SK_ERR_INVALID_ARG),
    ("token_logprobs_backward", dict(dlogits=None), sk.SK_ERR_INVALID_ARG),
    *[(n, c, sk.SK_ERR_INVALID_ARG) for n in ("policy_loss", "preference_loss") for c in (
        dict(offsets=None), dict(n=0), dict(n=(1 << 20) + 1), dict(loss=None), dict(flags=64))],
    *[("policy_loss", c, sk.SK_ERR_INVALID_ARG) for c in (
        dict(old=None), dict(adv=None), dict(klo=None), dict(lo=1.0), dict(lo=-0.1), dict(hi=-0.1),
        dict(hi=math.nan), dict(kl=math.inf))],
    *[("preference_loss", c, sk.SK_ERR_INVALID_ARG) for c in (
        dict(reward=None), dict(logp=None), dict(kind=2), dict(beta=0.0), dict(beta=math.inf),
        dict(eps=-0.1), dict(eps=1.1), dict(flags=4))],
    *[("distill_loss", c, sk.SK_ERR_INVALID_ARG) for c in (
        dict(index=None), dict(teacher=None), dict(loss=None), dict(K=0), dict(K=1025),
        dict(tau=0.0), dict(tau=-1.0), dict(tau=math.nan))],
    *[("balance_loss", c, sk.SK_ERR_INVALID_ARG) for c in (
        dict(index=None), dict(loss=None), dict(zloss=None), dict(counts=None), dict(K=0),
        dict(K=65), dict(G=0), dict(G=(1 << 20) + 1), dict(G=2, offsets=None), dict(V=1025, ld=1025, dld=1025),
        dict(flags=1), dict(bal=math.nan), dict(z=math.inf))],
])
def test_refusals(lib, name, changes, code):
    assert _call(lib, name, changes) == code, lib.sinkhorn_last_error()
    assert lib.sinkhorn_last_error()


def test_refusals_write_nothing(lib):
    loss = np.full(8, 3.0, dtype=np.float32)
    p = loss.ctypes.data_as(ctypes.c_void_p)
    for name in SPACE:
        assert _call(lib, name, dict(loss=p, logp=p, lse=p, ws_bytes=0)) == sk.SK_ERR_WORKSPACE
    assert np.all(loss == 3.0)


def test_no_rows_need_no_row_pointers(lib):
    none = dict(T=0, logits=None, labels=None, index=None, old=None, adv=None, teacher=None)
    for name in ("token_logprobs", "distill_loss"):
        assert _call(lib, name, none) == sk.SK_OK, lib.sinkhorn_last_error()
    assert _call(lib, "token_logprobs_backward", dict(none, grad=None)) == sk.SK_OK


@pytest.mark.parametrize("n", [2, 40])
def test_no_rows_with_a_gradient_buffer(n):
    """Any number of sequences without rows, a gradient buffer given: a launch on no device is an
    error (5), and the process lives."""
    program = f"""
import ctypes
import sinkhorn_point_cloud_amd as sk
lib, P = sk.load_library(), ctypes.c_void_p(4096)
F = [ctypes.c_void_p(4096 * (k + 2)) for k in range(4)]
tail = (ctypes.c_void_p(1 << 32), 1 << 40, None)
print(lib.sinkhorn_policy_loss(None, 0, 16, None, 0, 16, P, {n}, None, None, None, None, 1.0, 0.2,
                               0.2, 0.0, 0, F[0], F[1], None, F[2], 16, *tail),
      lib.sinkhorn_preference_loss(None, 0, 16, None, 0, 16, P, {n}, None, None, 1.0, 0, 0.1, 0.0, 0,
                                   F[0], F[1], None, F[2], 16, *tail),
      lib.sinkhorn_balance_loss(None, 0, 16, 0, 16, None, 2, P, {n}, 1.0, 0.0, 0, F[0], F[1], F[2],
                                F[3], 16, *tail))
"""
    run = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True,
                         env=dict(os.environ, HIP_VISIBLE_DEVICES="-1"))
    assert run.returncode == 0 and run.stdout.split() == ["5", "5", "5"], run


def test_binding_refusals():
    z = torch.zeros(4, 8)
    y = torch.zeros(4, dtype=torch.int32)
    off = torch.tensor([0, 4])
    calls = (lambda x: sk.token_logprobs(x, y), lambda x: sk.policy_loss(x, y, off, z[:, 0], z[:, 0]),
             lambda x: sk.preference_loss(x, y, off), lambda x: sk.balance_loss(x, y[:, None]),
             lambda x: sk.distill_loss(x, y[:, None], z[:, :1]),
             lambda x: sk.token_logprobs_backward(x, y, z[:, 0]))
    for call in calls:
        with pytest.raises(ValueError):
            call(z)                      # not on the GPU
        with pytest.raises(ValueError):
            call(z[0])                   # not a matrix
        with pytest.raises(TypeError):
            call(z.double())


def test_row_arrays_are_checked():
    dev = torch.device("cpu")
    ok = torch.zeros(4, dtype=torch.int32)
    assert sk.losses._row_array(ok, (4,), torch.int32, dev, "labels") is not None
    assert sk.losses._row_array(None, (4,), torch.int32, dev, "ref", optional=True) is None
    with pytest.raises(TypeError):
        sk.losses._row_array(ok.long(), (4,), torch.int32, dev, "labels")
    with pytest.raises(TypeError):
        sk.losses._row_array(None, (4,), torch.int32, dev, "labels")
    with pytest.raises(ValueError):
        sk.losses._row_array(ok, (5,), torch.int32, dev, "labels")
    z = torch.zeros(4, 8)
    for d in (torch.zeros(4, 9), torch.zeros(8, 4).t(), torch.zeros(4, 8).bfloat16(),
              torch.zeros(1, 8).expand(4, 8)):
        with pytest.raises(ValueError):
            sk.losses._check_gradient(d, z)
    assert sk.losses._check_gradient(torch.zeros(4, 12)[:, :8], z) == 12


# --- the formulas themselves

def _case(T=9, V=13, seed=0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, V, generator=g) * 2
    y = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    y[2] = -1
    return g, z, y


def _grad_of(f, z):
    """Gradient of the scalar f(z) by central differences in float64."""
    z = z.double()
    out = torch.zeros_like(z)
    h = 1e-5
    for i in range(z.shape[0]):
        for j in range(z.shape[1]):
            d = torch.zeros_like(z)
            d[i, j] = h
            out[i, j] = (f(z + d) - f(z - d)) / (2 * h)
    return out


# central differences at h = 1e-5 of a loss of size < 100: rounding 2^-53 * 100 / h = 1e-9, and
# h^2 / 6 times a third derivative below 100: 2e-9
DIFF = 1e-7


@pytest.mark.parametrize("mean", [False, True])
def test_policy_formula_against_differences(mean):
    g, z, y = _case()
    off = torch.tensor([0, 4, 4, 8])
    lp = F.Rows(z).logp(y)[0]
    old = (lp + 0.3 * torch.randn(9, generator=g).double()).float()
    ref = (lp + 0.2 * torch.randn(9, generator=g).double()).float()
    adv = torch.randn(9, generator=g)
    w = torch.tensor([1.0, 2.0, 0.5])
    kw = dict(ref=ref, clip=(0.2, 0.3), kl=0.1, weights=w, mean=mean)
    loss, kl, _, (grad, _), border = F.policy(z, y, off, old, adv, **kw)
    assert border.min() > 1e-3          # no ratio at a border, where there is no derivative
    want = _grad_of(lambda x: F.policy(x.double(), y, off, old, adv, **kw)[0][0].sum().item(), z)
    assert (grad - want).abs().max() < DIFF
    assert (grad[8] == 0).all() and (grad[2] == 0).all()   # behind the sequences, not scored


@pytest.mark.parametrize("kind,mean,eps", [("sigmoid", False, 0.0), ("sigmoid", True, 0.1),
                                           ("square", True, 0.0)])
def test_preference_formula_against_differences(kind, mean, eps):
    g, z, y = _case(seed=1)
    off = torch.tensor([0, 2, 5, 5, 9])
    ref = torch.randn(9, generator=g)
    kw = dict(ref=ref, beta=0.3, smoothing=eps, kind=kind, mean=mean,
              weights=torch.tensor([1.0, 0.5]))
    grad = F.preference(z, y, off, **kw)[3][0]
    want = _grad_of(lambda x: F.preference(x.double(), y, off, **kw)[0][0].sum().item(), z)
    assert (grad - want).abs().max() < DIFF * 10   # a square loss of size up to 1000


@pytest.mark.parametrize("tau,lse", [(1.0, False), (2.0, True)])
def test_distill_formula_against_differences(tau, lse):
    g, z, y = _case(seed=2)
    idx = torch.randint(0, 13, (9, 5), generator=g, dtype=torch.int32)
    idx[0, 1] = -1
    idx[1, 2] = idx[1, 3] = idx[1, 0]
    u = torch.randn(9, 5, generator=g)
    U = torch.logsumexp(u / tau, 1) + 0.5 if lse else None
    w = torch.rand(9, generator=g)
    kw = dict(teacher_lse=U, temperature=tau, weights=w)
    grad = F.distill(z, idx, u, **kw)[1][0]
    want = _grad_of(lambda x: F.distill(x.double(), idx, u, **kw)[0][0].sum().item(), z)
    assert (grad - want).abs().max() < DIFF


@pytest.mark.parametrize("grouped", [False, True])
def test_balance_formula_against_differences(grouped):
    g, z, _ = _case(seed=3)
    idx = torch.randint(0, 13, (9, 3), generator=g, dtype=torch.int32)
    idx[4] = -1
    idx[5, 1] = -1
    off = torch.tensor([0, 3, 3, 8]) if grouped else None

    def total(x):
        a, b, _, _ = F.balance(x.double(), idx, off, balance=0.7, z=0.2)
        return (0.7 * a[0] + 0.2 * b[0]).sum().item()

    grad = F.balance(z, idx, off, balance=0.7, z=0.2)[3][0]
    assert (grad - _grad_of(total, z)).abs().max() < DIFF
    loss = F.balance(torch.zeros(12, 4), torch.arange(12, dtype=torch.int32)[:, None] % 4)[0][0]
    assert abs(loss.item() - 1.0) < 1e-12      # all alike


def test_logp_formula_against_torch():
    _, z, y = _case(seed=4)
    r = F.Rows(z, 0.7)
    want = torch.log_softmax(z.double() * 0.7, 1).gather(1, y.long().clamp(min=0)[:, None])[:, 0]
    want[2] = 0
    assert (r.logp(y)[0] - want).abs().max() < 1e-12


# --- outputs on top of inputs

AT = {name: (k + 1) << 32 for k, name in enumerate(
    "logits labels grad offsets old adv ref weights index teacher tlse loss klo reward zloss counts "
    "logp lse dlogits ws".split())}
T_, V_, N_, K_, LD_ = 10, 64, 3, 4, 80
READS = {
    "token_logprobs": "logits labels",
    "token_logprobs_backward": "logits labels grad",
    "policy_loss": "logits labels offsets old adv ref weights",
    "preference_loss": "logits labels offsets ref weights",
    "distill_loss": "logits index teacher tlse weights",
    "balance_loss": "logits index offsets",
}
WRITES = {
    "token_logprobs": "logp lse ws",
    "token_logprobs_backward": "dlogits ws",
    "policy_loss": "loss klo logp dlogits ws",
    "preference_loss": "loss reward logp dlogits ws",
    "distill_loss": "loss dlogits ws",
    "balance_loss": "loss zloss counts dlogits ws",
}
PAIRS = [(n, o, i) for n in ALL for o in WRITES[n].split()
         for i in READS[n].split() + WRITES[n].split() if o != i and (o, i) != ("dlogits", "logits")]


def _sizes(name):
    """Bytes of each array of the calls below; rows of logits and gradient are LD_ apart."""
    seqs = 2 * N_ if name == "preference_loss" else N_
    per = 4 * (N_ if name in ("policy_loss", "preference_loss") else T_)
    op = {"token_logprobs": 0, "token_logprobs_backward": 0, "policy_loss": 1, "preference_loss": 2,
          "distill_loss": 3, "balance_loss": 4}[name]
    rows = ((T_ - 1) * LD_ + V_) * 4
    loss = 4 * (T_ if name == "distill_loss" else N_)
    return dict(logits=rows, dlogits=rows, labels=4 * T_, grad=4 * T_, offsets=8 * (seqs + 1),
                old=4 * T_, adv=4 * N_, ref=4 * T_, weights=per, index=4 * T_ * K_,
                teacher=4 * T_ * K_, tlse=4 * T_, loss=loss, klo=loss, reward=4 * seqs, zloss=loss,
                counts=4 * N_ * V_, logp=4 * T_, lse=4 * T_,
                ws=sk.losses_workspace_bytes(op, T_, V_, {3: K_, 4: N_}.get(op, 0), 0))


def _placed(at):
    p = {k: ctypes.c_void_p(v) for k, v in at.items()}
    return dict(p, T=T_, V=V_, ld=LD_, dld=LD_, n=N_, G=N_, K=K_)


@pytest.mark.parametrize("name,out,other", PAIRS)
def test_outputs_over_other_arrays_are_refused(lib, name, out, other):
    size = _sizes(name)
    # the first and the last element of either array in the other
    for at in (AT[other], AT[other] + size[other] - 4, AT[other] - size[out] + 4):
        assert _call(lib, name, _placed(dict(AT, **{out: at}))) == sk.SK_ERR_INVALID_ARG
        assert b"overlap" in lib.sinkhorn_last_error()


def test_arrays_side_by_side_are_accepted():
    """One array right behind another, and arrays in the gaps between padded rows: those calls reach
    the launch, which fails without a device."""
    program = f"""
import sys
sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, "tests")!r}]
import test_losses_cpu as t
lib = t.sk.load_library()
for name, out, other in t.PAIRS:
    size, at = t._sizes(name), dict(t.AT)
    for place in (at[other] + size[other], at[other] - size[out]):
        code = t._call(lib, name, t._placed(dict(at, **{{out: place}})))
        assert code == 5, (name, out, other, code, lib.sinkhorn_last_error())
    if size[out] <= 64 and other in ("logits", "dlogits"):
        for gap, code in ((256, 5), (256 + 64 - size[out], 5), (252, 1), (256 + 68 - size[out], 1)):
            place = at[other] + 3 * 320 + gap
            got = t._call(lib, name, t._placed(dict(at, **{{out: place}})))
            assert got == code, (name, out, other, gap, got, lib.sinkhorn_last_error())
print("done")
"""
    run = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True,
                         env=dict(os.environ, HIP_VISIBLE_DEVICES="-1"))
    assert run.returncode == 0 and run.stdout.split() == ["done"], run


@pytest.mark.parametrize("name", GRADS)
def test_matrices_beyond_the_address_space_are_refused(lib, name):
    """2^24 rows 2^38 elements apart end where they begin, modulo 2^64 bytes."""
    far = dict(_placed(dict(AT, logits=1 << 40, dlogits=(1 << 40) + 128)), T=1 << 24)
    for changes in (dict(ld=1 << 38, dld=1 << 38), dict(dld=1 << 38)):
        assert _call(lib, name, dict(far, **changes)) == sk.SK_ERR_INVALID_ARG
        assert b"elements apart" in lib.sinkhorn_last_error(), lib.sinkhorn_last_error()


# --- offsets that the documentation does not allow

def _bits(T):
    """Chunk sizes of the balance loss, as powers of two (to count, for the gradient)."""
    return (max(8, (T // 128 + 1).bit_length() - 1), max(4, (T // 1024 + 1).bit_length() - 1))


def _place(off, T, chunk, bits, count_bits):
    """A work-group's search for its chunk, as balance.hip does it with the 64 lanes of a wave;
    every index it reads is checked.  (group, first, last, first counting chunk, how many)."""
    G = len(off) - 1
    row = lambda i: min(max(off[i], 0), T)  # noqa: E731
    g, count = 0, G
    while True:
        step = (count + 63) // 64
        at = [min(g + lane * step, G) for lane in range(64)]
        begun = [g + lane * step < g + count and at[lane] + (row(at[lane]) >> bits) <= chunk
                 for lane in range(64)]
        lane = max(sum(begun) - 1, 0)
        g += lane * step
        assert 0 <= g < G
        if step == 1:
            b = row(at[lane])
            e = max(row(at[lane + 1]) if lane + 1 < 64 else row(g + 1), b)
            break
        count = min(step, count - lane * step)
        assert count >= 1
    chunks = lambda rows, k: (rows + (1 << k) - 1) >> k  # noqa: E731
    i = chunk - (g + (b >> bits))
    if i < 0 or i >= chunks(e - b, bits):
        return None
    first = b + (i << bits)
    return (g, first, min(first + (1 << bits), e), g + (b >> count_bits), chunks(e - b, count_bits))


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("ordered", [True, False])
def test_balance_chunks_stay_in_bounds(seed, ordered):
    """Whatever the offsets hold, no chunk lies outside the rows, the groups or the partial counts and
    sums; in order, every row of every group is in one chunk of it, once."""
    g = np.random.default_rng(seed)
    T = int(g.integers(1025, 300000))
    G = int(g.choice([1, 2, 63, 64, 65, 200, 5000]))
    off = g.integers(-1000, T + 1000, G + 1)
    if ordered:
        off = np.sort(off.clip(0, T))
    elif seed % 2:
        off[g.integers(0, G + 1, 3)] = [2 ** 40, -2 ** 62, 2 ** 62]
    off = [int(v) for v in off]
    cb, gb = _bits(T)
    for bits in (cb, gb):
        total = (T >> bits) + G
        seen = 0
        for chunk in range(total):
            place = _place(off, T, chunk, bits, cb)
            if place is None:
                continue
            group, first, last, count0, counts = place
            assert 0 <= group < G and 0 <= first < last <= T
            assert 0 <= count0 < (T >> cb) + G
            # the gradient's cap on what it reads of the partial counts
            assert min(counts, (T >> cb) + G - count0) >= 1
            if ordered:
                assert off[group] <= first and last <= off[group + 1]
                assert count0 + counts <= (T >> cb) + G
                seen += last - first
        if ordered:
            assert seen == off[-1] - off[0]
    for grp in range(G):    # the sums' launch
        assert 0 <= grp + (min(max(off[grp], 0), T) >> gb) < (T >> gb) + G
