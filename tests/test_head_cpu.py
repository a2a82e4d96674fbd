"""The output end of a model, host side: its header, its refusals, and the formulas of the tests
against automatic differentiation and against torch."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import sinkhorn_point_cloud_amd as sk

import head_formulas as H

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sinkhorn_head.h")


@pytest.fixture(scope="module")
def lib():
    return sk.load_library()


def test_header_library_and_binding_name_the_same_functions(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(sinkhorn_\w+)\s*\(", text))
    assert names == set(sk.HEAD_EXPORTS)
    out = os.popen(f"nm -D --defined-only {sk.library_path()}").read()
    for name in names:
        assert re.search(rf"\bT {name}$", out, flags=re.M), name
    for name in ("rms_norm", "rms_norm_int8", "rms_norm_backward", "quantize_int8", "int8_linear",
                 "token_scores", "token_scores_backward", "head_workspace_bytes"):
        assert name in sk.__all__ and callable(getattr(sk, name))


def test_workspace_bytes(lib):
    ws = sk.head_workspace_bytes
    for op, V, k in ((0, 64, 0), (1, 64, 64), (2, 64, 16), (3, 64, 0)):
        assert ws(op, 100, V, k, 0) > 0 and ws(op, 0, V, k, 1) > 0
        assert ws(op, -1, V, k, 0) == 0 and ws(op, 100, 0, k, 0) == 0
        assert ws(op, 100, V, k, 7) == 0 and ws(op, (1 << 24) + 1, V, k, 0) == 0
    assert ws(4, 1, 1, 1, 0) == 0 and ws(-1, 1, 1, 1, 0) == 0
    assert ws(0, 10, 32769, 0, 0) == 0
    assert ws(1, 10, 64, 0, 0) == 0 and ws(1, 10, 64, 131072, 0) == 0
    assert ws(2, 10, 64, 129, 0) == 0 and ws(2, 10, 64, -1, 0) == 0 and ws(3, 10, 64, 1, 0) == 0
    # nothing of the size of the logits or the weights
    assert ws(1, 4096, 131072, 4096, 1) < 1 << 20 and ws(2, 4096, 131072, 64, 1) < 1 << 20


def at(mb):
    """An address that nothing else of the call lies near; never dereferenced."""
    return ctypes.c_void_p((mb + 1) << 20)


def _call(lib, name, changes):
    """One entry point with arguments that are in order but for `changes`."""
    base = dict(x=at(0), dtype=0, ldx=64, res=None, ldr=64, weight=at(1), T=10, d=64, eps=1e-6,
                y=at(2), ldy=64, h=at(3), ldh=64, q=at(4), ldq=64, scale=at(5), dy=at(6), lddy=64,
                dh=at(7), lddh=64, dx=at(8), lddx=64, dw=at(9), ws=at(4096), ws_bytes=1 << 40,
                x8=at(10), ldx8=64, xs=at(11), w8=at(12), ldw8=64, wsc=at(13), bias=None, K=64,
                N=32, out=at(14), ldo=32, z=at(15), ld=64, labels=at(16), V=64, s=1.0, top=4,
                logp=at(17), lse=at(18), ent=at(19), index=at(20), best=at(21), grad=at(22),
                gent=at(23), dz=at(24), dld=64)
    base.update(changes)
    order = {
        "rms_norm": "x dtype ldx res ldr weight T d eps y ldy h ldh",
        "rms_norm_int8": "x dtype ldx res ldr weight T d eps q ldq scale h ldh",
        "quantize_int8": "x dtype ldx T d q ldq scale",
        "rms_norm_backward": "dy dtype lddy h ldh weight dh lddh T d eps dx lddx dw ws ws_bytes",
        "int8_linear": "x8 ldx8 xs w8 ldw8 wsc bias T K N dtype out ldo ws ws_bytes",
        "token_scores": "z dtype ld labels T V s top logp lse ent index best ws ws_bytes",
        "token_scores_backward": "z dtype ld labels grad gent T V s dz dld ws ws_bytes",
    }[name]
    return getattr(lib, "sinkhorn_" + name)(*[base[n] for n in order.split()], None)


ALL = ("rms_norm", "rms_norm_int8", "quantize_int8", "rms_norm_backward", "int8_linear",
       "token_scores", "token_scores_backward")
NORMS = ALL[:4]
SCORES = ALL[5:]
BAD = sk.SK_ERR_INVALID_ARG


@pytest.mark.parametrize("name,changes,code", [
    *[(n, c, BAD) for n in ALL for c in (dict(dtype=2), dict(T=-1), dict(T=(1 << 24) + 1))],
    *[(n, c, BAD) for n in NORMS for c in (dict(d=0), dict(d=32769, ldx=1 << 16, ldh=1 << 16))],
    *[(n, c, BAD) for n in NORMS[:3] for c in (
        dict(x=None), dict(ldx=63), dict(x=ctypes.c_void_p((1 << 20) + 2)))],
    *[(n, c, BAD) for n in (NORMS[0], NORMS[1], NORMS[3]) for c in (
        dict(eps=0.0), dict(eps=math.nan), dict(eps=math.inf), dict(eps=-1.0), dict(ldh=63))],
    *[("rms_norm", c, BAD) for c in (
        dict(y=None), dict(ldy=60), dict(res=at(50), ldr=10), dict(y=at(3)),
        dict(h=at(2)), dict(y=ctypes.c_void_p((1 << 20) + 256)), dict(y=at(0), ldy=65),
        dict(weight=ctypes.c_void_p((3 << 20) + 64)))],
    *[(n, c, BAD) for n in ("rms_norm_int8", "quantize_int8") for c in (
        dict(q=None), dict(scale=None), dict(ldq=63), dict(q=at(0)), dict(scale=at(4)),
        dict(scale=ctypes.c_void_p((6 << 20) + 2)))],
    *[("rms_norm_backward", c, BAD) for c in (
        dict(dy=None), dict(h=None), dict(dx=None), dict(lddx=63), dict(dx=at(6), lddx=65),
        dict(dw=at(6)), dict(dw=at(8)), dict(ws=at(6)), dict(dx=at(1)))],
    ("rms_norm_backward", dict(ws=None), sk.SK_ERR_WORKSPACE),
    ("rms_norm_backward", dict(ws_bytes=64), sk.SK_ERR_WORKSPACE),
    *[("int8_linear", c, BAD) for c in (
        dict(x8=None), dict(w8=None), dict(xs=None), dict(wsc=None), dict(out=None), dict(K=0),
        dict(K=131072, ldx8=1 << 18, ldw8=1 << 18), dict(N=0), dict(N=(1 << 24) + 1), dict(ldx8=48),
        dict(ldx8=72), dict(ldw8=72), dict(ldo=31), dict(out=at(10)), dict(out=at(12)),
        dict(x8=ctypes.c_void_p((11 << 20) + 8)), dict(w8=ctypes.c_void_p((13 << 20) + 4)),
        dict(out=ctypes.c_void_p((15 << 20) + 2)), dict(ws=at(14)),
        dict(T=1 << 24, N=1 << 24, ldo=1 << 24))],
    ("int8_linear", dict(ws=None), sk.SK_ERR_WORKSPACE),
    *[(n, c, BAD) for n in SCORES for c in (
        dict(z=None), dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25, dld=1 << 25), dict(ld=63),
        dict(s=0.0), dict(s=1e-21), dict(s=1e21), dict(s=math.nan), dict(s=-1.0),
        dict(z=ctypes.c_void_p((16 << 20) + 2)))],
    *[(n, c, sk.SK_ERR_WORKSPACE) for n in SCORES for c in (dict(ws=None), dict(ws_bytes=8))],
    *[("token_scores", c, BAD) for c in (
        dict(top=-1), dict(top=129), dict(index=None), dict(best=None), dict(top=0),
        dict(labels=None), dict(top=0, logp=None, lse=None, ent=None, index=None, best=None),
        dict(lse=at(17)), dict(index=at(15)), dict(best=at(20)), dict(logp=at(16)), dict(ws=at(15)),
        dict(ent=ctypes.c_void_p((20 << 20) + 1)))],
    *[("token_scores_backward", c, BAD) for c in (
        dict(grad=None, gent=None), dict(labels=None), dict(dz=None), dict(dld=63),
        dict(dz=ctypes.c_void_p((16 << 20) + 256)), dict(dz=at(15), dld=65), dict(dz=at(22)),
        dict(ws=at(24)))],
])
def test_refusals(lib, name, changes, code):
    assert _call(lib, name, changes) == code, lib.sinkhorn_last_error()
    assert lib.sinkhorn_last_error()


def test_no_rows_need_no_row_pointers(lib):
    none = dict(T=0, x=None, y=None, h=None, q=None, scale=None, x8=None, xs=None, out=None, z=None,
                labels=None, logp=None, lse=None, ent=None, index=None, best=None, grad=None,
                gent=None, dz=None, dy=None, dx=None, dh=None, dw=None)
    for name in ALL:
        assert _call(lib, name, none) == sk.SK_OK, (name, lib.sinkhorn_last_error())


def test_refusals_write_nothing(lib):
    # host memory: a launch would not be allowed to touch it, a refusal does not try
    x = np.full(64, 3.0, dtype=np.float32)
    p = x.ctypes.data_as(ctypes.c_void_p)
    for name in ("rms_norm_backward", "token_scores", "token_scores_backward", "int8_linear"):
        changes = dict(dw=p, logp=p, lse=None, ent=None, ws_bytes=0)
        assert _call(lib, name, changes) == sk.SK_ERR_WORKSPACE
    assert np.all(x == 3.0)


def test_overlaps_that_are_none(lib):
    """Columns of one buffer side by side, and outputs that are inputs themselves, pass the checks:
    what refuses them here is the absence of a device."""
    side = dict(x=at(0), ldx=128, y=ctypes.c_void_p((1 << 20) + 256), ldy=128)
    for name, changes in (("rms_norm", side), ("rms_norm", dict(y=at(0))),
                          ("rms_norm", dict(res=at(30), h=at(30))), ("rms_norm", dict(h=None)),
                          ("rms_norm_backward", dict(dx=at(6))), ("rms_norm_backward", dict(dx=at(3))),
                          ("rms_norm_backward", dict(dx=at(7))),
                          ("token_scores_backward", dict(dz=at(15))),
                          ("token_scores", dict(top=0, index=None, best=None))):
        code = _call(lib, name, changes) if not torch.cuda.is_available() else sk.SK_ERR_HIP
        assert code == sk.SK_ERR_HIP, (name, lib.sinkhorn_last_error())


def test_binding_refusals():
    z = torch.zeros(4, 8)
    e = z.to(torch.int8)
    for call in (sk.rms_norm, sk.rms_norm_int8, sk.quantize_int8, sk.token_scores,
                 lambda x: sk.rms_norm_backward(x, x), lambda x: sk.token_scores_backward(x, None)):
        with pytest.raises(ValueError):
            call(z)                      # not on the GPU
        with pytest.raises(ValueError):
            call(z[0])                   # not a matrix
        with pytest.raises(TypeError):
            call(z.double())
    with pytest.raises(ValueError):
        sk.int8_linear(e, z[:, 0], e, z[:, 0])
    with pytest.raises(TypeError):
        sk.int8_linear(z, z[:, 0], e, z[:, 0])


# --- the formulas themselves

def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_norm_formula_against_autograd():
    g = gen(0)
    h = torch.randn(5, 12, generator=g).double().requires_grad_()
    w = torch.randn(12, generator=g).double().requires_grad_()
    dy, dh = torch.randn(5, 12, generator=g).double(), torch.randn(5, 12, generator=g).double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 0.01) * w
    want = torch.autograd.grad((y * dy).sum() + (h * dh).sum(), (h, w))
    assert torch.allclose(H.norm(h.detach(), w.detach(), 0.01, torch.float64)[0], y.detach(), atol=1e-12)
    (dx, _), (dw, _) = H.norm_backward(dy, h.detach(), w.detach(), dh, 0.01)
    assert torch.allclose(dx, want[0], atol=1e-12) and torch.allclose(dw, want[1], atol=1e-12)


def test_eight_bits_formula():
    x = torch.tensor([[1.0, -0.5, 0.25, 0.0], [0.0] * 4, [math.inf, 1.0, 0, 0], [math.nan, 1, 2, 3]])
    q, scale, _ = H.eight(x, None, None)
    assert q.tolist() == [[127, -64, 32, 0], [0] * 4, [0] * 4, [0] * 4]      # 63.5 and 31.75
    assert scale[:2].tolist() == [1.0 / 127, 0.0] and scale[2:].isnan().all()


def test_scores_formula_against_autograd():
    g = gen(1)
    z = torch.randn(6, 9, generator=g).double()
    z[1, 3:] = -math.inf
    y = torch.tensor([0, 1, 2, -1, 8, 4], dtype=torch.int32)
    gl, ge = torch.randn(6, generator=g), torch.randn(6, generator=g)
    S = H.Scores(z, y, 0.7, 5)
    x = z.clone().requires_grad_()
    logq = torch.log_softmax(0.7 * x, 1)
    q = logq.exp()
    ent = -torch.where(q > 0, q * torch.where(q > 0, logq, 0.0), 0.0).sum(1)
    logp = logq.gather(1, y.clamp(min=0).long()[:, None])[:, 0]
    keep = y >= 0
    assert torch.allclose(S.entropy[0][keep], ent.detach()[keep], atol=1e-12)
    assert torch.allclose(S.logp[0][keep], logp.detach()[keep], atol=1e-12)
    total = (gl.double() * logp)[keep].sum() + (ge.double() * ent)[keep].sum()
    want = torch.autograd.grad(total, x)[0]
    assert torch.allclose(S.backward(y, gl, ge)[0], want.nan_to_num(), atol=1e-12)
    top = logq.detach().topk(5, dim=1)
    assert torch.equal(S.index[0], top.indices[0].int())
    assert torch.allclose(S.best[0][0], top.values[0], atol=1e-12)
    assert S.index[1].tolist()[3:] == [-1, -1] and S.index[3].tolist() == [-1] * 5


def test_gradient_formula_against_differences():
    g = gen(2)
    z = torch.randn(3, 7, generator=g).double()
    y = torch.tensor([1, 0, 6], dtype=torch.int32)
    gl, ge = torch.randn(3, generator=g), torch.randn(3, generator=g)
    grad = H.Scores(z, y, 1.3).backward(y, gl, ge)[0]

    def total(z):
        S = H.Scores(z, y, 1.3)
        return (gl.double() * S.logp[0] + ge.double() * S.entropy[0]).sum()
    step = 1e-5
    for t in range(3):
        for v in range(7):
            e = torch.zeros_like(z)
            e[t, v] = step
            assert abs((total(z + e) - total(z - e)) / (2 * step) - grad[t, v]) < 1e-8


def test_equal_values_come_in_the_order_of_their_index():
    z = torch.tensor([[0.0, -0.0, 1.0, 0.0, -math.inf, 1.0, math.nan, math.inf]])
    index, best = H.alternatives(z, [True], torch.tensor([math.nan]).double(), 1.0, 8)
    assert index[0].tolist() == [6, 7, 2, 5, 0, 1, 3, -1]
    assert best[0, :7].isnan().all() and best[0, 7] == -math.inf
