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
