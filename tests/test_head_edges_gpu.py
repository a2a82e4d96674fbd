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
