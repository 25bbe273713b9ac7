"""Small calls of 16-bit types on the GPU: what rounds their gradients is the results' type alone."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests import loss_ref as R
from tests.dense_ref import HALF, TINY, U
from tests.test_gpu_loss import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("size", [(17, 100, 64), (65, 128, 257), (130, 33, 1001), (5, 1000, 130),
                                  (3, 64, 20001), (2001, 40, 10), (40, 24, 2), (300, 100, 3001)],
                         ids=str)
@pytest.mark.parametrize("reduction,e", [("none", 0.0), ("mean", 0.1)])
def test_gradients(size, dtype, reduction, e):
    rows, cols, classes = size
    assert L.linear_cross_entropy_plan(*size, dtype, backward=True)["direct"]
    x, w, t = make(*size, dtype)
    # what all classes share leaves dx again, as a row of g adds up to nothing
    w[:, ::2] += 8.0
    dl = torch.rand(rows, device="cuda") + 0.5 if reduction == "none" else \
        torch.tensor(0.7, device="cuda")
    lse = L.linear_cross_entropy_forward(x, w, t)[1]
    dx, dw = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction=reduction, label_smoothing=e)
    xc, wd, c = R.clean(x, t), w.double(), R.factors(dl, t, reduction)[:, None]
    less = xc @ wd.T - lse.double()[:, None]
    p = torch.exp(less)
    y = torch.full_like(p, e / classes)
    y.scatter_add_(1, t.clamp(min=0)[:, None], torch.full_like(p[:, :1], 1 - e))
    g = torch.where(c != 0, c * (p - y), 0.0)
    ez = R.product_bound(xc, wd.T.contiguous(), cols, False)
    eg = c.abs() * (p * (ez + 3 * U * less.abs() + 6 * U) + 6 * U * y + 2 * U * (p - y).abs()
                    + 2.0 ** -126)
    # g as two of the type: what the second leaves, and float16's smallest step beside 2^13
    eg = eg + HALF[dtype] ** 2 * g.abs()
    if dtype == torch.float16:
        eg = eg + 2.0 ** -38 * c.abs().max()
    dx64, dw64 = g @ wd, g.T @ xc
    R.within(dx, dx64, HALF[dtype] * dx64.abs() + TINY[dtype]
             + 2 * (eg @ wd.abs() + R.product_bound(g, wd, 2 * classes, False)), "dx")
    R.within(dw, dw64, HALF[dtype] * dw64.abs() + TINY[dtype]
             + 2 * (eg.T @ xc.abs() + R.product_bound(g.T.contiguous(), xc, 2 * rows, False)),
             "dweight")
