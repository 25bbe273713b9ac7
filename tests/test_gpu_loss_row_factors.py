"""Rows of very different factors on the GPU: each row's dx to its own accuracy, whichever kernels
the size takes, and dweight to that of the largest."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests import loss_ref as R
from tests.dense_ref import HALF, TINY, U
from tests.test_gpu_loss import make

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def reference(dl, x, w, t, lse, e, float32_g):
    """(dx, dweight, their bounds): g is off relative to its own row's factor."""
    dtype, (rows, cols), classes = x.dtype, x.shape, w.shape[0]
    split = dtype == F32 and not float32_g
    xc, wd, c = R.clean(x, t), w.double(), R.factors(dl, t, "none")[:, None]
    less = xc @ wd.T - lse.double()[:, None]
    p = torch.exp(less)
    y = torch.full_like(p, e / classes)
    y.scatter_add_(1, t.clamp(min=0)[:, None], torch.full_like(p[:, :1], 1 - e))
    g = torch.where(c != 0, c * (p - y), 0.0)
    ez = R.product_bound(xc, wd.T.contiguous(), cols, split)
    eg = c.abs() * (p * (ez + 3 * U * less.abs() + 6 * U) + 6 * U * y + 2 * U * (p - y).abs()
                    + 2.0 ** -126)
    # g's rounding: float16's smallest step where a row's factor is brought to 2^13 at least
    if split:
        eg = eg + 2.0 ** -22 * g.abs() + 2.0 ** -38 * c.abs()
    elif not float32_g:
        eg = eg + HALF[dtype] * g.abs() + (2.0 ** -38 * c.abs() if dtype == F16 else 0.0)
    top = c.abs().max()
    dx, dw = g @ wd, g.T @ xc
    # sums in float32; of two float16 the operands' last bits and lo lo as well
    k = 3 * 2.0 ** -22 if split else 0.0
    e_dx = eg @ wd.abs() + (2 * U * (classes + 8) + k) * (g.abs() @ wd.abs())
    e_dw = eg.T @ xc.abs() + (2 * U * (rows + 8) + k) * (g.abs().T @ xc.abs())
    if split:
        e_dx = e_dx + 2.0 ** -39 * wd.abs().max() * g.abs().sum(1, keepdim=True)
    if dtype != BF16 and not float32_g:
        # what float16 takes of a row's c x, or of its g beside the largest's
        e_dw = e_dw + 2.0 ** -37 * top * (g != 0).double().T @ (xc.abs() + xc.abs().max())
    return (dx, dw, HALF[dtype] * dx.abs() + TINY[dtype] + 2 * e_dx,
            HALF[dtype] * dw.abs() + TINY[dtype] + 2 * e_dw)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("size", [(30, 64, 1500), (70, 61, 40), (500, 256, 30001), (500, 250, 30001),
                                  (1500, 130, 9001)], ids=str)
@pytest.mark.parametrize("e", [0.0, 0.1])
def test_factors_of_many_sizes(size, dtype, e):
    """Factors from 2^12 down to 2^-12: in the rows of small ones all classes together count as much
    as the target does."""
    rows, cols, classes = size
    direct = L.linear_cross_entropy_plan(*size, dtype, backward=True)["direct"]
    assert direct == (rows < 100)
    x, w, t = make(*size, dtype, scale=0.5)
    w[:, 0] = 1.0
    g = torch.Generator(device="cuda").manual_seed(5)
    dl = torch.exp2(12 - 24 * torch.rand(rows, device="cuda", generator=g))
    dl[0], dl[1], dl[2], dl[3] = 2.0 ** 12, -(2.0 ** -12), 0.0, -1.5
    t[0] = t[1] = 3
    lse = L.linear_cross_entropy_forward(x, w, t)[1]
    dx, dw = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none", label_smoothing=e)
    rx, rw, bx, bw = reference(dl, x, w, t, lse, e, dtype == F32 and direct)
    R.within(dx, rx, bx, "dx")
    R.within(dw, rw, bw, "dweight")
    # each alone gives the same
    a, b = (L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none", label_smoothing=e,
                                            want_dx=k, want_dweight=not k) for k in (True, False))
    assert torch.equal(a[0], dx) and torch.equal(b[1], dw)


@pytest.mark.parametrize("dtype", [F32, F16], ids=str)
@pytest.mark.parametrize("size", [(30, 64, 150), (500, 250, 30001)], ids=str)
def test_factors_at_the_ends(size, dtype):
    """The smallest and the largest that float32 holds beside each other; and factors that are not
    finite leave the other rows' dx alone."""
    x, w, t = make(*size, dtype, ignored=0.0)
    lse = L.linear_cross_entropy_forward(x, w, t)[1]
    dl = torch.ones(size[0], device="cuda")
    want = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none")[0]
    for big in (2.0 ** 126, float("inf"), float("nan")):
        dl[5] = big
        dl[7], dl[8] = 2.0 ** -149, -(2.0 ** -126)
        dx = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none")[0]
        rest = torch.ones(size[0], dtype=torch.bool, device="cuda")
        rest[[5, 7, 8]] = False
        # powers of two apart, in a scale of another mantissa's: the same but for roundings
        assert (dx[rest].double() - want[rest].double()).norm() < 2.0 ** -9 * want[rest].double().norm()
        assert torch.isfinite(dx[7]).all() and torch.isfinite(dx[8]).all()
        if dtype == F32:
            assert float(dx[8].abs().max()) > 2.0 ** -130
        assert not torch.isfinite(dx[5]).all() or big == 2.0 ** 126


@pytest.mark.parametrize("dtype", [F32, F16], ids=str)
@pytest.mark.parametrize("size", [(30, 64, 150), (500, 250, 30001), (9000, 64, 2000)], ids=str)
def test_captured(size, dtype):
    x, w, t = make(*size, dtype)
    dl = torch.rand(size[0], device="cuda")

    def gradients():
        lse = L.linear_cross_entropy_forward(x, w, t)[1]
        return L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none")
    gradients()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gradients()
    for k in range(4):
        dl[k::3] *= 2.0 ** (7 - 4 * k)
        x.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, gradients()))
