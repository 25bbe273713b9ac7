"""Many rows of few classes on the GPU: what is found out about all rows is found out once."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests import loss_ref as R
from tests.test_gpu_loss import make

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("size", [(50001, 40, 10), (300001, 64, 10), (9000, 250, 1000),
                                  (40000, 64, 2000)], ids=str)
def test_values(size, reduction, dtype):
    """Few classes take the kernels of small calls, the others those of large ones; a workspace
    that holds anything."""
    rows, cols, classes = size
    assert L.linear_cross_entropy_plan(*size, dtype, backward=True)["direct"] == (classes <= 10)
    x, w, t = make(*size, dtype)
    loss, lse = L.linear_cross_entropy_forward(x, w, t, reduction=reduction)
    dl = torch.rand(rows, device="cuda") + 0.1 if reduction == "none" else \
        torch.tensor(0.7, device="cuda")
    space = torch.full((L.linear_cross_entropy_workspace_size(*size, dtype, backward=True),), 255,
                       dtype=torch.uint8, device="cuda")
    dx, dw = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction=reduction, workspace=space)
    rl, rs, bl, bs = R.forward(x, w, t, reduction, 0.0)
    R.within(lse, rs, bs, "lse")
    R.within(loss, rl, bl, "loss")
    rx, rw, bx, bw = R.backward(dl, x, w, t, lse, reduction, 0.0)
    R.within(dx, rx, bx, "dx")
    R.within(dw, rw, bw, "dweight")


@pytest.mark.parametrize("dtype,reduction", [(F32, "mean"), (F32, "none"), (BF16, "none")], ids=str)
def test_time_grows_with_the_rows(dtype, reduction):
    """Four times the rows may take eight times as long; work that grows with their square takes
    sixteen times as long."""
    took = []
    for rows in (250_000, 1_000_000):
        x, w, t = make(rows, 64, 10, dtype)
        loss, lse = L.linear_cross_entropy_forward(x, w, t, reduction=reduction)
        dl = torch.ones_like(loss)
        space = torch.empty(L.linear_cross_entropy_workspace_size(rows, 64, 10, dtype, backward=True),
                            dtype=torch.uint8, device="cuda")
        each = []
        for _ in range(5):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction=reduction, workspace=space)
            end.record()
            torch.cuda.synchronize()
            each.append(begin.elapsed_time(end))
        took.append(min(each))
    assert took[1] < 8 * took[0], took


def test_captured():
    """A graph of a call whose rows are scanned, replayed with other targets and factors."""
    x, w, t = make(60000, 40, 12, BF16)
    dl = torch.rand(60000, device="cuda")
    lse = L.linear_cross_entropy_forward(x, w, t)[1]

    def gradients():
        return L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none") + \
            L.linear_cross_entropy_backward(dl[:1], x, w, t, lse)
    gradients()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gradients()
    for k in range(3):
        t[k::5] = R.IGNORED
        dl.mul_(1.5 + k)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, gradients()))
