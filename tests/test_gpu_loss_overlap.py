"""Outputs of the loss and of dropout that lie where an input does, on the GPU: refused where a
kernel would read what it has written."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests.test_gpu_loss import make

pytestmark = pytest.mark.gpu


def test_loss():
    x, w, t = make(16, 16, 16, torch.float32)
    f, b = L.linear_cross_entropy_forward, L.linear_cross_entropy_backward
    lse = torch.empty(16, device="cuda")
    space = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for kw in (dict(out=lse, lse=lse), dict(lse=w.flatten()[:16]), dict(out=x.flatten()[:16]),
               dict(workspace=w.view(-1).view(torch.uint8)),
               dict(lse=space[:64].view(torch.float32), workspace=space)):
        with pytest.raises(ValueError, match="may not be"):
            f(x, w, t, reduction="none", **kw)
    f(x, w, t, reduction="none", lse=lse)
    dl = torch.ones(16, device="cuda")
    for kw in (dict(out=x), dict(out=w), dict(dweight=x), dict(dweight=w),
               dict(out=space[:1024].view(torch.float32).view(16, 16), workspace=space),
               dict(out=space[:1024].view(torch.float32).view(16, 16),
                    dweight=space[:1024].view(torch.float32).view(16, 16))):
        before = x.clone(), w.clone()
        with pytest.raises(ValueError, match="may not be"):
            b(dl, x, w, t, lse, reduction="none", **kw)
        assert torch.equal(x, before[0]) and torch.equal(w, before[1])
    # beside one another in one buffer
    both = torch.empty(32, 16, device="cuda")
    dx, dw = b(dl, x, w, t, lse, reduction="none", out=both[:16], dweight=both[16:])
    want = b(dl, x, w, t, lse, reduction="none")
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_dropout():
    buf = torch.randn(40, 16, device="cuda")
    x = buf[:8, :10]
    other = buf.flatten()[:80].view(8, 10)      # x's values, as rows without gaps
    for call in (lambda: L.dropout_forward(x, 0.5, 1, out=other),
                 lambda: L.dropout_forward(buf[9:17, :10], 0.5, 1, residual=x, out=other),
                 lambda: L.dropout_backward(x, 0.5, 1, out=other)):
        with pytest.raises(ValueError, match="may not be"):
            call()
    want = L.dropout_forward(x, 0.5, 1)
    assert torch.equal(L.dropout_forward(x, 0.5, 1, out=x), want)
