"""The smallest eps that are accepted: constant rows give the bias, zero matrices zeros."""
import pytest
import torch

import lazy_optimizer_step_amd as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [5, 64, 1001, 20000])
@pytest.mark.parametrize("eps", [1e-45, 1e-38, 1e-5])
def test_constant_rows(cols, eps):
    x = torch.full((3, cols), 2.5, device="cuda")
    w, b = torch.rand(cols, device="cuda"), torch.rand(cols, device="cuda")
    y, mean, rstd = L.layer_norm_forward(x, w, b, eps=eps)
    assert torch.equal(y, b.expand(3, cols)) and torch.equal(mean, x[:, 0])
    assert rstd.isfinite().all()
