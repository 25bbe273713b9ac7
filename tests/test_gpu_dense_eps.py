"""The smallest eps that are accepted: constant rows give the bias, zero matrices zeros."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests import dense_ref as R
from tests import ns_form as F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [5, 64, 1001, 20000])
@pytest.mark.parametrize("eps", [1e-45, 1e-38, 1e-5])
def test_constant_rows(cols, eps):
    x = torch.full((3, cols), 2.5, device="cuda")
    w, b = torch.rand(cols, device="cuda"), torch.rand(cols, device="cuda")
    y, mean, rstd = L.layer_norm_forward(x, w, b, eps=eps)
    assert torch.equal(y, b.expand(3, cols)) and torch.equal(mean, x[:, 0])
    assert rstd.isfinite().all()


@pytest.mark.parametrize("shape", [(3, 40, 60), (3, 64, 1100), (3, 200, 150)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("eps", [5e-324, 1e-320, 1e-307, 1e-300])
def test_zero_and_tiny_matrices(shape, eps):
    """One launch, panels and tiles; the others of the batch have any size."""
    g = F.rand(*shape)
    g[0] = 0
    g[1] *= 1e-30
    out = L.newton_schulz(g.cuda(), eps=eps)
    assert not out[0].any()
    ref = R.newton_schulz(g[1:], eps=eps)
    off = (R.d(out[1:]) - ref).flatten(-2).norm(dim=-1)
    assert (off < (F.LOW + R.HALF[torch.bfloat16]) * ref.flatten(-2).norm(dim=-1)).all()
