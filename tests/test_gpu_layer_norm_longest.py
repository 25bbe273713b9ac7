"""Layer norm's weight gradients of a row longer than one grid's blocks along the columns take."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests import dense_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [(1 << 25) + 7, (1 << 30) + 33])
def test_weight_gradients(cols):
    gen = torch.Generator(device="cuda").manual_seed(cols % 1000)
    x = torch.empty(1, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    dy = torch.empty(1, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    mean, rstd = torch.tensor([0.25], device="cuda"), torch.tensor([0.75], device="cuda")
    dw = torch.full((cols,), float("nan"), device="cuda")
    db = torch.full((cols,), float("nan"), device="cuda")
    L.layer_norm_backward(dy, x, mean, rstd, None, want_dx=False, dweight=dw, dbias=db)
    step = 1 << 26
    for at in range(0, cols, step):
        g, v = dy[0, at:at + step].float(), x[0, at:at + step].float()
        # one row: its products alone, of three rounded operations
        want = g.double() * ((v.double() - 0.25) * 0.75)
        off = (dw[at:at + step].double() - want).abs()
        assert (off <= 4 * R.U * g.double().abs() * (v.double().abs() + 0.25) * 0.75).all()
        assert torch.equal(db[at:at + step], g)
