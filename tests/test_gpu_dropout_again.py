"""Passes with dropout that are run again for their gradients, on the GPU."""
import pytest
import torch
from torch.utils.checkpoint import checkpoint

import lazy_optimizer_step_amd as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reentrant", [False, True])
def test_another_mask_is_refused(reentrant):
    """Without an offset the second run would draw the next mask, and the gradients would be those
    of another pass."""
    m = L.Dropout(0.5, seed=6)
    x = torch.randn(50, 60, device="cuda", requires_grad=True)
    y = checkpoint(lambda t: torch.square(m(t)), x, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="offset"):
        y.sum().backward()
    x.grad = None
    y = checkpoint(lambda t: torch.square(m(t, offset=4)), x, use_reentrant=reentrant)
    y.sum().backward()
    # kept values are doubled, and so are their gradients: (2 x)^2
    assert torch.equal(x.grad, 8.0 * x.detach() * (y.detach() != 0)) and m.offset == 1
