"""Long tables of classes of which one, early in the table, has nearly all the probability: what the
others share must not be lost beside it in a sum over thousands of them."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests import loss_ref as R

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("e", [0.0, 0.1])
def test_a_class_near_one_early(dtype, e):
    """65536 rows: so many tiles of rows that a block goes through all classes."""
    rows, cols, classes, first = 65536, 64, 131072, 300
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(rows, cols, device="cuda", generator=g)
    w = torch.randn(classes, cols, device="cuda", generator=g) * 0.01
    x[:, 0] = 4.0
    w[:, 0] = 0.25
    # e^18.7 is 999 times the 131071 others' share: a loss of about 1e-3
    w[first, 0] = 0.25 + 18.7 / 4
    x, w = x.to(dtype), w.to(dtype)
    t = torch.full((rows,), first, device="cuda")
    loss, lse = L.linear_cross_entropy_forward(x, w, t, reduction="none", label_smoothing=e)
    some = torch.arange(0, rows, 997, device="cuda")
    xd, wd = x[some].double(), w.double()
    z = xd @ wd.T
    ez = R.product_bound(xd, wd.T.contiguous(), cols, dtype == F32)
    want = torch.logsumexp(z, 1)
    top = z[:, first:first + 1]
    p = torch.exp(z - want[:, None])
    # the sum itself, of magnitudes: a tile's values in a lane, the lane's double rounded, joins of
    # lanes and waves, factors where bases differ: 64 + 1 + 8 + 3 + 3 half steps at most
    e_sum = 79 * R.U
    each = p * (ez + 3 * R.U * (top - z))
    # the target's logit is the one value in its loss and in the sum: its error counts by 1 - p
    rest = torch.cat([each[:, :first], each[:, first + 1:]], 1).sum(1)
    at = ez[:, first] * ((1 - p[:, first]) if e == 0 else 1.0)
    ref = want - (1 - e) * z[:, first] - e * z.mean(1)
    # a tile's logits are added in float32: 64 half steps at most, their sum rounded once more
    bound = rest + at + e_sum + R.U * ref.abs() + e * (ez.mean(1) + 66 * R.U * z.abs().mean(1))
    R.within(loss[some], ref, 2 * bound, "loss")
    R.within(lse[some], want, 2 * (each.sum(1) + e_sum + R.U * want.abs()), "lse")
    if e == 0:
        # the bound is a small part of what the other classes give
        assert float((2 * bound / ref).max()) < 0.03
