"""The loss's largest tiles on the GPU against 64 bits, at sizes that take them in the loss, in g and in
both gradients."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests.test_gpu_loss import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("cols,classes,pieces", [(4090, 4000, 1), (4096, 4000, 1), (4096, 39960, 2)],
                         ids=str)
def test_256_tiles(dtype, cols, classes, pieces):
    """Rows that are copied and rows that are read in place; remainders in rows and classes, and
    columns too."""
    rows = 3990
    f, b = (L.linear_cross_entropy_plan(rows, cols, classes, dtype, backward=k) for k in (False, True))
    assert f["tile_logits"] == b["tile_logits"] == b["tile_dx"] == b["tile_dw"] == 256
    assert not f["direct"] and not b["direct"]
    assert -(-classes // f["piece"]) == -(-classes // b["piece"]) == pieces
    a = make(rows, cols, classes, dtype)
    check(*a, "none", 0.1)
    check(*a, "mean")
