"""Which kernels the loss takes at a size: the query, and sizes that tests and documents speak of."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from lazy_optimizer_step_amd import _lib

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def plan(*size, backward=True):
    return L.linear_cross_entropy_plan(*size, backward=backward)


def test_sizes():
    assert plan(8, 128, 1001, F32)["direct"] and plan(8, 128, 1001, F16)["direct"]
    for backward in (False, True):
        p = plan(8192, 4096, 131072, BF16, backward=backward)
        assert not p["direct"] and p["tile_logits"] == 256
        assert (p["tile_dx"], p["tile_dw"]) == ((256, 256) if backward else (0, 0))
    p = plan(8192, 128, 50021, F32)
    assert not p["direct"] and p["piece"] < 50021 and p["piece"] % 256 == 0


def test_refusals():
    for bad in [(0, 8, 10), (-1, 8, 10), (4, 0, 10), (4, 8, 0)]:
        with pytest.raises(L.SparseOptError) as e:
            plan(*bad, F32)
        assert e.value.code == _lib.EINVAL
    assert _lib.lib().linear_cross_entropy_plan(4, 8, 10, 0, 0, None) == _lib.EINVAL
    assert _lib.lib().linear_cross_entropy_plan(4, 8, 10, 3, 0, _lib.CePlan()) == _lib.EINVAL
