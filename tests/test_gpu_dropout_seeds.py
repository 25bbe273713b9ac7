"""Seeds of Dropout modules on the GPU: drawn ones, and what a state dict keeps."""
import copy

import pytest
import torch

import lazy_optimizer_step_amd as L

pytestmark = pytest.mark.gpu


def mask(m, n=4096):
    return m(torch.ones(n, device="cuda")) != 0


def test_modules_without_a_seed_differ():
    torch.manual_seed(3)
    a, b = L.Dropout(0.5), L.Dropout(0.5)
    layers = [copy.deepcopy(a) for _ in range(2)]
    masks = [mask(m) for m in (a, b, *layers)]
    for i in range(4):
        for j in range(i):
            # 4096 fair coins agree at half of their places, 32 is one deviation
            assert abs(int((masks[i] == masks[j]).sum()) - 2048) < 6 * 32
    torch.manual_seed(3)
    assert torch.equal(mask(L.Dropout(0.5)), masks[0])


def test_state_dict_goes_on_with_the_same_masks():
    m = L.Dropout(0.5)
    mask(m)
    again = L.Dropout(0.5)
    again.load_state_dict(m.state_dict())
    assert torch.equal(mask(again), mask(m))
    # into a seed on the device: in place
    seed = torch.zeros(1, dtype=torch.int64, device="cuda")
    on_device = L.Dropout(0.5, seed=seed)
    on_device.load_state_dict(m.state_dict())
    assert on_device.seed is seed and torch.equal(mask(on_device), mask(m))
    # and out of one, which the caller then changes
    state = on_device.state_dict()
    seed.fill_(5)
    other = L.Dropout(0.5, seed=1)
    other.load_state_dict(state)
    assert torch.equal(mask(other), mask(m))
