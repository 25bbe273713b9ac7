"""Dropout's module without a GPU."""
import torch

import lazy_optimizer_step_amd as L


def test_seed_in_the_state_dict():
    m = L.Dropout(0.5, seed=77)
    m.offset = 4
    again = L.Dropout(0.5)
    again.load_state_dict(m.state_dict())
    assert (again.seed, again.offset) == (77, 4)
    # one that was not drawn yet, or a state that holds none, leaves the module's
    again.load_state_dict(L.Dropout(0.5).state_dict())
    assert (again.seed, again.offset) == (77, 0)
    again.set_extra_state({"offset": 9})
    assert (again.seed, again.offset) == (77, 9)


def test_no_seed_until_the_first_training_pass():
    m = L.Dropout(0.5)
    before = torch.get_rng_state()
    x = torch.ones(3)
    assert m.eval()(x) is x and m.seed is None
    assert torch.equal(before, torch.get_rng_state())
