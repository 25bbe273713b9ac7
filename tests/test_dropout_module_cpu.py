"""Dropout's module without a GPU."""
import pytest
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


class _Again(torch.autograd.Function):
    """What activation checkpointing does: the pass is run in the backward pass."""
    @staticmethod
    def forward(ctx, x, run):
        ctx.run = run
        return x.clone()

    @staticmethod
    def backward(ctx, dy):
        ctx.run()
        return dy, None


def test_a_run_inside_a_backward_pass_needs_its_offset():
    m = L.Dropout(0.5, seed=1)
    x = torch.ones(3, requires_grad=True)
    with pytest.raises(RuntimeError, match="offset"):
        _Again.apply(x, lambda: m(x)).sum().backward()
    assert m.offset == 0
    # with one, it is the kernels' call that a CPU tensor stops
    with pytest.raises(ValueError, match="ROCm"):
        _Again.apply(x, lambda: m(x, offset=3)).sum().backward()
    m.eval()
    _Again.apply(x, lambda: m(x)).sum().backward()


def test_evaluation_takes_the_residuals_that_training_takes():
    m = L.Dropout(0.5, seed=1).eval()
    x = torch.ones(2, 3)
    assert torch.equal(m(x, 2 * x), 3 * x)
    with pytest.raises(ValueError, match="residual has shape"):
        m(x, torch.ones(3))
    with pytest.raises(TypeError, match="residual must be"):
        m(x, x.double())
