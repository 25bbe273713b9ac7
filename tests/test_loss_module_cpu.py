"""LinearCrossEntropy's table without a GPU."""
import pytest
import torch

import lazy_optimizer_step_amd as L


def test_a_table_without_a_gradient_is_refused():
    """It would train everything but the table, and say nothing."""
    with pytest.raises(ValueError, match="no gradient"):
        L.LinearCrossEntropy(8, 10, weight=torch.zeros(10, 8))


def test_tables_that_are_taken():
    p = torch.nn.Parameter(torch.zeros(10, 8))
    assert L.LinearCrossEntropy(8, 10, weight=p).weight is p
    fixed = torch.nn.Parameter(torch.zeros(10, 8), requires_grad=False)
    assert L.LinearCrossEntropy(8, 10, weight=fixed).weight is fixed
    made = 2 * p
    assert L.LinearCrossEntropy(8, 10, weight=made).weight is made
    own = L.LinearCrossEntropy(8, 10, device="cpu").weight
    assert isinstance(own, torch.nn.Parameter) and own.requires_grad and own.shape == (10, 8)
