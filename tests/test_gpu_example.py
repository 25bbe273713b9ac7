"""The example that runs the table, the layer norm and Muon together."""
import importlib.util
import os

import pytest
import torch

import lazy_optimizer_step_amd as L
from lazy_optimizer_step_amd.embedding import SparseEmbedding
from tests import dense_ref as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_learns():
    spec = importlib.util.spec_from_file_location(
        "embedding_classifier", os.path.join(ROOT, "examples", "embedding_classifier.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(steps=60, rows=4000, classes=10, bags=256, bag=8)
    # 10 classes at random: ln 10 = 2.30; chance stays there
    assert losses[0] > 1.8
    assert sum(losses[-5:]) / 5 < 0.7


def test_gradient_that_reaches_the_table():
    """The per-lookup rows the table's step takes are the layer norm's gradient by the formula."""
    torch.manual_seed(3)
    emb = SparseEmbedding(500, 48, init_std=1.0)
    norm = L.LayerNorm(48)
    with torch.no_grad():
        norm.weight.uniform_(0.5, 1.5)
    ids = torch.randint(500, (7, 9), device="cuda")
    dy = torch.randn(7, 9, 48, device="cuda")
    norm(emb(ids)).backward(dy)
    (got_ids, rows), = emb._pending
    assert torch.equal(got_ids, ids.flatten())
    x = emb.weight[got_ids]
    _, mean, rstd = L.layer_norm_forward(x, norm.weight.detach(), norm.bias.detach())
    args = (dy.view(63, 48), x, mean, rstd, norm.weight)
    R.within(rows, R.ln_backward(*args)[0], R.ln_backward_bounds(*args, torch.float32)[0], "dx")
    assert emb.step() == 63
