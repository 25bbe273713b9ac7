"""The table, dropout, layer norm and the loss over a table of classes in one training step."""
import importlib.util
import os

import pytest
import torch

import lazy_optimizer_step_amd as L
from lazy_optimizer_step_amd.embedding import SparseEmbedding
from tests import dense_ref as D
from tests import loss_ref as R

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_gradient_of_a_step():
    """Each stage's gradient against its 64-bit form, from the gradient that reached it."""
    torch.manual_seed(3)
    emb = SparseEmbedding(500, 48, init_std=1.0)
    drop, norm = L.Dropout(0.25, seed=11), L.LayerNorm(48)
    head = L.LinearCrossEntropy(48, 300, label_smoothing=0.1)
    with torch.no_grad():
        norm.weight.uniform_(0.5, 1.5)
    ids = torch.randint(500, (7, 9), device="cuda")
    t = torch.randint(300, (7, 9), device="cuda")
    t[3, 4:] = R.IGNORED
    kept = drop(emb(ids))
    kept.retain_grad()
    h = norm(kept)
    h.retain_grad()
    loss = head(h, t)
    loss.backward()
    flat = lambda a: a.detach().view(63, -1)  # noqa: E731
    goal = t.view(63)
    # the loss
    args = flat(h), head.weight.detach(), goal
    want, lse, bound, _ = R.forward(*args, "mean", 0.1)
    R.within(loss.detach(), want, bound, "loss")
    lse = L.linear_cross_entropy_forward(*args, label_smoothing=0.1)[1]
    dl = torch.ones((), device="cuda")
    dx, dw, bx, bw = R.backward(dl, *args, lse, "mean", 0.1)
    R.within(flat(h.grad), dx, bx, "dx")
    R.within(head.weight.grad, dw, bw, "dweight")
    assert not h.grad[3, 4:].any()
    # the norm
    x = flat(kept)
    _, mean, rstd = L.layer_norm_forward(x, norm.weight.detach(), norm.bias.detach())
    args = flat(h.grad), x, mean, rstd, norm.weight
    ref, bounds = D.ln_backward(*args), D.ln_backward_bounds(*args, torch.float32)
    for got, r, b, name in zip((flat(kept.grad), norm.weight.grad, norm.bias.grad), ref, bounds,
                               ("dx", "dweight", "dbias")):
        D.within(got, r, b, name)
    # dropout, and the rows that the table's step takes
    (got_ids, rows), = emb._pending
    assert torch.equal(got_ids, ids.flatten())
    want, bound = R.dropout(flat(kept.grad), 0.25, 11, 0)
    R.within(rows, want, bound, "rows")
    assert torch.equal((rows != 0).cpu() | (flat(kept.grad) == 0).cpu(),
                       R.kept((63, 48), 0.25, 11) | (flat(kept.grad) == 0).cpu())
    before = emb.weight.clone()
    assert emb.step() == 63
    touched = torch.zeros(500, dtype=torch.bool, device="cuda")
    touched[ids.flatten()] = True
    assert torch.equal(emb.weight[~touched], before[~touched])


def test_captured_step():
    """Forward and backward of a step in one graph, replayed with other lookups, targets and
    masks, against the same calls outside it."""
    torch.manual_seed(4)
    table = torch.randn(400, 64, device="cuda")
    gain, shift = torch.rand(64, device="cuda") + 0.5, torch.randn(64, device="cuda")
    out = torch.randn(1001, 64, device="cuda") / 8
    ids = torch.randint(400, (130,), device="cuda")
    t = torch.randint(1001, (130,), device="cuda")
    seed = torch.tensor([1], device="cuda")
    one = torch.ones((), device="cuda")

    def step():
        rows = L.read_rows(table, ids)
        x = L.dropout_forward(rows, 0.1, seed, residual=rows)
        h, mean, rstd = L.layer_norm_forward(x, gain, shift)
        loss, lse = L.linear_cross_entropy_forward(h, out, t)
        dh, dout = L.linear_cross_entropy_backward(one, h, out, t, lse)
        dx, dgain, dshift = L.layer_norm_backward(dh, x, mean, rstd, gain)
        return [loss, lse, dout, dgain, dshift, L.dropout_backward(dx, 0.1, seed)]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(3):
        ids.copy_(torch.randint(400, (130,), device="cuda"))
        t.copy_(torch.randint(1001, (130,), device="cuda"))
        t[::7] = R.IGNORED
        seed.fill_(100 + k)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_example_runs_with_dropout():
    spec = importlib.util.spec_from_file_location(
        "embedding_classifier", os.path.join(ROOT, "examples", "embedding_classifier.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(steps=3, rows=4000, classes=10, bags=64, bag=8, dropout=0.2)
    assert len(losses) == 3 and all(x == x and x > 0 for x in losses)
