"""A classifier over bags of tokens, trained with the library's own steps only.

One training step runs everything the package has between a table and its loss:

  rows   = SparseEmbedding(ids)        gather of the table's rows
  rows   = Dropout(rows)               the mask from a counter, never stored
  normed = LayerNorm(rows)             forward kernel; its backward makes the per-lookup gradients
  loss   = LinearCrossEntropy(bags)    one dense matrix W and the loss, the logits never stored
  loss.backward()
  table.step()                         sparse Adam on the touched rows
  muon.step(W.grad)                    Muon on the matrix

    python examples/embedding_classifier.py [--steps 200] [--dropout 0.1]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lazy_optimizer_step_amd import Dropout, LayerNorm, LinearCrossEntropy, Muon  # noqa: E402
from lazy_optimizer_step_amd.embedding import SparseEmbedding  # noqa: E402


def batches(rows: int, classes: int, bags: int, bag: int, seed: int):
    """Bags of tokens; a token's class is its id modulo the classes, a bag's that of most of its
    tokens (three of four are drawn from the bag's class)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def draw(high, *shape):
        return torch.randint(high, shape, device="cuda", generator=g)
    while True:
        label = draw(classes, bags)
        own = draw(rows // classes, bags, bag) * classes + label[:, None]
        any_ = draw(rows, bags, bag)
        yield torch.where(draw(4, bags, bag) > 0, own, any_), label


def train(steps: int = 200, rows: int = 100_000, dim: int = 128, classes: int = 40,
          bags: int = 512, bag: int = 16, seed: int = 0, log=None,
          dropout: float = 0.0) -> list[float]:
    """Trains for `steps` batches; returns the losses."""
    torch.manual_seed(seed)
    table = SparseEmbedding(rows, dim, lr=1e-2, mode="lazy", init_std=0.05)
    drop, norm = Dropout(dropout, seed=seed), LayerNorm(dim)
    weight = torch.nn.Parameter(torch.randn(classes, dim, device="cuda") / dim ** 0.5)
    head = LinearCrossEntropy(dim, classes, weight=weight)
    muon = Muon(weight.detach(), lr=0.02, weight_decay=0.01)
    losses = []
    for step, (ids, label) in zip(range(steps), batches(rows, classes, bags, bag, seed)):
        loss = head(norm(drop(table(ids))).mean(1), label)
        loss.backward()
        table.step()
        muon.step(weight.grad)
        with torch.no_grad():
            for p in (norm.weight, norm.bias):
                p -= 0.01 * p.grad
        for p in (weight, norm.weight, norm.bias):
            p.grad = None
        losses.append(float(loss.detach()))
        if log and step % 20 == 0:
            log(f"step {step}: loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--dropout", type=float, default=0.0)
    args = ap.parse_args()
    got = train(args.steps, dropout=args.dropout, log=lambda s: print(s, flush=True))
    print(f"loss {got[0]:.3f} -> {sum(got[-10:]) / len(got[-10:]):.3f}")
