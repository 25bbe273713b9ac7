"""Batches of small matrices beyond what one grid of the one-launch kernels takes: the 16-wave
forms have 1024 threads a block, and a grid fewer than 2^32 threads along an axis."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests import dense_ref as R

pytestmark = pytest.mark.gpu

N = 129   # one row of 129 and more columns: 16 waves
GRID = 1 << 20


def rows(batch, dtype):
    g = torch.empty(batch, 1, N, dtype=dtype, device="cuda")
    return g.normal_(generator=torch.Generator(device="cuda").manual_seed(batch % 1000))


def factor(steps=5):
    """A row's singular value is 1 at first (eps is far below its norm)."""
    s = 1.0
    for _ in range(steps):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    return s


def test_more_than_two_to_the_22():
    batch = (1 << 22) + 3
    g = rows(batch, torch.bfloat16)
    out = torch.full(g.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    L.newton_schulz(g, out=out)
    want = factor()
    # every matrix: its norm, off by the form's error (1e-2) and half a step of bfloat16
    norm = torch.linalg.vector_norm(out, dim=(1, 2), dtype=torch.float32)
    assert ((norm - want).abs() <= (1e-2 + R.HALF[torch.bfloat16]) * want).all()
    for at in (0, GRID - 1, GRID, 2 * GRID, 3 * GRID - 1, (1 << 22) - 1, 1 << 22, batch - 1):
        x = R.d(g[at])
        assert (R.d(out[at]) - want * x / x.norm()).norm() <= (1e-2 + R.HALF[torch.bfloat16]) * want


def test_momentum_and_weight_of_every_matrix():
    batch = GRID + 3
    g = rows(batch, torch.bfloat16)
    buf = torch.ones(batch, 1, N, device="cuda")
    p = torch.zeros(batch, 1, N, device="cuda")
    L.muon_step(p, g, buf, lr=1.0, momentum=0.5, nesterov=False, scale=-1.0)
    assert torch.equal(buf, 0.5 + g.float())
    norm = torch.linalg.vector_norm(p, dim=(1, 2))
    assert ((norm - factor()).abs() <= 1e-2 * factor()).all()
    for at in (0, GRID - 1, GRID, batch - 1):
        x = R.d(buf[at])
        assert (R.d(p[at]) - factor() * x / x.norm()).norm() <= 1e-2 * factor()
