"""The Newton-Schulz kernels against 64 bits within fixed bounds, on inputs that are hard on
rounding: low rank, few rows that are not zero, gradients of few samples, constant values.

The result is taken in float32, as a Muon step on a weight of zeros writes it."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests import dense_ref as R
from tests import ns_form as F

pytestmark = pytest.mark.gpu


def orthogonal(g, **kw):
    p = torch.zeros(g.shape, device="cuda")
    L.muon_step(p, g.cuda(), lr=1.0, momentum=0.0, scale=-1.0, **kw)
    return p


def check(g, bound, name, steps=5, coefficients=F.MUON, on="cpu"):
    ref = R.newton_schulz(g, steps=steps, coef=coefficients, on=on)
    got = orthogonal(g, steps=steps, coefficients=coefficients).to(ref.device).double()
    norm = ref.norm()
    assert (got - ref).norm() < bound * norm, (name, float((got - ref).norm() / norm))
    out = L.newton_schulz(g.cuda(), steps=steps, coefficients=coefficients).to(ref.device).double()
    assert (out - ref).norm() < (bound + R.HALF[torch.bfloat16]) * norm, name


# every form: one launch by 8 and 16 waves, panels, tiles; both orientations
SIZES = [(8, 8), (40, 128), (64, 64), (64, 200), (500, 60), (64, 1024), (128, 128), (250, 128),
         (60, 1100), (128, 512), (1001, 128), (256, 256), (300, 520), (700, 260)]


@pytest.mark.parametrize("shape", SIZES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_matrices_that_lack_directions(shape):
    for name, g in F.low_inputs(*shape):
        check(g, F.LOW, name)
        check(g, F.MORE, name + ", 8 steps", steps=8)
        check(g, F.LOW, name + ", 10 steps", steps=10, coefficients=(2.0, -1.5, 0.5))


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (1, 3000), (2, 2), (2, 5), (3, 5), (5, 3),
                                   *SIZES], ids=lambda s: f"{s[0]}x{s[1]}")
def test_any_matrix(shape):
    for name, g in F.other_inputs(*shape):
        check(g, F.ANY, name)


@pytest.mark.parametrize("shape", [(1100, 1100), (2048, 2100), (4100, 4096)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_large_matrices(shape):
    """The larger tiles; the 64-bit iteration runs on the GPU."""
    for name, g in (("rank 1", F.rank(*shape, 1)), ("4 rows", F.rows(*shape, 4))):
        check(g, F.LOW, name, on="cuda")


def test_a_batch_of_them():
    g = torch.stack([x for _, x in F.low_inputs(96, 80)])
    got = R.d(orthogonal(g))
    ref = R.newton_schulz(g)
    off = (got - ref).flatten(-2).norm(dim=-1) / ref.flatten(-2).norm(dim=-1)
    assert off.max() < F.LOW
