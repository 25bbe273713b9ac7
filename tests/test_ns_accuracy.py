"""Accuracy of the Newton-Schulz kernels' roundings, emulated in 64 bits, against fixed bounds."""
import pytest

from tests import dense_ref as R
from tests import ns_form as F

SIZES = [(8, 8), (16, 24), (40, 128), (64, 64), (64, 300), (128, 128), (300, 100), (256, 512)]


def off(got, ref):
    return float((got - ref).norm() / ref.norm())


@pytest.mark.parametrize("shape", SIZES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_matrices_that_lack_directions(shape):
    for name, g in F.low_inputs(*shape):
        assert off(F.kernel_form(g), R.newton_schulz(g)) < F.LOW, name
        assert off(F.kernel_form(g, steps=8), R.newton_schulz(g, steps=8)) < F.MORE, name


@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (2, 2), (2, 5), (3, 5), (5, 3), *SIZES],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_any_matrix(shape):
    for name, g in F.other_inputs(*shape):
        assert off(F.kernel_form(g), R.newton_schulz(g)) < F.ANY, name


def test_the_bound_tells_the_forms_apart():
    """With float32 X at the diagonal in every step (the form dense_ref rounds by), rounding grows
    in the directions that these lack."""
    for g in (F.rank(64, 64, 1), F.rows(512, 512, 4), F.softmax_gradient(1, 40, 128)):
        ref = R.newton_schulz(g)
        assert off(R.newton_schulz(g, rounded=True), ref) > F.LOW
        assert off(F.kernel_form(g), ref) < F.LOW
