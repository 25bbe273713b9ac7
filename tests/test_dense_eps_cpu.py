"""Values of eps that the kernels' arithmetic cannot hold are refused on the host."""
import pytest

from lazy_optimizer_step_amd import _lib

FAKE = 256  # a non-NULL address that is never dereferenced


@pytest.mark.parametrize("eps", [1e-46, 5e-324, 1e39, 1.7e308])
def test_layer_norm_refuses_what_float32_does_not_hold(eps):
    rc = _lib.lib().layer_norm_forward(FAKE, 8, 4, 8, 0, FAKE, FAKE, 0, eps, FAKE, 8, FAKE, FAKE,
                                       None, 0)
    assert rc == _lib.EINVAL
    assert b"eps" in _lib.lib().sparse_opt_last_error()


@pytest.mark.parametrize("eps", [1e-45, 1e-38, 1e-5, 3e38])
def test_layer_norm_takes_the_rest(eps):
    """No rows: the arguments are checked and nothing is launched."""
    assert _lib.lib().layer_norm_forward(None, 8, 0, 8, 0, None, None, 0, eps, None, 8, None, None,
                                         None, 0) == 0
