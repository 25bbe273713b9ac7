"""Checks of the loss over a table of classes and of dropout that need no GPU: refusals of the C ABI
before any device work, workspace sizes, and the 64-bit forms themselves."""
import numpy as np
import pytest
import torch

import lazy_optimizer_step_amd as L
from lazy_optimizer_step_amd import _lib
from tests import loss_ref as R

FAKE = 256  # a non-NULL, 16-byte aligned address that is never dereferenced
NAN, INF = float("nan"), float("inf")


def fwd(x=FAKE, xs=8, w=FAKE, ws=8, rows=4, cols=8, classes=10, dt=0, t=FAKE, ign=-100, e=0.0, how=2,
        loss=FAKE, lse=FAKE, work=FAKE, have=1 << 40, flags=0):
    return _lib.lib().linear_cross_entropy_forward(x, xs, w, ws, rows, cols, classes, dt, t, ign, e,
                                                   how, loss, lse, work, have, None, flags)


def bwd(dl=FAKE, x=FAKE, xs=8, w=FAKE, ws=8, rows=4, cols=8, classes=10, dt=0, t=FAKE, ign=-100,
        e=0.0, how=2, lse=FAKE, dx=FAKE, dxs=8, dw=FAKE, dws=8, work=FAKE, have=1 << 40, flags=0):
    return _lib.lib().linear_cross_entropy_backward(dl, x, xs, w, ws, rows, cols, classes, dt, t, ign,
                                                    e, how, lse, dx, dxs, dw, dws, work, have, None,
                                                    flags)


BOTH = [{"x": None}, {"w": None}, {"t": None}, {"lse": None}, {"rows": -1}, {"cols": 0},
        {"classes": 0}, {"dt": 3}, {"dt": -1}, {"how": 3}, {"how": -1}, {"e": -0.1}, {"e": 1.5},
        {"e": NAN}, {"xs": 7}, {"ws": 7}, {"rows": (1 << 28) + 1}, {"cols": (1 << 20) + 1},
        {"classes": (1 << 30) + 1}, {"rows": 1 << 28, "cols": 1 << 20, "xs": 1 << 20, "ws": 1 << 20}]


@pytest.mark.parametrize("kw", BOTH + [{"loss": None}, {"loss": None, "rows": 0}], ids=str)
def test_loss_forward_refuses(kw):
    assert fwd(**kw) == _lib.EINVAL
    assert b"linear_cross_entropy_forward" in _lib.lib().sparse_opt_last_error()


@pytest.mark.parametrize("kw", BOTH + [{"dl": None}, {"dxs": 7}, {"dws": 7}], ids=str)
def test_loss_backward_refuses(kw):
    assert bwd(**kw) == _lib.EINVAL
    assert b"linear_cross_entropy_backward" in _lib.lib().sparse_opt_last_error()


@pytest.mark.parametrize("kw", [{"work": None}, {"work": 8}, {"have": 1000}], ids=str)
def test_loss_refuses_workspaces(kw):
    assert fwd(**kw) == _lib.EWORKSPACE
    assert bwd(**kw) == _lib.EWORKSPACE


def test_loss_without_work_touches_nothing():
    assert fwd(rows=0, x=None, t=None, loss=None, lse=None, work=None, have=0, how=0) == _lib.OK
    assert bwd(dx=None, dw=None, work=None, have=0) == _lib.OK
    assert bwd(rows=0, dl=None, x=None, t=None, lse=None, dw=None, work=None, have=0) == _lib.OK


def test_loss_workspace_size():
    size = L.linear_cross_entropy_workspace_size
    assert size(0, 8, 10, torch.float32, backward=True) == 0
    # the logits of a large batch are never there: 8192 x 131072 of them are 4 GiB
    assert size(8192, 4096, 131072, torch.bfloat16, backward=False) < 1 << 29
    assert size(8192, 4096, 131072, torch.bfloat16, backward=True) < 1 << 30
    for bad in [(-1, 8, 10), (4, 0, 10), (4, 8, 0), (4, 8, 1 << 31)]:
        with pytest.raises(L.SparseOptError) as e:
            size(*bad, torch.float32, backward=False)
        assert e.value.code == _lib.EINVAL
    assert _lib.lib().linear_cross_entropy_workspace_size(4, 8, 10, 0, 0, None) == _lib.EINVAL


def drop(x=FAKE, xs=8, res=None, rs=8, rows=4, cols=8, dt=0, p=0.5, seed=1, ds=None, off=0, y=FAKE,
         ys=8):
    return _lib.lib().dropout_forward(x, xs, res, rs, rows, cols, dt, p, seed, ds, off, y, ys, None, 0)


@pytest.mark.parametrize("kw", [{"x": None}, {"y": None}, {"rows": -1}, {"cols": 0}, {"dt": 3},
                                {"p": -0.01}, {"p": 1.01}, {"p": NAN}, {"p": INF}, {"xs": 7},
                                {"ys": 7}, {"res": FAKE, "rs": 7},
                                {"rows": 1 << 40, "cols": 1 << 40}], ids=str)
def test_dropout_refuses(kw):
    assert drop(**kw) == _lib.EINVAL
    assert b"dropout_forward" in _lib.lib().sparse_opt_last_error()
    if "res" not in kw:
        k = dict(x=FAKE, xs=8, rows=4, cols=8, dt=0, p=0.5, y=FAKE, ys=8)
        k.update(kw)
        assert _lib.lib().dropout_backward(k["x"], k["xs"], k["rows"], k["cols"], k["dt"], k["p"], 1,
                                           None, 0, k["y"], k["ys"], None, 0) == _lib.EINVAL
        assert b"dropout_backward" in _lib.lib().sparse_opt_last_error()


def test_dropout_no_rows_needs_no_arrays():
    assert drop(rows=0, x=None, y=None) == _lib.OK


def test_python_refusals():
    x = torch.zeros(4, 8)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="ROCm"):
        L.linear_cross_entropy_forward(x, x, t)
    with pytest.raises(ValueError, match="ROCm"):
        L.dropout_forward(x, 0.5, 1)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        L.dropout_forward(x.double(), 0.5, 1)
    with pytest.raises(ValueError, match="p must lie"):
        L.Dropout(1.5)
    with pytest.raises(ValueError, match="reduction"):
        L.LinearCrossEntropy(8, 10, reduction="total", device="cpu")
    with pytest.raises(ValueError, match="weight has shape"):
        L.LinearCrossEntropy(8, 10, weight=torch.zeros(8, 10))


# ---- the 64-bit forms -----------------------------------------------------------------------

def test_generator_known_answers():
    """The published answers of Philox4x32-10 (the generator's known-answer vectors)."""
    ones = [0xFFFFFFFF] * 4
    for ctr, key, want in [
            ([0] * 4, (0, 0), [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
            (ones, (0xFFFFFFFF, 0xFFFFFFFF), [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], (0xA4093822, 0x299F31D0),
             [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])]:
        assert R.philox(np.array([ctr]), key)[0].tolist() == want


def test_mask_bits_by_hand():
    """Value i takes the i % 8 th 16 bits of counter i / 8, the lowest first."""
    words = R.philox(np.array([[0, 0, 5, 0], [1, 0, 5, 0]]), (7, 9))
    want = [int(w) >> s & 0xFFFF for row in words for w in row for s in (0, 16)]
    seed = 7 | 9 << 32
    assert R.bits16(0, 16, seed, 5).tolist() == want
    assert R.bits16(3, 10, seed, 5).tolist() == want[3:13]


@pytest.mark.parametrize("p", [0.1, 0.5, 0.9])
def test_mask_keeps_its_share(p):
    n = 1 << 16
    share = R.kept((n,), p, 12345).double().mean()
    assert abs(float(share) - (1 - p)) < 6 * (p * (1 - p) / n) ** 0.5


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("e", [0.0, 0.1])
def test_form_against_torch_and_differences(reduction, e):
    torch.manual_seed(3)
    x, w = torch.randn(9, 5, dtype=torch.float64), torch.randn(7, 5, dtype=torch.float64)
    t = torch.tensor([0, 6, R.IGNORED, 3, 3, 1, R.IGNORED, 2, 5])
    xt, wt = x.clone().requires_grad_(), w.clone().requires_grad_()
    ref = torch.nn.functional.cross_entropy(xt @ wt.T, t, reduction=reduction, label_smoothing=e)
    f32 = torch.float32  # the bounds' type; the forms take 64 bits whatever it is
    loss, lse, *_ = R.forward(x.to(f32), w.to(f32), t, reduction, e)
    assert torch.allclose(loss, ref.detach(), atol=1e-5)
    dl = torch.rand(9, dtype=torch.float64) if reduction == "none" else torch.tensor(0.7).double()
    ref.backward(dl)
    dx, dw, *_ = R.backward(dl, x.to(f32), w.to(f32), t, lse, reduction, e)
    assert torch.allclose(dx, xt.grad, atol=1e-5) and torch.allclose(dw, wt.grad, atol=1e-5)
    x32, w32 = x.to(f32).double(), w.to(f32).double()

    def value(a, b):
        z = a @ b.T
        rows = torch.logsumexp(z, 1) - (1 - e) * z.gather(1, t.clamp(min=0)[:, None])[:, 0] \
            - e * z.mean(1)
        return float((rows * R.factors(dl, t, reduction)).sum())
    ax, aw, h = torch.randn_like(x), torch.randn_like(w), 1e-6
    diff = (value(x32 + h * ax, w32 + h * aw) - value(x32 - h * ax, w32 - h * aw)) / (2 * h)
    assert abs(diff - float((dx * ax).sum() + (dw * aw).sum())) < 1e-7
