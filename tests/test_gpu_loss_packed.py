"""The loss's kernels for large calls on the GPU: operands copied or split, the table in pieces; and
those for small calls held to float32.  Every test says which kernels it means, so
that another rule cannot leave it without them."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from lazy_optimizer_step_amd import _lib
from tests import loss_ref as R
from tests.test_gpu_loss import make

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
# columns that 16-bit types read in place, and columns that they copy
COLS = pytest.mark.parametrize("cols", [256, 250])
ROWS, CLASSES = 500, 30001
NAN, INF = float("nan"), float("inf")


def packed(cols, dtype, rows=ROWS, classes=CLASSES):
    for backward in (False, True):
        assert not L.linear_cross_entropy_plan(rows, cols, classes, dtype, backward=backward)["direct"]


def both(x, w, t, dl, reduction="none", e=0.0, **kw):
    loss, lse = L.linear_cross_entropy_forward(x, w, t, reduction=reduction, label_smoothing=e, **kw)
    return loss, lse, *L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction=reduction,
                                                       label_smoothing=e, **kw)


def check(x, w, t, dl, reduction="none", e=0.0, tiny=0.0):
    got = both(x, w, t, dl, reduction, e)
    rl, rs, bl, bs = R.forward(x, w, t, reduction, e)
    R.within(got[1], rs, bs, "lse")
    R.within(got[0], rl, bl, "loss")
    rx, rw, bx, bw = R.backward(dl, x, w, t, got[1], reduction, e)
    R.within(got[2], rx, bx + tiny, "dx")
    R.within(got[3], rw, bw + tiny, "dweight")
    return got


def weights(rows=ROWS):
    return torch.rand(rows, device="cuda") + 0.5


@TYPES
@COLS
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_values(dtype, cols, reduction):
    packed(cols, dtype)
    x, w, t = make(ROWS, cols, CLASSES, dtype)
    dl = weights() if reduction == "none" else torch.tensor(0.7, device="cuda")
    check(x, w, t, dl, reduction, 0.1 if reduction == "mean" else 0.0)


@TYPES
@COLS
@pytest.mark.parametrize("bad", [NAN, INF, -INF, 1e30])
def test_ignored_rows_may_hold_anything(dtype, cols, bad):
    packed(cols, dtype)
    x, w, t = make(ROWS, cols, CLASSES, dtype, ignored=0.3)
    dl = weights()
    plain = both(x, w, t, dl, e=0.1)
    gone = t == R.IGNORED
    x[gone] = bad
    dl[gone] = bad
    got = both(x, w, t, dl, e=0.1)
    assert all(torch.equal(a, b) for a, b in zip(got, plain))
    L.linear_cross_entropy_forward(x, w, t, validate=True)
    assert not got[0][gone].any() and not got[1][gone].any() and not got[2][gone].any()


@TYPES
@COLS
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_no_row_counts(dtype, cols, reduction):
    packed(cols, dtype)
    x, w, t = make(ROWS, cols, CLASSES, dtype)
    t.fill_(R.IGNORED)
    x.fill_(NAN)
    dl = weights() if reduction == "none" else torch.ones((), device="cuda")
    assert not any(a.any() for a in both(x, w, t, dl, reduction))


@TYPES
@COLS
def test_another_ignore_index(dtype, cols):
    packed(cols, dtype)
    x, w, t = make(ROWS, cols, CLASSES, dtype, ignored=0.0)
    t[::3] = 7
    want = t.clone()
    want[::3] = R.IGNORED
    x[::3] = NAN
    dl = torch.ones((), device="cuda")
    a = both(x, w, t, dl, "mean", ignore_index=7)
    b = both(x, w, want, dl, "mean")
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@TYPES
@COLS
@pytest.mark.parametrize("target", [CLASSES, -1, -(1 << 62), 1 << 62])
def test_target_outside_the_classes(dtype, cols, target):
    packed(cols, dtype)
    x, w, t = make(ROWS, cols, CLASSES, dtype, ignored=0.0)
    good, lse0 = L.linear_cross_entropy_forward(x, w, t, reduction="none")
    t[4] = target
    dl = weights()
    loss, lse, dx, dw = both(x, w, t, dl)
    keep = torch.arange(ROWS, device="cuda") != 4
    assert torch.isnan(loss[4]) and torch.equal(loss[keep], good[keep]) and torch.equal(lse, lse0)
    assert torch.isnan(dx[4]).all() and torch.isfinite(dx[keep]).all() and torch.isnan(dw).all()
    with pytest.raises(L.SparseOptError) as err:
        L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none", validate=True)
    assert err.value.code == _lib.ERANGE


@TYPES
@COLS
@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_row_that_is_not_finite_stays_alone(dtype, cols, bad):
    packed(cols, dtype)
    x, w, t = make(ROWS, cols, CLASSES, dtype, ignored=0.0)
    w[:, 5] = w[:, 5].abs() + 0.01  # an infinity in x: every logit of its row is one
    dl = weights()
    good = both(x, w, t, dl)
    x[4, 5] = bad
    loss, lse, dx, dw = both(x, w, t, dl)
    keep = torch.arange(ROWS, device="cuda") != 4
    assert torch.isnan(loss[4]) and torch.isnan(dx[4]).all() and torch.isnan(dw).all()
    if dtype != F32:
        assert torch.equal(loss[keep], good[0][keep]) and torch.equal(dx[keep], good[2][keep])
    else:
        # the row's finite values still count for the power of two in front of x
        want, _, bound, _ = R.forward(x[keep], w, t[keep], "none", 0.0)
        R.within(loss[keep], want, bound, "loss")
        assert torch.isfinite(dx[keep]).all()


@TYPES
@COLS
@pytest.mark.parametrize("pad,first", [(3, 1), (64, 8)])
def test_strides(dtype, cols, pad, first):
    """Rows with gaps, from odd and from even addresses; gaps of the outputs keep what they hold."""
    packed(cols, dtype)
    x0, w0, t = make(ROWS, cols, CLASSES, dtype)
    xb = torch.full((ROWS, cols + pad), 9.0, device="cuda", dtype=dtype)
    wb = torch.full((CLASSES, cols + pad), 9.0, device="cuda", dtype=dtype)
    cut = slice(first, first + cols)
    xb[:, cut], wb[:, cut] = x0, w0
    dl = weights()
    want = both(x0, w0, t, dl)
    loss, lse = L.linear_cross_entropy_forward(xb[:, cut], wb[:, cut], t, reduction="none")
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
    dxb, dwb = torch.full_like(xb, 7.0), torch.full_like(wb, 7.0)
    dx, dw = L.linear_cross_entropy_backward(dl, xb[:, cut], wb[:, cut], t, lse, reduction="none",
                                             out=dxb[:, cut], dweight=dwb[:, cut])
    assert torch.equal(dx, want[2]) and torch.equal(dw, want[3])
    for buf in (dxb, dwb):
        assert (buf[:, :first] == 7).all() and (buf[:, first + cols:] == 7).all()


def test_range_of_float32():
    """Powers of two in front of the operands cancel; what does not fit beside the largest value
    is small beside it."""
    packed(250, F32)
    x, w, t = make(ROWS, 250, CLASSES, F32, ignored=0.1)
    dl = weights()
    for a, b in ((2.0 ** 60, 2.0 ** -60), (2.0 ** -100, 2.0 ** 100), (2.0 ** 120, 2.0 ** -120)):
        # the gradients leave float32's normal values at these ends: dx beside 2^-120, dweight
        # beside 2^-100, where a step is 2^-149
        check(x * a, w * b, t, dl, tiny=2.0 ** -149)
    w[7] *= 2.0 ** 10
    check(x * 2.0 ** -10, w, t, dl)
    check(torch.zeros_like(x), torch.zeros_like(w), t, dl)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_large_logits(dtype):
    packed(256, dtype)
    x, w, t = make(ROWS, 256, CLASSES, dtype, ignored=0.1)
    check(x * 64, w * 64, t, weights())
    check(x * 64, w * 64, t, torch.tensor(0.7, device="cuda"), "mean", 0.1)


@pytest.mark.parametrize("factor", [0.0, 1e-30, 1e30, -2.0])
@pytest.mark.parametrize("size", [(30, 64, 150), (ROWS, 250, CLASSES)], ids=str)
@TYPES
def test_factors_of_any_size(dtype, factor, size):
    """Also where float16 cannot hold the result: an infinity of its sign there."""
    x, w, t = make(*size, dtype)
    direct = L.linear_cross_entropy_plan(*size, dtype, backward=True)["direct"]
    assert direct == (size[0] == 30)
    _, lse = L.linear_cross_entropy_forward(x, w, t)
    dl = torch.full((size[0],), factor, device="cuda")
    dl[::5] *= 2.0 ** -12
    got = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none")
    *ref, bx, bw = R.backward(dl, x, w, t, lse, "none", 0.0)
    tiny = 2.0 ** -149 if dtype != F16 else 0.0
    most = torch.finfo(dtype).max
    for a, r, b, name in zip(got, ref, (bx, bw), ("dx", "dweight")):
        # within the bound of the largest finite value: either
        over, under = r.abs() - b > most, r.abs() + b < most
        assert torch.equal(a[over].double(), r[over].sign() * INF)
        R.within(torch.where(under, a.double(), 0.0), torch.where(under, r, 0.0), b + tiny, name)


@pytest.mark.parametrize("dtype,classes", [(F32, 70001), (BF16, 140001)], ids=str)
def test_copies_of_the_table_in_pieces(dtype, classes):
    for backward in (False, True):
        p = L.linear_cross_entropy_plan(1000, 1000, classes, dtype, backward=backward)
        assert not p["direct"] and p["piece"] < classes
    x, w, t = make(1000, 1000, classes, dtype)
    got = both(x, w, t, torch.ones((), device="cuda"), "mean")
    # 64 bits of a part of the rows at a time
    n = (t != R.IGNORED).sum()
    total = bound = 0.0
    dw = torch.zeros(classes, 1000, device="cuda", dtype=torch.float64)
    bw = torch.zeros_like(dw)
    for k in range(0, 1000, 250):
        a = x[k:k + 250], w, t[k:k + 250]
        rl, rs, bl, bs = R.forward(*a, "sum", 0.0)
        R.within(got[1][k:k + 250], rs, bs, "lse")
        total, bound = total + rl, bound + bl
        rx, rw, bx, b = R.backward(1.0 / n, *a, got[1][k:k + 250], "sum", 0.0)
        R.within(got[2][k:k + 250], rx, bx, "dx")
        dw += rw
        bw += b
    R.within(got[0], total / n, bound / n, "loss")
    R.within(got[3], dw, bw, "dweight")


@TYPES
def test_captured_and_the_same_bits(dtype):
    packed(250, dtype)
    sets = [make(ROWS, 250, CLASSES, dtype, seed=k) for k in range(3)]
    x, w, t = (a.clone() for a in sets[0])
    dl = weights()
    both(x, w, t, dl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(x, w, t, dl)
    for k in (1, 2, 1, 0):
        for a, b in zip((x, w, t), sets[k]):
            a.copy_(b)
        dl.copy_(weights())
        graph.replay()
        torch.cuda.synchronize()
        for _ in range(2):
            assert all(torch.equal(a, b) for a, b in zip(out, both(x, w, t, dl)))


# ---- small calls, to float32's accuracy -------------------------------------------------------

@pytest.mark.parametrize("size", [(17, 100, 64), (65, 128, 257), (130, 33, 1001), (5, 1000, 130),
                                  (3, 64, 20001), (2001, 40, 10)], ids=str)
def test_float32_of_small_calls(size):
    """Operands and g as they are: no value is taken as two float16."""
    rows, cols, classes = size
    for backward in (False, True):
        assert L.linear_cross_entropy_plan(*size, F32, backward=backward)["direct"]
    x, w, t = make(*size, F32)
    # values that would lose bits beside the largest
    w[:, ::3] *= 2.0 ** -22
    x[:, 1::3] *= 2.0 ** -22
    dl = weights(rows)
    loss, lse, dx, dw = both(x, w, t, dl)
    rl, rs, bl, bs = R.forward(x.double(), w.double(), t, "none", 0.0)  # bounds without a split
    R.within(lse, rs, bs, "lse")
    R.within(loss, rl, bl, "loss")
    xc, wd = R.clean(x, t), w.double()
    c = R.factors(dl, t, "none")[:, None]
    less = xc @ wd.T - lse.double()[:, None]
    p = torch.exp(less)
    y = torch.zeros_like(p).scatter_(1, t.clamp(min=0)[:, None], 1.0)
    g = c * (p - y)
    ez = R.product_bound(xc, wd.T.contiguous(), cols, False)
    eg = c.abs() * (p * (ez + 3 * R.U * less.abs() + 6 * R.U) + 2 * R.U * (p - y).abs() + 2.0 ** -126)
    dx64, dw64 = g @ wd, g.T @ xc
    R.within(dx, dx64, R.U * dx64.abs() + 2 * (eg @ wd.abs() + R.product_bound(g, wd, classes, False)),
             "dx")
    R.within(dw, dw64, R.U * dw64.abs()
             + 2 * (eg.T @ xc.abs() + R.product_bound(g.T.contiguous(), xc, rows, False)), "dweight")
