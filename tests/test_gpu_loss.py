"""The loss over a table of classes on the GPU against its formula in 64 bits."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from lazy_optimizer_step_amd import _lib
from tests import loss_ref as R

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


def make(rows, cols, classes, dtype, seed=0, ignored=0.2, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows + 7 * cols + 13 * classes)
    w = torch.randn(classes, cols, device="cuda", generator=g) * (scale / cols ** 0.5)
    t = torch.randint(classes, (rows,), device="cuda", generator=g)
    x = torch.randn(rows, cols, device="cuda", generator=g) + w[t]
    t[torch.rand(rows, device="cuda", generator=g) < ignored] = R.IGNORED
    return x.to(dtype), w.to(dtype), t


def check(x, w, t, reduction="mean", e=0.0, want_dx=True, want_dw=True, **kw):
    """Both passes against 64 bits; returns what they gave."""
    loss, lse = L.linear_cross_entropy_forward(x, w, t, reduction=reduction, label_smoothing=e, **kw)
    rl, rs, bl, bs = R.forward(x, w, t, reduction, e)
    R.within(lse, rs, bs, "lse")
    R.within(loss, rl, bl, "loss")
    n = len(t)
    dl = torch.rand(n, device="cuda") - 0.3 if reduction == "none" else torch.tensor(0.7, device="cuda")
    dx, dw = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction=reduction,
                                             label_smoothing=e, want_dx=want_dx,
                                             want_dweight=want_dw, **kw)
    rx, rw, bx, bw = R.backward(dl, x, w, t, lse, reduction, e)
    if want_dx:
        R.within(dx, rx, bx, "dx")
    if want_dw:
        R.within(dw, rw, bw, "dweight")
    return loss, lse, dx, dw


SIZES = [(1, 1, 1), (1, 16, 2), (3, 7, 5), (2, 64, 63), (17, 100, 64), (64, 64, 65), (65, 128, 257),
         (130, 33, 1001), (200, 192, 300), (5, 1000, 130), (257, 65, 70)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_small(size, dtype):
    for k, reduction in enumerate(("mean", "sum", "none")):
        check(*make(*size, dtype, seed=k), reduction, 0.1 * (k % 2))


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_one_row_of_many_classes(dtype):
    """The inner axis of dx cut into parts."""
    check(*make(1, 128, 20001, dtype, ignored=0))
    check(*make(65, 72, 20001, dtype), "none", 0.1)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("steps", [13, 17, 20, 25, 31, 33, 47])
def test_cut_axes_of_any_length(dtype, steps):
    """Inner axes of a number of steps that no power of two divides, cut for either gradient."""
    k = steps * (32 if dtype == F32 else 64) - 5
    check(*make(4, 64, k, dtype), "none")
    check(*make(k, 64, 4, dtype), "none")


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_many_rows_of_few_classes(dtype):
    """The inner axis of dweight cut into parts."""
    check(*make(20001, 40, 10, dtype), "mean", 0.1)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_large_tiles(dtype):
    check(*make(2050, 576, 8200, dtype))


@pytest.mark.parametrize("dtype,cols", [(BF16, 4000), (F16, 4000), (BF16, 4096)], ids=str)
def test_largest_tiles(dtype, cols):
    """Sizes that fill the card with the largest tiles in all three products; rows that are
    copied (in two pieces in the forward pass) and rows that are read in place."""
    check(*make(3990, cols, 33003, dtype))


def test_more_values_than_an_int_counts():
    """A table of more than 2^31 values: its last rows."""
    rows, cols, classes, last = 3, 2048, 1_100_000, 500
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, device="cuda", generator=g).to(BF16)
    w = torch.empty(classes, cols, device="cuda", dtype=BF16)
    for part in w.split(100_000):
        part.copy_(torch.randn(part.shape, device="cuda", generator=g) / 32)
    t = torch.tensor([classes - 1, 5, classes - 7], device="cuda")
    loss, lse = L.linear_cross_entropy_forward(x, w, t, reduction="none")
    xd, z, ez = x.double(), [], []
    for part in w.split(100_000):
        z.append(xd @ part.double().T)
        ez.append(R.product_bound(xd, part.double().T.contiguous(), cols, False))
    z, ez = torch.cat(z, 1), torch.cat(ez, 1)
    want = torch.logsumexp(z, 1)
    p = torch.exp(z - want[:, None])
    bound = (p * (ez + 3 * R.U * (z.max() - z))).sum(1) + 100 * R.U + R.U * want.abs()
    R.within(lse, want, 2 * bound, "lse")
    at = t[:, None]
    R.within(loss, want - z.gather(1, at)[:, 0],
             2 * (bound + ez.gather(1, at)[:, 0] + R.U * want.abs()), "loss")
    dl = torch.ones(rows, device="cuda")
    dx, dw = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none")
    # the last rows' gradients, as of a table of their own under the same lse
    own = t - (classes - last)
    own[own < 0] = R.IGNORED
    p = torch.exp(z[:, -last:] - lse.double()[:, None])
    eg = p * (ez[:, -last:] + 3 * R.U * (z[:, -last:] - lse.double()[:, None]).abs() + 8 * R.U)
    for i in range(rows):
        if own[i] >= 0:
            p[i, own[i]] -= 1
    eg = eg + (2.0 ** -8 + 8 * R.U) * p.abs()
    ref = p.T @ xd
    R.within(dw[-last:], ref, 2.0 ** -8 * ref.abs() + 2 * eg.T @ xd.abs(), "dweight")
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_pieces_backward(dtype):
    """g of all classes at once would pass the workspace's share: pieces, the last one short."""
    check(*make(66000, 24, 9000 if dtype == BF16 else 4500, dtype))


def test_pieces_forward():
    """Copies of the table in pieces."""
    check(*make(5, 1000, 70001, F32, ignored=0), want_dw=False)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_only_what_is_wanted(dtype):
    a = make(33, 48, 500, dtype)
    *_, dx, dw = check(*a)
    *_, dx1, none = check(*a, want_dw=False)
    assert none is None and torch.equal(dx, dx1)
    *_, none, dw1 = check(*a, want_dx=False)
    assert none is None and torch.equal(dw, dw1)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("bad", [NAN, INF, -INF, 1e30])
def test_ignored_rows_may_hold_anything(dtype, bad):
    x, w, t = make(70, 80, 300, dtype, ignored=0.3)
    plain = check(x, w, t, "none", 0.1)
    x[t == R.IGNORED] = bad
    got = check(x, w, t, "none", 0.1)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    L.linear_cross_entropy_forward(x, w, t, validate=True)
    gone = t == R.IGNORED
    assert not got[0][gone].any() and not got[1][gone].any() and not got[2][gone].any()


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_no_row_counts(reduction):
    x, w, t = make(40, 64, 100, BF16)
    t.fill_(R.IGNORED)
    x.fill_(NAN)
    loss, lse, dx, dw = check(x, w, t, reduction)
    assert not loss.any() and not lse.any() and not dx.any() and not dw.any()


def test_another_ignore_index():
    x, w, t = make(40, 64, 100, F32, ignored=0.0)
    t[::3] = 7
    want = t.clone()
    want[::3] = R.IGNORED
    a = L.linear_cross_entropy_forward(x, w, t, ignore_index=7)
    b = L.linear_cross_entropy_forward(x, w, want)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dl = torch.ones((), device="cuda")
    ga = L.linear_cross_entropy_backward(dl, x, w, t, a[1], ignore_index=7)
    gb = L.linear_cross_entropy_backward(dl, x, w, want, b[1])
    assert torch.equal(ga[0], gb[0]) and torch.equal(ga[1], gb[1])


@pytest.mark.parametrize("dtype", [F32, F16], ids=str)
@pytest.mark.parametrize("target", [100, -1, -(1 << 62), (1 << 62)])
def test_target_outside_the_classes(dtype, target):
    x, w, t = make(20, 64, 100, dtype, ignored=0.0)
    good, lse0 = L.linear_cross_entropy_forward(x, w, t, reduction="none")
    t[4] = target
    loss, lse = L.linear_cross_entropy_forward(x, w, t, reduction="none")
    assert torch.isnan(loss[4]) and torch.isfinite(lse).all()
    keep = torch.arange(20, device="cuda") != 4
    assert torch.equal(loss[keep], good[keep]) and torch.equal(lse, lse0)
    dl = torch.ones(20, device="cuda")
    dx, dw = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none")
    assert torch.isnan(dx[4]).all() and torch.isfinite(dx[keep]).all() and torch.isnan(dw).all()
    for call in (lambda: L.linear_cross_entropy_forward(x, w, t, validate=True),
                 lambda: L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none",
                                                         validate=True)):
        with pytest.raises(L.SparseOptError) as err:
            call()
        assert err.value.code == _lib.ERANGE


@pytest.mark.parametrize("where", ["x", "weight"])
def test_validation_finds_non_finite(where):
    x, w, t = make(20, 70, 100, BF16, ignored=0.0)
    (x if where == "x" else w)[3, 69] = NAN
    out = torch.full((), 5.0, device="cuda")
    with pytest.raises(L.SparseOptError) as err:
        L.linear_cross_entropy_forward(x, w, t, out=out, validate=True)
    assert err.value.code == _lib.ENONFINITE and float(out) == 5.0


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_a_row_of_nan_stays_alone(dtype):
    x, w, t = make(20, 64, 100, dtype, ignored=0.0)
    good, _ = L.linear_cross_entropy_forward(x, w, t, reduction="none")
    x[4, 5] = NAN
    loss, lse = L.linear_cross_entropy_forward(x, w, t, reduction="none")
    keep = torch.arange(20, device="cuda") != 4
    assert torch.isnan(loss[4]) and torch.isnan(lse[4]) and torch.equal(loss[keep], good[keep])


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_one_class(dtype):
    """A single class: the loss is zero, and so are the gradients."""
    x, w, t = make(9, 20, 1, dtype, ignored=0.0)
    loss, lse, dx, dw = check(x, w, t, "none")
    assert not loss.any()
    assert float(dx.abs().max()) < 1e-6


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("cols", [64, 61])
def test_strides(dtype, cols):
    """Rows with gaps, at odd distances, from unaligned addresses; gaps of the outputs keep what
    they hold."""
    rows, classes = 37, 131
    x0, w0, t = make(rows, cols, classes, dtype)
    pad, first = 3, 1
    xb = torch.full((rows, cols + pad), 9.0, device="cuda", dtype=dtype)
    wb = torch.full((classes, cols + pad), 9.0, device="cuda", dtype=dtype)
    x, w = xb[:, first:first + cols], wb[:, first:first + cols]
    x.copy_(x0)
    w.copy_(w0)
    a = L.linear_cross_entropy_forward(x, w, t)
    b = L.linear_cross_entropy_forward(x0, w0, t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dxb, dwb = torch.full_like(xb, 7.0), torch.full_like(wb, 7.0)
    dl = torch.ones((), device="cuda")
    dx, dw = L.linear_cross_entropy_backward(dl, x, w, t, a[1], out=dxb[:, first:first + cols],
                                             dweight=dwb[:, first:first + cols])
    rx, rw = L.linear_cross_entropy_backward(dl, x0, w0, t, b[1])
    assert torch.equal(dx, rx) and torch.equal(dw, rw)
    for buf in (dxb, dwb):
        assert (buf[:, :first] == 7).all() and (buf[:, first + cols:] == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_more_than_two_axes_and_no_rows(dtype):
    x, w, t = make(24, 40, 90, dtype)
    a = L.linear_cross_entropy_forward(x, w, t, reduction="none")
    b = L.linear_cross_entropy_forward(x.view(2, 3, 4, 40), w, t.view(2, 3, 4), reduction="none")
    assert b[0].shape == (2, 3, 4) and torch.equal(a[0], b[0].view(-1))
    one = L.linear_cross_entropy_forward(x[0], w, t[0])
    assert one[0].shape == () and one[1].shape == ()
    no, not_ = x[:0], t[:0]
    for reduction in ("none", "sum", "mean"):
        out = torch.full((0,) if reduction == "none" else (), 5.0, device="cuda")
        loss, lse = L.linear_cross_entropy_forward(no, w, not_, reduction=reduction, out=out)
        assert lse.shape == (0,) and not loss.any()
        dl = torch.ones_like(loss)
        dx, dw = L.linear_cross_entropy_backward(dl, no, w, not_, lse, reduction=reduction)
        assert dx.shape == (0, 40) and not dw.any()


def test_range_of_float32():
    """Powers of two in front of the operands cancel; what does not fit beside the largest value
    is small beside it."""
    x, w, t = make(50, 64, 200, F32, ignored=0.0)
    for a, b in ((2.0 ** 60, 2.0 ** -60), (2.0 ** -100, 2.0 ** 100), (2.0 ** -126, 2.0 ** 120)):
        check(x * a, w * b, t, "none")
    w[7] = w[7] * 2.0 ** 10
    check(x * 2.0 ** -10, w, t, "none")
    check(torch.zeros_like(x), torch.zeros_like(w), t, "none")


@pytest.mark.parametrize("dtype", [BF16, F16], ids=str)
def test_large_logits(dtype):
    """Logits of thousands: all but one of the exponentials vanish."""
    x, w, t = make(50, 64, 200, dtype, ignored=0.1)
    check(x * 64, w * 64, t, "none")
    check(x * 64, w * 64, t, "mean", 0.1)


@pytest.mark.parametrize("factor", [0.0, 1e-30, 1e30, -2.0])
@pytest.mark.parametrize("dtype", [F32, F16], ids=str)
def test_factors_of_any_size(dtype, factor):
    x, w, t = make(30, 64, 150, dtype)
    _, lse = L.linear_cross_entropy_forward(x, w, t)
    # an output that its type cannot hold says nothing
    dl = torch.full((30,), factor, device="cuda")
    dl[::5] *= 2.0 ** -12
    dx, dw = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none")
    if dtype == F16 and factor == 1e30:
        return
    rx, rw, bx, bw = R.backward(dl, x, w, t, lse, "none", 0.0)
    tiny = 2.0 ** -149 if dtype == F32 else 0.0
    R.within(dx, rx, bx + tiny, "dx")
    R.within(dw, rw, bw + tiny, "dweight")


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_the_same_bits_every_run(dtype):
    x, w, t = make(300, 100, 3001, dtype)
    dl = torch.ones((), device="cuda")
    first = None
    for _ in range(3):
        loss, lse = L.linear_cross_entropy_forward(x, w, t)
        dx, dw = L.linear_cross_entropy_backward(dl, x, w, t, lse)
        now = [loss, lse, dx, dw]
        if first:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = first or now


def test_streams_and_given_outputs():
    x, w, t = make(129, 96, 777, BF16)
    loss0, lse0 = L.linear_cross_entropy_forward(x, w, t)
    dl = torch.ones((), device="cuda")
    dx0, dw0 = L.linear_cross_entropy_backward(dl, x, w, t, lse0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    loss, lse = torch.empty((), device="cuda"), torch.empty(129, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    size = L.linear_cross_entropy_workspace_size
    ws = [torch.full((size(129, 96, 777, BF16, backward=b),), 255, dtype=torch.uint8, device="cuda")
          for b in (False, True)]
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        got = L.linear_cross_entropy_forward(x, w, t, out=loss, lse=lse, workspace=ws[0], stream=stream)
        assert got[0] is loss and got[1] is lse
        got = L.linear_cross_entropy_backward(dl, x, w, t, lse, out=dx, dweight=dw, workspace=ws[1],
                                              stream=stream)
        assert got[0] is dx and got[1] is dw
        s.synchronize()
        assert torch.equal(loss, loss0) and torch.equal(lse, lse0)
        assert torch.equal(dx, dx0) and torch.equal(dw, dw0)


def test_two_streams_at_once():
    sets = [make(200, 128, 5000, BF16, seed=k) for k in range(2)]
    want = [check(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    dl = torch.tensor(0.7, device="cuda")
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for a, s in zip(sets, streams):
            loss, lse = L.linear_cross_entropy_forward(*a, stream=s)
            got.append((loss, lse, *L.linear_cross_entropy_backward(dl, *a, lse, stream=s)))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("size", [(8, 128, 1001), (300, 100, 3001), (1500, 520, 9001),
                                  (3990, 2048, 33003)], ids=str)
def test_captured(size, dtype):
    x, w, t = make(*size, dtype)
    dl = torch.tensor(0.7, device="cuda")

    def both():
        loss, lse = L.linear_cross_entropy_forward(x, w, t)
        return [loss, lse, *L.linear_cross_entropy_backward(dl, x, w, t, lse)]
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for k in range(3):
        nx, nw, nt = make(*size, dtype, seed=10 + k)
        x.copy_(nx)
        w.copy_(nw)
        t.copy_(nt)
        dl.fill_(0.5 + k)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, both()))


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_module_gradients(reduction):
    torch.manual_seed(5)
    m = L.LinearCrossEntropy(48, 200, reduction=reduction, label_smoothing=0.1)
    x = torch.randn(6, 7, 48, device="cuda", requires_grad=True)
    t = torch.randint(200, (6, 7), device="cuda")
    t[2, 3:] = -100
    loss = m(x, t)
    lse = L.linear_cross_entropy_forward(x.detach(), m.weight.detach(), t)[1]
    # a gradient of one value expanded over the rows
    (loss.sum() if reduction == "none" else loss).backward()
    dl = torch.ones(42 if reduction == "none" else (), device="cuda")
    dx, dw, bx, bw = R.backward(dl, x.detach().view(42, 48), m.weight.detach(), t.view(42),
                                lse.view(42), reduction, 0.1)
    R.within(x.grad.view(42, 48), dx, bx, "dx")
    R.within(m.weight.grad, dw, bw, "dweight")


def test_module_takes_any_layout_and_a_shared_table():
    table = torch.nn.Parameter(torch.randn(90, 32, device="cuda"))
    m = L.LinearCrossEntropy(32, 90, weight=table, reduction="sum")
    assert m.weight is table
    x = torch.randn(32, 11, device="cuda")
    t = torch.randint(90, (22,), device="cuda")[::2]
    a = m(x.t(), t)
    b = L.linear_cross_entropy_forward(x.t().contiguous(), table.detach(), t.contiguous(),
                                       reduction="sum")[0]
    assert torch.equal(a.detach(), b)


def test_gradient_against_differences():
    """The kernels' loss, moved by a step along a direction, against the kernels' gradient."""
    x, w, t = make(40, 64, 300, F32)
    loss, lse = L.linear_cross_entropy_forward(x, w, t, reduction="none")
    dl = torch.rand(40, device="cuda")
    dx, dw = L.linear_cross_entropy_backward(dl, x, w, t, lse, reduction="none")
    ax, aw = torch.randn_like(x), torch.randn_like(w) / 8
    h = 2.0 ** -7
    out, bound = [], 0.0
    for s in (h, -h):
        a, b = x + s * ax, w + s * aw
        got = L.linear_cross_entropy_forward(a, b, t, reduction="none")[0].double()
        out.append((got * dl).sum())
        bound += float((R.forward(a, b, t, "none", 0.0)[2] * dl).sum())
    slope = float((out[0] - out[1]) / (2 * h))
    want = float((dx.double() * ax).sum() + (dw.double() * aw).sum())
    # what the difference itself leaves out, from the formula in 64 bits
    f = [float((R.forward(x.double() + s * ax, w.double() + s * aw, t, "none", 0.0)[0] * dl).sum())
         for s in (h, -h)]
    third = abs((f[0] - f[1]) / (2 * h) - want)
    assert third < 0.02 * abs(want) + 0.05
    assert abs(slope - want) <= bound / (2 * h) + third + 1e-4 * abs(want)


def test_refusals():
    x, w, t = make(8, 16, 20, F32)
    f = L.linear_cross_entropy_forward
    with pytest.raises(TypeError, match="weight must be"):
        f(x, w.half(), t)
    with pytest.raises(ValueError, match="weight must be"):
        f(x, w[:, :8], t)
    with pytest.raises(TypeError, match="targets must be"):
        f(x, w, t.int())
    with pytest.raises(ValueError, match="targets has shape"):
        f(x, w, t[:4])
    with pytest.raises(ValueError, match="reduction"):
        f(x, w, t, reduction="average")
    with pytest.raises(ValueError, match="out must hold 1 values"):
        f(x, w, t, out=torch.empty(8, device="cuda"))
    with pytest.raises(L.SparseOptError) as err:
        f(x, w, t, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert err.value.code == _lib.EWORKSPACE
    _, lse = f(x, w, t)
    with pytest.raises(ValueError, match="dloss must hold 8 values"):
        L.linear_cross_entropy_backward(torch.ones((), device="cuda"), x, w, t, lse, reduction="none")
    with pytest.raises(ValueError, match="dweight has shape"):
        L.linear_cross_entropy_backward(torch.ones((), device="cuda"), x, w, t, lse,
                                        dweight=torch.empty(19, 16, device="cuda"))


def test_another_current_device(monkeypatch):
    x, w, t = make(8, 16, 20, F32)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        L.linear_cross_entropy_forward(x, w, t)
    with pytest.raises(ValueError, match="current device"):
        L.dropout_forward(x, 0.5, 1)


def test_workspace_of_another_device():
    """A tensor that says it lies on the next device stands in for one that does."""
    class Elsewhere(torch.Tensor):
        device = torch.device("cuda", 1)

    x, w, t = make(8, 16, 20, F32)
    space = torch.empty(1 << 20, dtype=torch.uint8, device="cuda").as_subclass(Elsewhere)
    loss, lse = L.linear_cross_entropy_forward(x, w, t)
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        L.linear_cross_entropy_forward(x, w, t, workspace=space)
    with pytest.raises(ValueError, match="workspace is on cuda:1"):
        L.linear_cross_entropy_backward(loss, x, w, t, lse, workspace=space)
