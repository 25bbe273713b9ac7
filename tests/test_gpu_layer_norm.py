"""Layer norm forward and backward against their formulas in 64 bits."""
import pytest
import torch

import lazy_optimizer_step_amd as L
from tests import dense_ref as R

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16

# one column to past every width at which the kernels change, odd ones among them
SHAPES = [(1, 1), (3, 1), (5, 2), (7, 63), (4, 64), (9, 65), (33, 128), (130, 200), (3, 511),
          (6, 512), (5, 513), (17, 1001), (4, 1024), (5, 2047), (3, 2048), (3, 2056), (6, 4096),
          (3, 5003), (2, 8192), (3, 8200), (2, 16384), (3, 16385), (2, 40000), (1, 70001),
          (700, 96), (4099, 24)]


def inputs(rows, cols, dtype, wdtype, seed=0):
    g = torch.Generator().manual_seed(seed + 7 * rows + cols)
    x = (torch.randn(rows, cols, generator=g) * (1 + torch.rand(rows, 1, generator=g)) + 0.5)
    w = 1 + 0.2 * torch.randn(cols, generator=g)
    b = 0.3 * torch.randn(cols, generator=g)
    dy = torch.randn(rows, cols, generator=g)
    return (x.to(dtype).cuda(), w.to(wdtype).cuda(), b.to(wdtype).cuda(), dy.to(dtype).cuda())


def check_both(x, w, b, dy, eps=1e-5, wdtype=None, **kw):
    y, mean, rstd = L.layer_norm_forward(x, w, b, eps=eps, **kw)
    ref = R.ln_forward(x, w, b, eps)
    for got, r, e, what in zip((y, mean, rstd), ref, R.ln_forward_bounds(x, w, b, eps),
                               ("y", "mean", "rstd")):
        R.within(got, r, e, what)
    dx, dw, db = L.layer_norm_backward(dy, x, mean, rstd, w, **kw)
    assert dx.dtype == x.dtype and dw.dtype == db.dtype
    ref = R.ln_backward(dy, x, mean, rstd, w)
    for got, r, e, what in zip((dx, dw, db), ref,
                               R.ln_backward_bounds(dy, x, mean, rstd, w, dw.dtype),
                               ("dx", "dweight", "dbias")):
        R.within(got, r, e, what)
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F16), (F16, F32)],
                         ids=lambda t: "-".join(str(x)[6:] for x in t))
def test_widths_and_types(shape, types):
    check_both(*inputs(*shape, *types))


@pytest.mark.parametrize("rows,cols", [(16384, 128), (40001, 40), (2500, 1024)])
def test_many_rows(rows, cols):
    check_both(*inputs(rows, cols, BF16, F32))


@pytest.mark.parametrize("weight,bias", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("cols", [200, 1001, 20000])
def test_without_weight_or_bias(weight, bias, cols):
    x, w, b, dy = inputs(11, cols, F32, F32)
    check_both(x, w if weight else None, b if bias else None, dy)


def test_only_what_is_wanted():
    x, w, b, dy = inputs(37, 300, BF16, F32)
    _, mean, rstd = L.layer_norm_forward(x, w, b)
    full = L.layer_norm_backward(dy, x, mean, rstd, w)
    for keep in range(8):
        want = [bool(keep >> k & 1) for k in range(3)]
        got = L.layer_norm_backward(dy, x, mean, rstd, w, want_dx=want[0], want_dweight=want[1],
                                    want_dbias=want[2])
        for g, f, k in zip(got, full, want):
            assert (g is None) != k
            assert g is None or torch.equal(g, f)


def test_no_rows():
    x = torch.empty(0, 40, device="cuda")
    w = torch.ones(40, device="cuda")
    y, mean, rstd = L.layer_norm_forward(x, w)
    assert y.shape == (0, 40) and mean.shape == (0,) and rstd.shape == (0,)
    dw, db = torch.full((40,), 7.0, device="cuda"), torch.full((40,), 7.0, device="cuda")
    dx, _, _ = L.layer_norm_backward(x, x, mean, rstd, w, dweight=dw, dbias=db)
    assert dx.shape == (0, 40)
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,stride,offset", [(128, 384, 128), (128, 131, 0), (128, 136, 3),
                                                (1000, 1001, 1), (4096, 4104, 8)])
def test_rows_of_a_larger_array(dtype, cols, stride, offset):
    """Row strides and bases that 16-byte accesses take, and some that they do not."""
    rows = 19
    big = torch.randn(rows, stride, device="cuda").to(dtype)
    flat = torch.cat([big.flatten(), torch.zeros(64, dtype=dtype, device="cuda")])
    x = flat.as_strided((rows, cols), (stride, 1), offset)
    _, w, b, dy = inputs(rows, cols, dtype, F32)
    check_both(x, w, b, dy)
    check_both(x, w, b, x)
    # a strided output leaves what lies between its rows alone
    room = torch.full_like(flat, 3.0)
    out = room.as_strided((rows, cols), (stride, 1), offset)
    y, mean, rstd = L.layer_norm_forward(x, w, b, out=out)
    plain, _, _ = L.layer_norm_forward(x.contiguous(), w, b)
    # widths of accesses change the order of the sums: the same values within their bounds
    R.within(y, R.ln_forward(x, w, b, 1e-5)[0], R.ln_forward_bounds(x, w, b, 1e-5)[0], "y")
    R.within(plain, R.ln_forward(x, w, b, 1e-5)[0], R.ln_forward_bounds(x, w, b, 1e-5)[0], "y")
    out.fill_(3.0)
    assert (room == 3.0).all()


@pytest.mark.parametrize("cols", [128, 1001, 4096, 20000])
def test_in_place(cols):
    x, w, b, dy = inputs(23, cols, BF16, F32)
    y, mean, rstd = L.layer_norm_forward(x, w, b)
    grads = L.layer_norm_backward(dy, x, mean, rstd, w)
    x2 = x.clone()
    y2, _, _ = L.layer_norm_forward(x2, w, b, out=x2)
    assert y2 is x2 and torch.equal(y2, y)
    for over in ("dy", "x"):
        d2, x2 = dy.clone(), x.clone()
        out = d2 if over == "dy" else x2
        got = L.layer_norm_backward(d2, x2, mean, rstd, w, out=out)
        for g, f in zip(got, grads):
            assert torch.equal(g, f)


def test_leading_axes():
    x, w, b, dy = inputs(24, 96, F32, F32)
    y, mean, rstd = L.layer_norm_forward(x.view(2, 3, 4, 96), w, b)
    assert y.shape == (2, 3, 4, 96) and mean.shape == (2, 3, 4)
    assert torch.equal(y.view(24, 96), L.layer_norm_forward(x, w, b)[0])
    dx, dw, db = L.layer_norm_backward(dy.view(2, 3, 4, 96), x.view(2, 3, 4, 96), mean, rstd, w)
    for g, f in zip((dx.view(24, 96), dw, db),
                    L.layer_norm_backward(dy, x, mean.view(-1), rstd.view(-1), w)):
        assert torch.equal(g, f)


@pytest.mark.parametrize("cols", [64, 1001, 4096, 20000])
def test_special_values(cols):
    """A row's NaN or infinity stays in that row; constant rows give the bias; a far mean keeps
    its digits."""
    x, w, b, dy = inputs(12, cols, F32, F32)
    clean, cm, cr = L.layer_norm_forward(x, w, b)
    x2 = x.clone()
    x2[3, cols // 2] = float("nan")
    x2[7, cols - 1] = float("inf")
    x2[9, 0] = float("-inf")
    x2[10] = 2.5
    y, mean, rstd = L.layer_norm_forward(x2, w, b)
    for k in (3, 7, 9):
        assert y[k].isnan().all()
    assert torch.equal(y[10], b)
    rest = [0, 1, 2, 4, 5, 6, 8, 11]
    assert torch.equal(y[rest], clean[rest])
    dx, _, _ = L.layer_norm_backward(dy, x2, mean, rstd, w)
    assert torch.equal(dx[rest], L.layer_norm_backward(dy, x, cm, cr, w)[0][rest])
    check_both(x + 1000.0, w, b, dy)


@pytest.mark.parametrize("cols", [100, 2999, 20000])
def test_repeats_and_streams(cols):
    x, w, b, dy = inputs(301, cols, BF16, BF16)
    first = check_both(x, w, b, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = L.layer_norm_forward(x, w, b, stream=s)
    grads = L.layer_norm_backward(dy, x, mean, rstd, w, stream=s)
    s.synchronize()
    for g, f in zip((y, mean, rstd, *grads), first):
        assert torch.equal(g, f)


def test_graph():
    x, w, b, dy = inputs(500, 256, BF16, F32)
    ws = torch.empty(L.layer_norm_backward_workspace_size(500, 256), dtype=torch.uint8,
                     device="cuda")
    y, mean, rstd = L.layer_norm_forward(x, w, b)
    dx, dw, db = L.layer_norm_backward(dy, x, mean, rstd, w, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.layer_norm_forward(x, w, b, out=y, mean=mean, rstd=rstd)
        L.layer_norm_backward(dy, x, mean, rstd, w, out=dx, dweight=dw, dbias=db, workspace=ws)
    for k in range(4):
        x.copy_(torch.randn(500, 256, device="cuda") + k)
        dy.copy_(torch.randn(500, 256, device="cuda"))
        want = L.layer_norm_forward(x, w, b)
        want = (*want, *L.layer_norm_backward(dy, x, want[1], want[2], w))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for got, f in zip((y, mean, rstd, dx, dw, db), want):
            assert torch.equal(got, f)


def test_offsets_beyond_32_bits():
    cols = 96
    rows = (1 << 31) // cols + 1000
    x = torch.empty(rows, cols, dtype=BF16, device="cuda").normal_()
    w = torch.ones(cols, device="cuda")
    y, mean, rstd = L.layer_norm_forward(x, w)
    for at in (slice(0, 50), slice(rows - 50, rows)):
        R.within(y[at], R.ln_forward(x[at], w, None, 1e-5)[0],
                 R.ln_forward_bounds(x[at], w, None, 1e-5)[0], "y")
    dx, dw, db = L.layer_norm_backward(y, x, mean, rstd, w)
    for at in (slice(0, 50), slice(rows - 50, rows)):
        args = (y[at], x[at], mean[at], rstd[at], w)
        R.within(dx[at], R.ln_backward(*args)[0], R.ln_backward_bounds(*args, F32)[0], "dx")
    # dweight = sum of y * xhat is near rows (the mean square of xhat is 1 - eps / var)
    assert (dw.double() / rows - 1).abs().max() < 5e-3


def test_difference_quotient():
    """<dx, v> against (loss(x + h v) - loss(x - h v)) / 2h of the forward kernel."""
    x, w, b, dy = inputs(8, 160, F32, F32)
    v = torch.randn(8, 160, device="cuda")
    h = 2.0 ** -6
    _, mean, rstd = L.layer_norm_forward(x, w, b)
    dx, dw, db = L.layer_norm_backward(dy, x, mean, rstd, w)

    def loss(y):
        return (R.d(y) * R.d(dy)).sum()
    hi, lo = x + h * v, x - h * v
    step = R.d(hi) - R.d(lo)                        # what the float32 inputs moved by
    kernel = loss(L.layer_norm_forward(hi, w, b)[0]) - loss(L.layer_norm_forward(lo, w, b)[0])
    formula = loss(R.ln_forward(hi, w, b, 1e-5)[0]) - loss(R.ln_forward(lo, w, b, 1e-5)[0])
    rounding = sum((R.ln_forward_bounds(t, w, b, 1e-5)[0] * R.d(dy).abs()).sum() for t in (hi, lo))
    assert abs(kernel - formula) <= rounding
    # the third-order term: halving h takes the quotient's distance to the slope down by four
    slope = (R.d(dx) * step).sum() / (2 * h)
    q1 = formula / (2 * h)
    f2 = loss(R.ln_forward(R.d(x) + h / 2 * R.d(v), w, b, 1e-5)[0]) - \
        loss(R.ln_forward(R.d(x) - h / 2 * R.d(v), w, b, 1e-5)[0])
    truncation = 4.0 / 3.0 * abs(q1 - f2 / h)
    e_dx = (R.ln_backward_bounds(dy, x, mean, rstd, w, F32)[0] * R.d(v).abs()).sum()
    assert abs(kernel / (2 * h) - slope) <= 2 * truncation + rounding / (2 * h) + e_dx
    # y is linear in weight and bias
    _, rw, rb = R.ln_backward(dy, x, mean, rstd, w)
    _, ew, eb = R.ln_backward_bounds(dy, x, mean, rstd, w, F32)
    R.within(dw, rw, ew, "dweight")
    R.within(db, rb, eb, "dbias")


@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, F32), (BF16, BF16)])
def test_module(dtype, wdtype):
    ln = L.LayerNorm(96, dtype=wdtype)
    x, w, b, dy = inputs(40, 96, dtype, wdtype)
    with torch.no_grad():
        ln.weight.copy_(w)
        ln.bias.copy_(b)
    xin = x.view(5, 8, 96).clone().requires_grad_()
    y = ln(xin.transpose(0, 1))                     # rows that do not collapse
    y.backward(dy.view(5, 8, 96).transpose(0, 1))
    _, mean, rstd = L.layer_norm_forward(x, w, b)
    ref = R.ln_backward(dy, x, mean, rstd, w)
    e = R.ln_backward_bounds(dy, x, mean, rstd, w, wdtype)
    R.within(xin.grad.view(40, 96), ref[0], e[0], "dx")
    R.within(ln.weight.grad, ref[1], e[1], "dweight")
    R.within(ln.bias.grad, ref[2], e[2], "dbias")
    frozen = L.LayerNorm(96, weight=False, bias=False)
    xin = x.clone().requires_grad_()
    frozen(xin).backward(dy)
    args = (dy, x, mean, rstd, None)
    R.within(xin.grad, R.ln_backward(*args)[0], R.ln_backward_bounds(*args, F32)[0], "dx")


def test_validate_refuses_and_writes_nothing():
    x, w, b, dy = inputs(9, 70, F32, F32)
    y, mean, rstd = L.layer_norm_forward(x, w, b, validate=True)
    bad = x.clone()
    bad[8, 69] = float("inf")
    keep = torch.full_like(y, 5.0)
    with pytest.raises(L.SparseOptError) as e:
        L.layer_norm_forward(bad, w, b, out=keep, validate=True)
    assert e.value.code == -5
    for a, c in ((bad, x), (dy, bad)):
        with pytest.raises(L.SparseOptError) as e:
            L.layer_norm_backward(a, c, mean, rstd, w, out=keep, validate=True)
        assert e.value.code == -5
    torch.cuda.synchronize()
    assert (keep == 5.0).all()


def test_python_refusals():
    x, w, b, dy = inputs(6, 32, F32, F32)
    with pytest.raises(TypeError):
        L.layer_norm_forward(x.double(), w, b)
    with pytest.raises(TypeError):
        L.layer_norm_forward(x, w.half(), b.half())
    with pytest.raises(TypeError):
        L.layer_norm_forward(x.half(), w.half(), b)
    with pytest.raises(ValueError):
        L.layer_norm_forward(x, w[:31], b)
    with pytest.raises(ValueError):
        L.layer_norm_forward(x.t(), None, None)
    with pytest.raises(ValueError):
        L.layer_norm_forward(x[:1].expand(6, 32), w, b)
    with pytest.raises(ValueError):
        L.layer_norm_forward(x.cpu(), w, b)
    with pytest.raises(L.SparseOptError):
        L.layer_norm_forward(x, w, b, eps=0.0)
    _, mean, rstd = L.layer_norm_forward(x, w, b)
    with pytest.raises(ValueError):
        L.layer_norm_backward(dy[:5], x, mean, rstd, w)
    with pytest.raises(TypeError):
        L.layer_norm_backward(dy.half(), x, mean, rstd, w)
    with pytest.raises(ValueError):
        L.layer_norm_backward(dy, x, mean[:5], rstd, w)
    with pytest.raises(L.SparseOptError):
        L.layer_norm_backward(dy, x, mean, rstd, w,
                              workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
