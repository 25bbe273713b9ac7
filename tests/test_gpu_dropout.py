"""Dropout on the GPU: the mask bit for bit, the values against 64 bits."""
import pytest
import torch
import torch.utils.checkpoint

import lazy_optimizer_step_amd as L
from lazy_optimizer_step_amd import _lib
from tests import loss_ref as R

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SEED = 0x0123456789ABCDEF


def draw(shape, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, device="cuda", generator=g)
    return torch.where(x.abs() < 0.01, 0.01, x).to(dtype)  # a zero would not show its mask


SHAPES = [(1,), (7,), (8,), (9,), (1, 1), (3, 5), (5, 8), (2, 64), (33, 129), (4, 1024), (2, 3, 4, 10),
          (1000, 8), (77, 501), (2048, 1030)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(shape, dtype):
    x, r = draw(shape, dtype), draw(shape, dtype, 2)
    for p, seed, offset in ((0.1, SEED, 0), (0.5, 3, 7), (0.9, (1 << 64) - 1, (1 << 64) - 2)):
        y = L.dropout_forward(x, p, seed, offset=offset)
        assert torch.equal((y != 0).cpu(), R.kept(shape, p, seed, offset))
        want, bound = R.dropout(x, p, seed, offset)
        R.within(y, want, bound, "y")
        assert torch.equal(L.dropout_backward(x, p, seed, offset=offset), y)
        want, bound = R.dropout(x, p, seed, offset, r)
        R.within(L.dropout_forward(x, p, seed, offset=offset, residual=r), want, bound, "y")


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
def test_ends_of_p(dtype):
    x, r = draw((50, 33), dtype), draw((50, 33), dtype, 2)
    assert torch.equal(L.dropout_forward(x, 0.0, SEED), x)
    assert not L.dropout_forward(x, 1.0, SEED).any()
    assert torch.equal(L.dropout_forward(x, 1.0, SEED, residual=r), r)
    assert not L.dropout_backward(x, 1.0, SEED).any()


def test_offsets_and_seeds_differ():
    x = torch.ones(1 << 16, device="cuda")
    a, b, c = (L.dropout_forward(x, 0.5, s, offset=o) != 0 for s, o in ((1, 0), (1, 1), (2, 0)))
    for u, v in ((a, b), (a, c), (b, c)):
        assert abs(float((u == v).double().mean()) - 0.5) < 6 * 0.5 / 256


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=str)
@pytest.mark.parametrize("cols", [64, 61, 5, 1])
def test_strides(dtype, cols):
    """Rows with gaps keep the mask that they have without, and what lies between them."""
    rows = 37
    x0, r0 = draw((rows, cols), dtype), draw((rows, cols), dtype, 2)
    bufs = [torch.full((rows, cols + k), 9.0, device="cuda", dtype=dtype) for k in (3, 7, 5)]
    x, r, y = (b[:, 1:1 + cols] for b in bufs)
    x.copy_(x0)
    r.copy_(r0)
    assert torch.equal(L.dropout_forward(x, 0.3, SEED), L.dropout_forward(x0, 0.3, SEED))
    want = L.dropout_forward(x0, 0.3, SEED, residual=r0)
    assert L.dropout_forward(x, 0.3, SEED, residual=r, out=y) is y
    assert torch.equal(y, want)
    for b in bufs:
        assert (b[:, :1] == 9).all() and (b[:, 1 + cols:] == 9).all()
    L.dropout_backward(x, 0.3, SEED, out=y)
    assert torch.equal(y, L.dropout_backward(x0, 0.3, SEED))
    assert (bufs[2][:, :1] == 9).all() and (bufs[2][:, 1 + cols:] == 9).all()


def test_in_place():
    for make in (lambda t: t, lambda t: t[:, 1:60]):
        x, r = make(draw((40, 64), BF16).clone()), make(draw((40, 64), BF16, 2).clone())
        want = L.dropout_forward(x, 0.4, SEED, residual=r)
        a, b = make(draw((40, 64), BF16)), make(draw((40, 64), BF16, 2))
        assert torch.equal(L.dropout_forward(a, 0.4, SEED, residual=r, out=a), want)
        assert torch.equal(L.dropout_forward(x, 0.4, SEED, residual=b, out=b), want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_dropped_values_are_not_looked_at(bad):
    x = draw((64, 100), F16)
    keep = R.kept((64, 100), 0.5, SEED).cuda()
    want = L.dropout_forward(x, 0.5, SEED)
    x[~keep] = bad
    assert torch.equal(L.dropout_forward(x, 0.5, SEED), want)
    with pytest.raises(L.SparseOptError) as err:
        L.dropout_forward(x, 0.5, SEED, validate=True)
    assert err.value.code == _lib.ENONFINITE


def test_seed_on_the_device_and_captured():
    x, r = draw((123, 77), BF16), draw((123, 77), BF16, 2)
    seed = torch.tensor([5], dtype=torch.int64, device="cuda")
    want = L.dropout_forward(x, 0.2, 5, offset=3, residual=r)
    assert torch.equal(L.dropout_forward(x, 0.2, seed, offset=3, residual=r), want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = L.dropout_forward(x, 0.2, seed, offset=3, residual=r)
        dx = L.dropout_backward(x, 0.2, seed, offset=3)
    for s in (5, -1, 1 << 40, 5):
        seed.fill_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, L.dropout_forward(x, 0.2, s, offset=3, residual=r))
        assert torch.equal(dx, L.dropout_backward(x, 0.2, s, offset=3))


def test_streams():
    x = draw((300, 200), F32)
    want = L.dropout_forward(x, 0.2, 5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        y = L.dropout_forward(x, 0.2, 5, stream=stream)
        s.synchronize()
        assert torch.equal(y, want)


def test_no_rows():
    x = torch.empty(0, 8, device="cuda")
    assert L.dropout_forward(x, 0.5, 1).shape == (0, 8)
    assert L.dropout_backward(x, 0.5, 1).shape == (0, 8)


def test_more_values_than_an_int_counts():
    n = (1 << 31) + 24
    x = torch.ones(n, device="cuda", dtype=F16)
    y = L.dropout_forward(x, 0.5, SEED, out=x)
    for first in (0, (1 << 31) - 16, n - 1000):
        keep = torch.from_numpy(R.bits16(first, 1000 if first + 1000 <= n else n - first, SEED, 0)
                                >= 32768)
        assert torch.equal((y[first:first + len(keep)] != 0).cpu(), keep)


def test_module():
    torch.manual_seed(1)
    m = L.Dropout(0.25, seed=9)
    x = draw((20, 30), F32).requires_grad_()
    r = draw((20, 30), F32, 2).requires_grad_()
    for offset in range(2):
        y = m(x, r)
        assert torch.equal(y, L.dropout_forward(x.detach(), 0.25, 9, offset=offset,
                                                residual=r.detach()))
        dy = torch.randn_like(y)
        x.grad = r.grad = None
        y.backward(dy)
        assert torch.equal(x.grad, L.dropout_backward(dy, 0.25, 9, offset=offset))
        assert torch.equal(r.grad, dy)
    again = L.Dropout(0.25, seed=9)
    again.load_state_dict(m.state_dict())
    assert torch.equal(again(x), L.dropout_forward(x.detach(), 0.25, 9, offset=2))
    m.eval()
    assert torch.equal(m(x), x) and torch.equal(m(x, r), x + r)


def test_module_keeps_the_seed_that_its_forward_read():
    seed = torch.tensor([4], dtype=torch.int64, device="cuda")
    m = L.Dropout(0.5, seed=seed)
    x = draw((50, 60), F32).requires_grad_()
    y = m(x)
    seed.fill_(99)
    y.sum().backward()
    assert torch.equal(x.grad != 0, y != 0)


def test_module_with_a_pass_that_is_run_again():
    m = L.Dropout(0.5, seed=6)
    x = draw((50, 60), F32).requires_grad_()
    m(x)
    y = torch.utils.checkpoint.checkpoint(lambda t: m(t * 2, offset=40), x, use_reentrant=False)
    assert torch.equal(y, L.dropout_forward(x.detach() * 2, 0.5, 6, offset=40))
    y.sum().backward()
    assert torch.equal(x.grad, 4.0 * (y != 0)) and m.offset == 1


def test_module_takes_any_layout():
    x = draw((40, 24), F32)
    m = L.Dropout(0.5, seed=2)
    assert torch.equal(m(x.t()), L.dropout_forward(x.t().contiguous(), 0.5, 2))


def test_refusals():
    x = draw((4, 8), F32)
    with pytest.raises(L.SparseOptError) as err:
        L.dropout_forward(x, 1.5, 1)
    assert err.value.code == _lib.EINVAL
    with pytest.raises(TypeError, match="seed must be"):
        L.dropout_forward(x, 0.5, torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError, match="one value"):
        L.dropout_forward(x, 0.5, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="residual has shape"):
        L.dropout_forward(x, 0.5, 1, residual=x[:2])
    with pytest.raises(TypeError, match="residual must be"):
        L.dropout_forward(x, 0.5, 1, residual=x.half())
    with pytest.raises(ValueError, match="not evenly spaced|adjacent"):
        L.dropout_forward(x.t(), 0.5, 1)
