"""Checks of the dense operators that need no GPU: refusals of the C ABI before any device work,
workspace sizes, and the formulas of the 64-bit forms."""
import ctypes as C

import pytest
import torch

import lazy_optimizer_step_amd as L
from lazy_optimizer_step_amd import _lib
from tests import dense_ref as R

FAKE = 256  # a non-NULL address that is never dereferenced
NAN, INF = float("nan"), float("inf")


def ln_fwd(x=FAKE, xs=8, rows=4, cols=8, dt=0, w=FAKE, b=FAKE, wdt=0, eps=1e-5, y=FAKE, ys=8):
    return _lib.lib().layer_norm_forward(x, xs, rows, cols, dt, w, b, wdt, eps, y, ys, FAKE, FAKE,
                                         None, 0)


@pytest.mark.parametrize("kw", [
    {"x": None}, {"y": None}, {"rows": -1}, {"cols": 0}, {"dt": 3}, {"dt": -1}, {"wdt": 1},
    {"dt": 1, "wdt": 2}, {"eps": 0.0}, {"eps": NAN}, {"eps": INF}, {"eps": -1.0}, {"xs": 7},
    {"ys": 7}, {"rows": 1 << 40, "cols": 1 << 40}], ids=str)
def test_layer_norm_forward_refuses(kw):
    assert ln_fwd(**kw) == _lib.EINVAL
    assert b"layer_norm_forward" in _lib.lib().sparse_opt_last_error()


def test_layer_norm_no_rows_needs_no_arrays():
    assert ln_fwd(rows=0, x=None, y=None) == 0


def ln_bwd(dy=FAKE, ds=8, x=FAKE, xs=8, rows=4, cols=8, dt=0, mean=FAKE, rstd=FAKE, wdt=0,
           dx=FAKE, os=8, dw=FAKE, db=FAKE, ws=FAKE, wsb=1 << 20):
    return _lib.lib().layer_norm_backward(dy, ds, x, xs, rows, cols, dt, mean, rstd, FAKE, wdt, dx,
                                          os, dw, db, ws, wsb, None, 0)


@pytest.mark.parametrize("kw,code", [
    ({"dy": None}, "EINVAL"), ({"x": None}, "EINVAL"), ({"mean": None}, "EINVAL"),
    ({"rstd": None}, "EINVAL"), ({"rows": -1}, "EINVAL"), ({"cols": 0}, "EINVAL"),
    ({"dt": 5}, "EINVAL"), ({"wdt": 2}, "EINVAL"), ({"ds": 3}, "EINVAL"), ({"os": 7}, "EINVAL"),
    ({"ws": None}, "EWORKSPACE"), ({"wsb": 32}, "EWORKSPACE"), ({"ws": 260}, "EWORKSPACE")],
    ids=str)
def test_layer_norm_backward_refuses(kw, code):
    assert ln_bwd(**kw) == getattr(_lib, code)
    assert b"layer_norm_backward" in _lib.lib().sparse_opt_last_error()


def test_workspace_sizes():
    assert L.layer_norm_backward_workspace_size(1000, 128) >= 2 * 128 * 4
    assert L.layer_norm_backward_workspace_size(0, 1) > 0
    one = L.newton_schulz_workspace_size(1, 200, 300)
    assert one >= 200 * 300 * 4
    assert L.newton_schulz_workspace_size(1, 300, 200) == one
    assert L.newton_schulz_workspace_size(8, 200, 300) > one
    assert L.newton_schulz_workspace_size(0, 2, 3) >= 0
    for bad in [(-1, 4, 4), (1, 0, 4), (1, 4, 0), (1, 1 << 21, 4), (1 << 20, 1 << 15, 1 << 15)]:
        with pytest.raises(L.SparseOptError) as e:
            L.newton_schulz_workspace_size(*bad)
        assert e.value.code == _lib.EINVAL
    for bad in [(-1, 4), (4, 0)]:
        with pytest.raises(L.SparseOptError):
            L.layer_norm_backward_workspace_size(*bad)


def ns_cfg(coef=(3.4445, -4.7750, 2.0315), eps=1e-7, steps=5):
    return _lib.NsConfig((C.c_double * 3)(*coef), eps, steps)


def ns(g=FAKE, dt=0, batch=0, m=8, n=8, cfg=None, out=FAKE, ws=FAKE, wsb=0):
    return _lib.lib().newton_schulz(g, dt, batch, m, n, C.byref(cfg or ns_cfg()), out, ws, wsb,
                                    None, 0)


@pytest.mark.parametrize("kw", [
    {"g": None, "batch": 1}, {"out": None, "batch": 1}, {"dt": 2}, {"dt": 9}, {"batch": -1},
    {"m": 0}, {"n": 0}, {"m": 1 << 21}, {"cfg": ns_cfg(steps=0)}, {"cfg": ns_cfg(steps=65)},
    {"cfg": ns_cfg(eps=0.0)}, {"cfg": ns_cfg(eps=NAN)}, {"cfg": ns_cfg(coef=(NAN, 0, 0))},
    {"cfg": ns_cfg(coef=(1, INF, 0))}], ids=lambda k: ",".join(k))
def test_newton_schulz_refuses(kw):
    assert ns(**kw) == _lib.EINVAL
    assert b"newton_schulz" in _lib.lib().sparse_opt_last_error()


def test_newton_schulz_needs_its_workspace():
    assert ns(batch=1, ws=None) == _lib.EWORKSPACE
    assert ns(batch=1, wsb=100) == _lib.EWORKSPACE
    assert ns(batch=1, ws=264, wsb=1 << 30) == _lib.EWORKSPACE
    assert ns(batch=0, g=None, out=None, ws=None) == 0


@pytest.mark.parametrize("coef,steps", [
    ((3.4445, -4.7750, 2.0315), 64), ((2.0, -1.5, 0.5), 30), ((1.5, -0.5, 0.0), 30),
    ((1.0, 0.0, 0.0), 64), ((1.2, 0.0, 0.0), 4), ((4.0, 0.0, 0.0), 1), ((2.0, 0.0, 0.0), 2),
    ((0.0, 0.0, 0.0), 3), ((0.0, 0.0, 9.0), 1), ((1.0, -20.0, 20.0), 1), ((2.0, -12.0, 12.0), 1),
    ((1.0, -40.0, 40.0), 1), ((8.0, -9.0, 2.0), 3), ((-1.5, 0.5, 0.0), 4)])
def test_newton_schulz_coefficients(coef, steps):
    """Accepted exactly where a fine grid of starting values stays inside the bounds (values a
    hair above 1 in every step stand for rounding)."""
    a, b, c = coef
    hi, fine = 1.0, True
    for _ in range(steps):
        s = torch.linspace(0, hi * 1.01, 20001, dtype=torch.float64)
        fine &= bool((b * s ** 2 + c * s ** 4).abs().max() <= 8)
        hi = float((a * s + b * s ** 3 + c * s ** 5).abs().max())
        fine &= hi <= 2
    assert (ns(cfg=ns_cfg(coef=coef, steps=steps)) == 0) == fine


def muon(params=FAKE, pdt=0, buf=FAKE, g=FAKE, gdt=0, batch=0, m=8, n=8, lr=0.1, momentum=0.9,
         wd=0.0, scale=1.0, nesterov=1, cfg=None):
    c = _lib.MuonConfig(lr, momentum, wd, scale, nesterov, cfg or ns_cfg())
    return _lib.lib().muon_step(params, pdt, buf, g, gdt, batch, m, n, C.byref(c), FAKE, 0, None,
                                0)


@pytest.mark.parametrize("kw", [
    {"lr": -0.1}, {"lr": NAN}, {"lr": INF}, {"momentum": 1.0}, {"momentum": -0.1},
    {"momentum": NAN}, {"wd": -1.0}, {"wd": INF}, {"scale": NAN}, {"scale": INF},
    {"nesterov": 2}, {"pdt": 2}, {"gdt": 2}, {"batch": 1, "buf": None},
    {"batch": 1, "params": None}, {"batch": 1, "g": None}, {"m": 0}, {"cfg": ns_cfg(steps=0)},
    {"cfg": ns_cfg(coef=(9, 0, 0))}], ids=lambda k: ",".join(k))
def test_muon_refuses(kw):
    assert muon(**kw) == _lib.EINVAL
    assert b"muon_step" in _lib.lib().sparse_opt_last_error()
    assert muon() == 0


def test_layer_norm_formula_against_differences():
    g = torch.Generator().manual_seed(1)
    x, w, b, dy, v = (torch.randn(*s, generator=g, dtype=torch.float64)
                      for s in ((5, 24), (24,), (24,), (5, 24), (5, 24)))
    _, mu, rs = R.ln_forward(x, w, b, 1e-5)
    dx, dw, db = R.ln_backward(dy, x, mu, rs, w)
    f = lambda x_, w_, b_: float((R.ln_forward(x_, w_, b_, 1e-5)[0] * dy).sum())  # noqa: E731
    h = 1e-5
    for grad, at, move in ((dx, 0, v), (dw, 1, v[0]), (db, 2, v[1])):
        args = [x, w, b]
        hi, lo = list(args), list(args)
        hi[at], lo[at] = args[at] + h * move, args[at] - h * move
        slope = (f(*hi) - f(*lo)) / (2 * h)
        # h^2 of truncation and the 64-bit rounding of a sum of about 100 values over h
        assert abs(slope - float((grad * move).sum())) < 1e-7 * (1 + abs(slope))


def test_newton_schulz_formula_on_singular_values():
    """The iteration moves the singular values by its polynomial and keeps the vectors."""
    g = torch.Generator().manual_seed(2)
    m = torch.randn(12, 30, generator=g, dtype=torch.float64)
    u, s, vh = torch.linalg.svd(m, full_matrices=False)
    s = s / (s.norm() + 1e-7)
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    want = u @ torch.diag(s) @ vh
    assert (R.newton_schulz(m) - want).norm() < 1e-12 * want.norm()
    assert (R.newton_schulz(m.t().contiguous()) - want.t()).norm() < 1e-12 * want.norm()


def test_python_refuses_host_tensors():
    x = torch.zeros(4, 8)
    for call in (lambda: L.layer_norm_forward(x), lambda: L.newton_schulz(x),
                 lambda: L.layer_norm_backward(x, x, x[:, 0], x[:, 0]),
                 lambda: L.muon_step(x, x, x, lr=0.1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        L.newton_schulz([1.0])
