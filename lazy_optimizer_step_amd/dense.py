"""The dense operators beside a table's sparse step: layer norm, dropout, the Newton-Schulz
orthogonalisation and the Muon step (include/dense_ops.h).

A training step of the whole runs ``read_rows`` (or ``SparseEmbedding``), dropout,
layer norm and matrices forward, the loss (loss.py), their gradients backward,
``step_lookups`` for the table's touched rows and ``muon_step`` for each matrix.
The functions carry the C ABI's names and only marshal arguments, as the
package's other functions do; ``LayerNorm``, ``Dropout`` and ``Muon`` are the
modules and the optimizer over them.
"""
from __future__ import annotations

import ctypes as C
import functools
import math

import torch

from . import _alloc_on, _flags, _here, _lib, _need, _ptr, _stream, check

NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)

_DTYPES = {torch.float32: _lib.DTYPE_F32, torch.bfloat16: _lib.DTYPE_BF16,
           torch.float16: _lib.DTYPE_F16}


def _as_x(t, name, x):
    """t has x's shape and type and lies beside it."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != x.shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, x {tuple(x.shape)}")
    if t.dtype != x.dtype:
        raise TypeError(f"{name} must be {x.dtype}, got {t.dtype}")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, x on {x.device}")


def _apart(t, name, *others):
    """An output t does not begin where one of others, (tensor, name), does."""
    if t is None or t.numel() == 0:
        return
    for o, what in others:
        if o is not None and o.data_ptr() == t.data_ptr() and o.numel():
            raise ValueError(f"{name} may not be {what}")


def _rows(t, name, like=None):
    """(rows, cols, row stride) of a device tensor whose last axis holds adjacent values and
    whose leading axes collapse into evenly spaced rows; never a copy."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if like is not None:
        _as_x(t, name, like)
    else:
        if t.dtype not in _DTYPES:
            raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a ROCm device")
        if len(shape) < 1 or shape[-1] < 1:
            raise ValueError(f"{name} has no columns: shape {tuple(shape)}")
    cols = shape[-1]
    rows = t.numel() // cols
    if t.is_contiguous():
        return rows, cols, cols
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the values of a row must be adjacent")
    if rows <= 1:
        return rows, cols, cols
    try:
        stride = t.view(rows, cols).stride(0)
    except RuntimeError:
        raise ValueError(f"{name}: the rows of shape {tuple(shape)} with strides "
                         f"{t.stride()} are not evenly spaced") from None
    if stride < cols:
        raise ValueError(f"{name}: rows overlap (stride {stride} for {cols} columns)")
    return rows, cols, stride


def _like(x):
    """A new contiguous tensor of x's shape and type."""
    return torch.empty_like(x) if x.is_contiguous() else \
        torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _vector(t, name, x, cols, dtypes):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, x on {x.device}")
    if t.numel() != cols or not t.is_contiguous():
        raise ValueError(f"{name} must hold {cols} contiguous values, has shape {tuple(t.shape)}")


def layer_norm_forward(x: torch.Tensor, weight=None, bias=None, *, eps: float = 1e-5, out=None,
                       mean=None, rstd=None, stream=None, validate: bool = False):
    """y = (x - mean) * rstd * weight + bias over the last axis.  Returns (y, mean, rstd), the
    last two float32 with x's leading shape, as layer_norm_backward takes them.  x: float32,
    bfloat16 or float16, its rows evenly spaced; weight, bias: x's type or float32 (one type
    for both), or None.  out may be x."""
    rows, cols, xs = _rows(x, "x")
    allowed = (x.dtype, torch.float32)
    _vector(weight, "weight", x, cols, allowed)
    _vector(bias, "bias", x, cols, allowed)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError(f"weight is {weight.dtype}, bias {bias.dtype}: one type for both")
    w = weight if weight is not None else bias
    wdtype = _DTYPES[w.dtype] if w is not None else _lib.DTYPE_F32
    ys = cols
    if out is not None:
        _, _, ys = _rows(out, "out", x)
    if mean is not None:
        _need(mean, torch.float32, "mean", rows)
    if rstd is not None:
        _need(rstd, torch.float32, "rstd", rows)
    if out is None or mean is None or rstd is None:
        with _alloc_on(stream):
            if out is None:
                out = _like(x)
            if mean is None:
                mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
            if rstd is None:
                rstd = torch.empty_like(mean)
    check(_lib.lib().layer_norm_forward(
        x.data_ptr(), xs, rows, cols, _DTYPES[x.dtype], _ptr(weight), _ptr(bias), wdtype, eps,
        out.data_ptr(), ys, mean.data_ptr(), rstd.data_ptr(), _stream(stream), _flags(validate)))
    return out, mean, rstd


@functools.lru_cache(maxsize=1024)
def layer_norm_backward_workspace_size(rows: int, cols: int) -> int:
    out = C.c_size_t(0)
    check(_lib.lib().layer_norm_backward_workspace_size(rows, cols, C.byref(out)))
    return out.value


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight=None, *, out=None, dweight=None, dbias=None, want_dx=True,
                        want_dweight=True, want_dbias=True, workspace=None, stream=None,
                        validate: bool = False):
    """The gradients of layer_norm_forward: (dx, dweight, dbias), None for what is not wanted.
    dweight and dbias have the weight's type (without a weight, that of the tensors given, or
    float32).  out may be dy or x."""
    rows, cols, xs = _rows(x, "x")
    _, _, ds = _rows(dy, "dy", x)
    _vector(weight, "weight", x, cols, (x.dtype, torch.float32))
    given = weight if weight is not None else dweight if dweight is not None else dbias
    wt = given.dtype if given is not None else torch.float32
    if wt not in (x.dtype, torch.float32):
        raise TypeError(f"the weight's gradients must be {x.dtype} or float32, got {wt}")
    _vector(dweight, "dweight", x, cols, (wt,))
    _vector(dbias, "dbias", x, cols, (wt,))
    _need(mean, torch.float32, "mean", rows)
    _need(rstd, torch.float32, "rstd", rows)
    os_ = cols
    if out is not None:
        _, _, os_ = _rows(out, "out", x)
    if workspace is not None:
        _need(workspace, torch.uint8, "workspace")
    with _alloc_on(stream):
        if want_dx and out is None:
            out = _like(x)
        if want_dweight and dweight is None:
            dweight = x.new_empty(cols, dtype=wt)
        if want_dbias and dbias is None:
            dbias = torch.empty_like(dweight) if dweight is not None else x.new_empty(cols, dtype=wt)
        if workspace is None:
            workspace = x.new_empty(layer_norm_backward_workspace_size(rows, cols),
                                    dtype=torch.uint8)
    dx = out if want_dx else None
    dweight, dbias = dweight if want_dweight else None, dbias if want_dbias else None
    check(_lib.lib().layer_norm_backward(_ptr(dy), ds, _ptr(x), xs, rows, cols, _DTYPES[x.dtype],
                                         _ptr(mean), _ptr(rstd), _ptr(weight), _DTYPES[wt],
                                         _ptr(dx), os_, _ptr(dweight), _ptr(dbias),
                                         _ptr(workspace), workspace.numel(), _stream(stream),
                                         _flags(validate)))
    return dx, dweight, dbias


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        try:
            _rows(x, "x")
        except ValueError:
            x = x.contiguous()
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, mean, rstd, weight)
        ctx.bias = bias is not None
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        try:
            _rows(dy, "dy")
        except ValueError:
            dy = dy.contiguous()
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_backward(dy, x, mean, rstd, weight, want_dx=need[0],
                                         want_dweight=need[1], want_dbias=ctx.bias and need[2])
        return dx, dw, db, None


class LayerNorm(torch.nn.Module):
    """Layer norm over the last axis (``dim`` values), forward and backward in the library's
    kernels.  The parameters are ``dtype`` (float32 unless given); the input is that type, or
    bfloat16 or float16 with float32 parameters."""

    def __init__(self, dim: int, *, eps: float = 1e-5, weight: bool = True, bias: bool = True,
                 dtype=torch.float32, device="cuda"):
        super().__init__()
        self.dim, self.eps = dim, eps
        self.weight = torch.nn.Parameter(torch.ones(dim, dtype=dtype, device=device)) \
            if weight else None
        self.bias = torch.nn.Parameter(torch.zeros(dim, dtype=dtype, device=device)) \
            if bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.dim:
            raise ValueError(f"x has {x.shape[-1]} columns, the norm {self.dim}")
        return _LayerNorm.apply(x, self.weight, self.bias, self.eps)


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------

def _seed(seed, x):
    """(seed, device address of one or None) of a seed given as an int or a device tensor."""
    if isinstance(seed, torch.Tensor):
        _need(seed, torch.int64, "seed")
        if seed.numel() != 1:
            raise ValueError(f"seed must hold one value, has shape {tuple(seed.shape)}")
        if seed.device != x.device:
            raise ValueError(f"seed is on {seed.device}, x on {x.device}")
        return 0, seed.data_ptr()
    return int(seed) & 0xFFFFFFFFFFFFFFFF, None


def dropout_forward(x: torch.Tensor, p: float, seed, *, offset: int = 0, residual=None, out=None,
                    stream=None, validate: bool = False) -> torch.Tensor:
    """y = x / (1 - p) where it is kept, 0 where it is dropped, plus residual.  The mask is a
    function of (seed, offset) and the value's index and is never stored; dense_ops.h states
    it.  p counts in steps of 2^-16.  x: float32, bfloat16 or float16, its rows evenly spaced;
    residual: as x, or None.  seed: an int, or a device int64 tensor of one value that the
    kernel reads when it runs (a replayed graph then takes what it holds).  out may be x or
    residual (with the same row stride)."""
    rows, cols, xs = _rows(x, "x")
    _here(x, "x")
    rs = ys = cols
    if residual is not None:
        _, _, rs = _rows(residual, "residual", x)
    if out is not None:
        _, _, ys = _rows(out, "out", x)
    if out is not None and rows > 1:
        # In place, a value has to be written where it was read.
        if ys != xs:
            _apart(out, "out with another row stride", (x, "x"))
        if ys != rs:
            _apart(out, "out with another row stride", (residual, "residual"))
    seed, d_seed = _seed(seed, x)
    if out is None:
        with _alloc_on(stream):
            out = _like(x)
    check(_lib.lib().dropout_forward(
        x.data_ptr(), xs, _ptr(residual), rs, rows, cols, _DTYPES[x.dtype], p, seed, d_seed,
        offset & 0xFFFFFFFFFFFFFFFF, out.data_ptr(), ys, _stream(stream), _flags(validate)))
    return out


def dropout_backward(dy: torch.Tensor, p: float, seed, *, offset: int = 0, out=None, stream=None,
                     validate: bool = False) -> torch.Tensor:
    """dx of dropout_forward with the same p, seed and offset (the residual's gradient is dy).
    out may be dy."""
    rows, cols, ds = _rows(dy, "dy")
    _here(dy, "dy")
    os_ = cols
    if out is not None:
        _, _, os_ = _rows(out, "out", dy)
        if os_ != ds and rows > 1:
            _apart(out, "out with another row stride", (dy, "dy"))
    seed, d_seed = _seed(seed, dy)
    if out is None:
        with _alloc_on(stream):
            out = _like(dy)
    check(_lib.lib().dropout_backward(
        dy.data_ptr(), ds, rows, cols, _DTYPES[dy.dtype], p, seed, d_seed,
        offset & 0xFFFFFFFFFFFFFFFF, out.data_ptr(), os_, _stream(stream), _flags(validate)))
    return out


def _spaced(t):
    """t, or a copy of it where its rows are not evenly spaced."""
    try:
        _rows(t, "t")
        return t
    except ValueError:
        return t.contiguous()


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        if isinstance(seed, torch.Tensor):
            # What the caller writes there next belongs to the next mask.
            seed = seed.clone()
        ctx.p, ctx.seed, ctx.offset = p, seed, offset
        return dropout_forward(_spaced(x), p, seed, offset=offset,
                               residual=None if residual is None else _spaced(residual))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        dx = None
        if ctx.needs_input_grad[0]:
            dx = dropout_backward(_spaced(dy), ctx.p, ctx.seed, offset=ctx.offset)
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


class Dropout(torch.nn.Module):
    """Dropout of probability ``p`` in training, forward and backward in the library's kernels;
    ``forward(x, residual)`` adds the residual stream, of x's shape and type, in the same pass.

    Each training pass takes the next offset under ``seed``: modules of one seed have the same
    masks.  The seed is an int, or a device int64 tensor of one value, read when the kernel
    runs: a pass captured into a graph replays its offset, so change the tensor between
    replays.  None draws one from torch's default generator (``torch.manual_seed``) at the
    first training pass, so that modules that are copied before it differ too.  Seed and
    ``offset`` are part of the state dict.

    ``forward(x, residual, offset=k)`` takes offset k and leaves the count as it is: for a pass
    that is run again for its gradients (activation checkpointing), which needs the first
    run's mask.  Inside a backward pass, where such a run takes place, a training pass without
    ``offset`` is refused: it would take another mask."""

    def __init__(self, p: float, seed=None):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p must lie in [0, 1], got {p}")
        self.p, self.seed, self.offset = p, seed, 0

    def get_extra_state(self):
        seed = self.seed.clone() if isinstance(self.seed, torch.Tensor) else self.seed
        return {"offset": self.offset, "seed": seed}

    def set_extra_state(self, state):
        self.offset = state["offset"]
        seed = state.get("seed")
        if seed is None:
            return
        if isinstance(self.seed, torch.Tensor):
            # In place: a captured graph reads it there.
            self.seed.copy_(torch.as_tensor(seed))
        else:
            self.seed = int(seed)

    def forward(self, x: torch.Tensor, residual=None, *, offset=None) -> torch.Tensor:
        if not self.training:
            if residual is None:
                return x
            _as_x(residual, "residual", x)
            return x + residual
        if offset is None:
            if torch._C._current_graph_task_id() != -1:
                raise RuntimeError("Dropout is run again inside a backward pass (activation "
                                   "checkpointing): it needs the first run's mask, so give both "
                                   "runs the same offset, forward(x, offset=...)")
            offset, self.offset = self.offset, self.offset + 1
        if self.seed is None:
            self.seed = int(torch.randint(1 << 62, (), device="cpu"))
        return _Dropout.apply(x, residual, self.p, self.seed, offset)


# ---------------------------------------------------------------------------
# Orthogonalised updates
# ---------------------------------------------------------------------------

def _matrices(t, name):
    """(batch, m, n) of a contiguous device tensor of matrices."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.dim() < 2:
        raise ValueError(f"{name} must be a matrix or a batch of them, has shape "
                         f"{tuple(t.shape)}")
    _need(t, t.dtype, name)
    m, n = t.shape[-2:]
    if m < 1 or n < 1:
        raise ValueError(f"{name} has empty matrices: shape {tuple(t.shape)}")
    return t.numel() // (m * n), m, n


def _ns_config(coefficients, eps, steps) -> _lib.NsConfig:
    a, b, c = coefficients
    return _lib.NsConfig((C.c_double * 3)(a, b, c), eps, steps)


@functools.lru_cache(maxsize=1024)
def newton_schulz_workspace_size(batch: int, m: int, n: int) -> int:
    out = C.c_size_t(0)
    check(_lib.lib().newton_schulz_workspace_size(batch, m, n, C.byref(out)))
    return out.value


def _ns_workspace(workspace, batch, m, n, device):
    if workspace is None:
        return torch.empty(newton_schulz_workspace_size(batch, m, n), dtype=torch.uint8,
                           device=device)
    return _need(workspace, torch.uint8, "workspace")


def newton_schulz(g: torch.Tensor, *, steps: int = 5, coefficients=NS_COEFFICIENTS,
                  eps: float = 1e-7, out=None, workspace=None, stream=None,
                  validate: bool = False) -> torch.Tensor:
    """The Newton-Schulz iteration of a matrix (or each of a batch, leading axes), near its
    orthogonal factor.  g: float32 or bfloat16, contiguous; the result is bfloat16 (its
    products are taken in float16 for either, with float32 sums; dense_ops.h states the
    accuracy)."""
    batch, m, n = _matrices(g, "g")
    if out is not None:
        _need(out, torch.bfloat16, "out", g.numel())
    with _alloc_on(stream):
        if out is None:
            out = torch.empty_like(g, dtype=torch.bfloat16)
        workspace = _ns_workspace(workspace, batch, m, n, g.device)
    cfg = _ns_config(coefficients, eps, steps)
    check(_lib.lib().newton_schulz(_ptr(g), _DTYPES[g.dtype], batch, m, n, C.byref(cfg), _ptr(out),
                                   _ptr(workspace), workspace.numel(), _stream(stream),
                                   _flags(validate)))
    return out


def muon_step(params: torch.Tensor, grad: torch.Tensor, momentum_buf=None, *, lr: float,
              momentum: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0,
              scale: float = 1.0, steps: int = 5, coefficients=NS_COEFFICIENTS, eps: float = 1e-7,
              workspace=None, stream=None, validate: bool = False) -> None:
    """One Muon step of a weight matrix (or each of a batch), in place:
    buf = momentum * buf + grad; u = grad + momentum * buf (nesterov) or buf;
    params = (1 - lr * weight_decay) * params - lr * scale * newton_schulz(u).
    params, grad: float32 or bfloat16; momentum_buf: float32, None only for momentum 0."""
    batch, m, n = _matrices(params, "params")
    if grad.shape != params.shape:
        raise ValueError(f"grad has shape {tuple(grad.shape)}, params {tuple(params.shape)}")
    _matrices(grad, "grad")
    if momentum_buf is not None:
        _need(momentum_buf, torch.float32, "momentum_buf", params.numel())
    with _alloc_on(stream):
        workspace = _ns_workspace(workspace, batch, m, n, params.device)
    cfg = _lib.MuonConfig(lr, momentum, weight_decay, scale, 1 if nesterov else 0,
                          _ns_config(coefficients, eps, steps))
    check(_lib.lib().muon_step(_ptr(params), _DTYPES[params.dtype], _ptr(momentum_buf), _ptr(grad),
                               _DTYPES[grad.dtype], batch, m, n, C.byref(cfg), _ptr(workspace),
                               workspace.numel(), _stream(stream), _flags(validate)))


class Muon:
    """Muon over one weight: a matrix, or a batch of matrices stepped alike.

    adjust: the factor in front of the orthogonalised update, by the matrix's
    shape m x n: "spectral" sqrt(max(1, m / n)), "rms" 0.2 sqrt(max(m, n))
    (updates of the size Adam's have), or a number.  The object keeps its momentum and
    a workspace of newton_schulz_workspace_size bytes (12 a value of a large square
    matrix); weights that should share one take muon_step(workspace=...)."""

    def __init__(self, params: torch.Tensor, lr: float, momentum: float = 0.95,
                 nesterov: bool = True, weight_decay: float = 0.0, adjust="spectral",
                 steps: int = 5, coefficients=NS_COEFFICIENTS, eps: float = 1e-7):
        batch, m, n = _matrices(params, "params")
        if adjust == "spectral":
            scale = math.sqrt(max(1.0, m / n))
        elif adjust == "rms":
            scale = 0.2 * math.sqrt(max(m, n))
        elif isinstance(adjust, (int, float)):
            scale = float(adjust)
        else:
            raise ValueError(f"adjust {adjust!r}: 'spectral', 'rms' or a number")
        self.params = params
        self.lr, self.momentum, self.nesterov = lr, momentum, nesterov
        self.weight_decay, self.scale = weight_decay, scale
        self.steps, self.coefficients, self.eps = steps, coefficients, eps
        self.momentum_buf = torch.zeros(params.shape, dtype=torch.float32, device=params.device) \
            if momentum != 0.0 else None
        self._workspace = _ns_workspace(None, batch, m, n, params.device)

    def step(self, grad: torch.Tensor, *, stream=None, validate: bool = False) -> None:
        """One step from the weight's gradient.  The workspace is this object's: steps of one
        object on two streams need an order between them."""
        muon_step(self.params.detach(), grad, self.momentum_buf, lr=self.lr,
                  momentum=self.momentum, nesterov=self.nesterov, weight_decay=self.weight_decay,
                  scale=self.scale, steps=self.steps, coefficients=self.coefficients, eps=self.eps,
                  workspace=self._workspace, stream=stream, validate=validate)
