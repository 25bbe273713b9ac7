"""Softmax cross entropy of hidden states against a table of classes, without its logits
(include/dense_ops.h).

``linear_cross_entropy_forward`` gives the loss and each row's log of its sum of
exponentials, ``linear_cross_entropy_backward`` the gradients of the hidden
states and of the table.  Both carry the C ABI's names and only marshal
arguments; ``LinearCrossEntropy`` is the module over them.
"""
from __future__ import annotations

import ctypes as C
import functools

import torch

from . import _alloc_on, _flags, _here, _lib, _need, _ptr, _stream, check
from .dense import _DTYPES, _apart, _like, _rows, _spaced

_REDUCTIONS = {"none": _lib.REDUCE_NONE, "sum": _lib.REDUCE_SUM, "mean": _lib.REDUCE_MEAN}


@functools.lru_cache(maxsize=1024)
def _workspace_size(rows, cols, classes, dtype, backward) -> int:
    out = C.c_size_t(0)
    check(_lib.lib().linear_cross_entropy_workspace_size(rows, cols, classes, dtype, backward,
                                                         C.byref(out)))
    return out.value


def linear_cross_entropy_workspace_size(rows: int, cols: int, classes: int, dtype: torch.dtype, *,
                                        backward: bool) -> int:
    """Bytes of workspace the forward (or the backward) pass takes."""
    return _workspace_size(rows, cols, classes, _DTYPES[dtype], 1 if backward else 0)


def linear_cross_entropy_plan(rows: int, cols: int, classes: int, dtype: torch.dtype, *,
                              backward: bool) -> dict:
    """Which kernels the forward (or the backward) pass takes at a size: spopt_ce_plan of
    dense_ops.h."""
    p = _lib.CePlan()
    check(_lib.lib().linear_cross_entropy_plan(rows, cols, classes, _DTYPES[dtype],
                                               1 if backward else 0, C.byref(p)))
    return {name: getattr(p, name) for name, _ in p._fields_}


def _table(weight, name, x, cols):
    """(classes, row stride) of a classes x cols matrix of x's type."""
    if not isinstance(weight, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if weight.dtype != x.dtype:
        raise TypeError(f"{name} must be {x.dtype}, got {weight.dtype}")
    if weight.device != x.device:
        raise ValueError(f"{name} is on {weight.device}, x on {x.device}")
    if weight.dim() != 2 or weight.shape[0] < 1 or weight.shape[1] != cols:
        raise ValueError(f"{name} must be (classes, {cols}), has shape {tuple(weight.shape)}")
    return weight.shape[0], _rows(weight, name)[2]


def _inputs(x, weight, targets, reduction):
    rows, cols, xs = _rows(x, "x")
    _here(x, "x")
    classes, ws = _table(weight, "weight", x, cols)
    _need(targets, torch.int64, "targets")
    if targets.device != x.device:
        raise ValueError(f"targets is on {targets.device}, x on {x.device}")
    if targets.shape != x.shape[:-1]:
        raise ValueError(f"targets has shape {tuple(targets.shape)}, x {tuple(x.shape)}")
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction {reduction!r}: 'none', 'sum' or 'mean'")
    return rows, cols, xs, classes, ws, _REDUCTIONS[reduction]


def _floats(t, name, x, numel):
    _need(t, torch.float32, name)
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, x on {x.device}")
    if t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} values, has shape {tuple(t.shape)}")


def _space(workspace, x):
    if workspace is not None and _need(workspace, torch.uint8, "workspace").device != x.device:
        raise ValueError(f"workspace is on {workspace.device}, x on {x.device}")


def linear_cross_entropy_forward(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, *,
                                 reduction: str = "mean", ignore_index: int = -100,
                                 label_smoothing: float = 0.0, out=None, lse=None, workspace=None,
                                 stream=None, validate: bool = False):
    """Softmax cross entropy of x weight^T against targets, the logits never stored.  Returns
    (loss, lse): the loss float32, one value, or one a row for reduction "none"; lse float32,
    each row's log of its sum of exponentials, as linear_cross_entropy_backward takes it.  x:
    (..., cols) of float32, bfloat16 or float16, its rows evenly spaced; weight: (classes,
    cols) of x's type; targets: int64 of x's leading shape.  Rows whose target is ignore_index
    do not count: loss and lse are 0 there; with none that counts the loss is 0.  Outputs and
    workspace may not overlap one another or an input."""
    rows, cols, xs, classes, ws, how = _inputs(x, weight, targets, reduction)
    shape = x.shape[:-1] if reduction == "none" else ()
    if out is not None:
        _floats(out, "out", x, rows if reduction == "none" else 1)
    if lse is not None:
        _floats(lse, "lse", x, rows)
    _space(workspace, x)
    if out is not None or lse is not None or workspace is not None:
        read = (x, "x"), (weight, "weight"), (targets, "targets")
        _apart(out, "out", *read, (lse, "lse"))
        _apart(lse, "lse", *read)
        _apart(workspace, "workspace", *read, (out, "out"), (lse, "lse"))
    with _alloc_on(stream):
        if out is None:
            out = x.new_empty(shape, dtype=torch.float32)
        if lse is None:
            lse = x.new_empty(x.shape[:-1], dtype=torch.float32)
        if workspace is None:
            workspace = x.new_empty(_workspace_size(rows, cols, classes, _DTYPES[x.dtype], 0),
                                    dtype=torch.uint8)
    check(_lib.lib().linear_cross_entropy_forward(
        x.data_ptr(), xs, weight.data_ptr(), ws, rows, cols, classes, _DTYPES[x.dtype],
        targets.data_ptr(), ignore_index, label_smoothing, how, out.data_ptr(), lse.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream(stream), _flags(validate)))
    return out, lse


def linear_cross_entropy_backward(dloss: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                                  targets: torch.Tensor, lse: torch.Tensor, *,
                                  reduction: str = "mean", ignore_index: int = -100,
                                  label_smoothing: float = 0.0, out=None, dweight=None,
                                  want_dx=True, want_dweight=True, workspace=None, stream=None,
                                  validate: bool = False):
    """The gradients of linear_cross_entropy_forward: (dx, dweight), None for what is not
    wanted.  dloss: float32, one value, or one a row for reduction "none".  Outputs and workspace
    may not overlap one another or an input."""
    rows, cols, xs, classes, ws, how = _inputs(x, weight, targets, reduction)
    _floats(dloss, "dloss", x, rows if reduction == "none" else 1)
    _floats(lse, "lse", x, rows)
    os_ = dws = cols
    if out is not None:
        _, _, os_ = _rows(out, "out", x)
    if dweight is not None:
        if _table(dweight, "dweight", x, cols)[0] != classes:
            raise ValueError(f"dweight has shape {tuple(dweight.shape)}, weight "
                             f"{tuple(weight.shape)}")
        _, _, dws = _rows(dweight, "dweight")
    _space(workspace, x)
    if out is not None or dweight is not None or workspace is not None:
        read = (x, "x"), (weight, "weight"), (targets, "targets"), (dloss, "dloss"), (lse, "lse")
        _apart(out, "out", *read, (dweight, "dweight"))
        _apart(dweight, "dweight", *read)
        _apart(workspace, "workspace", *read, (out, "out"), (dweight, "dweight"))
    with _alloc_on(stream):
        if want_dx and out is None:
            out = _like(x)
        if want_dweight and dweight is None:
            dweight = _like(weight)
        if workspace is None:
            workspace = x.new_empty(_workspace_size(rows, cols, classes, _DTYPES[x.dtype], 1),
                                    dtype=torch.uint8)
    dx, dweight = out if want_dx else None, dweight if want_dweight else None
    check(_lib.lib().linear_cross_entropy_backward(
        dloss.data_ptr(), x.data_ptr(), xs, weight.data_ptr(), ws, rows, cols, classes,
        _DTYPES[x.dtype], targets.data_ptr(), ignore_index, label_smoothing, how, lse.data_ptr(),
        _ptr(dx), os_, _ptr(dweight), dws, workspace.data_ptr(), workspace.numel(),
        _stream(stream), _flags(validate)))
    return dx, dweight


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, reduction, ignore_index, label_smoothing):
        x, weight, targets = _spaced(x), _spaced(weight), targets.contiguous()
        loss, lse = linear_cross_entropy_forward(
            x, weight, targets, reduction=reduction, ignore_index=ignore_index,
            label_smoothing=label_smoothing)
        ctx.save_for_backward(x, weight, targets, lse)
        ctx.how = dict(reduction=reduction, ignore_index=ignore_index,
                       label_smoothing=label_smoothing)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        x, weight, targets, lse = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw = linear_cross_entropy_backward(dloss.contiguous(), x, weight, targets, lse,
                                               want_dx=need[0], want_dweight=need[1], **ctx.how)
        return dx, dw, None, None, None, None


class LinearCrossEntropy(torch.nn.Module):
    """The last layer and its loss: softmax cross entropy of hidden states of ``dim`` values
    against ``classes`` rows, the logits never stored.

    weight: the table to use, (classes, dim) (shared, not copied): a parameter, or a tensor that
    requires its gradient, which is dense; else one of its own, N(0, 1 / dim).  A table that is to
    stay as it is comes as ``torch.nn.Parameter(weight, requires_grad=False)``: a plain tensor, such
    as a SparseEmbedding's weight, whose step takes lookups' rows and no dense gradient, is refused.
    forward(x, targets) gives the loss: x of the table's type, (..., dim); targets int64 of x's
    leading shape.

    Before a backward pass is captured into a graph, let go of the losses of eager passes over
    the same parameters: while one lives, torch adds the parameters' gradients up on the stream
    of that pass, outside the capture."""

    def __init__(self, dim: int, classes: int, *, weight=None, reduction: str = "mean",
                 ignore_index: int = -100, label_smoothing: float = 0.0, dtype=torch.float32,
                 device="cuda"):
        super().__init__()
        if reduction not in _REDUCTIONS:
            raise ValueError(f"reduction {reduction!r}: 'none', 'sum' or 'mean'")
        if weight is None:
            weight = torch.nn.Parameter(torch.randn(classes, dim, dtype=dtype, device=device)
                                        / dim ** 0.5)
        if tuple(weight.shape) != (classes, dim):
            raise ValueError(f"weight has shape {tuple(weight.shape)}, needs ({classes}, {dim})")
        if not (weight.requires_grad or isinstance(weight, torch.nn.Parameter)):
            raise ValueError("weight is a plain tensor, which would get no gradient: pass a "
                             "torch.nn.Parameter, with requires_grad=False for a table that stays "
                             "as it is")
        self.weight = weight
        self.reduction, self.ignore_index = reduction, ignore_index
        self.label_smoothing = label_smoothing

    def forward(self, x: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        return _LinearCrossEntropy.apply(x, self.weight, targets, self.reduction,
                                         self.ignore_index, self.label_smoothing)
