"""The operators of a language model's training step, bound with ctypes.

* ``linear_cross_entropy`` and ``linear_cross_entropy_grad``: the softmax cross
  entropy of a linear layer over a large vocabulary, and its gradients, without
  the logits in memory.

As the operators of the expert layers, every call checks its arguments,
allocates its results with torch and enqueues the library's kernels on torch's
current stream; nothing waits for the device.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from .binding import PSGD_F32, CrossEntropyArgs, _check, lib
from .operators import _DTYPES, _HALF, _on, _result_check, _row_stride, _stream, _workspace, _written

_REDUCTIONS = ("mean", "sum", "none")


# ------------------------------------------- cross entropy over a vocabulary --

def _gradient_at(device: int, name: str, t: torch.Tensor, shape, kind: torch.dtype) -> int:
    """Checks a caller's buffer of a gradient; its data type."""
    if t.dtype is not torch.float32 and t.dtype is not kind:
        raise TypeError(f"{name} must be float32 or {kind} (got {t.dtype})")
    _result_check(t, shape, t.dtype, device, name)
    return _DTYPES[t.dtype]


def _loss_args(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, bias: Optional[torch.Tensor],
               ignore_index: int, reduction: str) -> Tuple[CrossEntropyArgs, int]:
    """The arguments that every call has, checked; and the device."""
    kind = x.dtype
    dtype = _HALF.get(kind)
    if dtype is None:
        raise TypeError(f"x must be bfloat16 or float16 (got {kind})")
    if w.dtype is not kind:
        raise TypeError(f"w must have x's type {kind} (got {w.dtype})")
    if target.dtype is not torch.int64 and target.dtype is not torch.int32:
        raise TypeError(f"target must be int64 or int32 (got {target.dtype})")
    if reduction not in _REDUCTIONS:
        raise ValueError(f"reduction must be one of {_REDUCTIONS} (got {reduction!r})")
    device = x.get_device()
    if device < 0 or w.get_device() != device or target.get_device() != device:
        raise ValueError("x, w and target must be CUDA tensors on one device")
    xshape, wshape = x.shape, w.shape
    if len(xshape) != 2 or len(wshape) != 2 or wshape[1] != xshape[1]:
        raise ValueError(f"x must be (rows, width) and w (vocab, width) (got {tuple(xshape)} and {tuple(wshape)})")
    if target.dim() != 1 or target.shape[0] != xshape[0] or not target.is_contiguous():
        raise ValueError(f"target must be a contiguous vector of {xshape[0]} values (got {tuple(target.shape)})")
    a = CrossEntropyArgs()
    a.rows, a.width = xshape
    a.vocab = wshape[0]
    a.x, a.ldx = x.data_ptr(), _row_stride("x", xshape, x.stride())
    a.w, a.ldw = w.data_ptr(), _row_stride("w", wshape, w.stride())
    a.target, a.target_bytes, a.ignore_index = target.data_ptr(), target.element_size(), int(ignore_index)
    a.dtype, a.mean, a.scale = dtype, reduction == "mean", 1.0
    if bias is not None:
        if bias.dtype is not torch.float32 and bias.dtype is not kind:
            raise TypeError(f"bias must be float32 or {kind} (got {bias.dtype})")
        if bias.get_device() != device or bias.shape != wshape[:1] or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous vector of {wshape[0]} values on x's device")
        a.bias, a.bias_dtype = bias.data_ptr(), _DTYPES[bias.dtype]
    return a, device


def _enqueue(a: CrossEntropyArgs, device: int) -> None:
    size = ctypes.c_size_t()
    at = ctypes.byref(a)
    _check(lib().psgd_cross_entropy_workspace(at, ctypes.byref(size)))
    with _on(device):
        stream = _stream(device)
        ws = _workspace(device, stream, size.value)
        _check(lib().psgd_cross_entropy(at, ws.data_ptr(), size.value, stream))


def _loss(x, w, target, bias, ignore_index, reduction) -> torch.Tensor:
    a, device = _loss_args(x, w, target, bias, ignore_index, reduction)
    out = torch.empty(x.shape[0] if reduction == "none" else (), dtype=torch.float32, device=x.device)
    if reduction == "none":
        a.losses = out.data_ptr()
        if not a.rows:
            return out
    else:
        a.loss = out.data_ptr()
    _enqueue(a, device)
    return out


def linear_cross_entropy_grad(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor,
                              bias: Optional[torch.Tensor] = None, ignore_index: int = -100, reduction: str = "mean",
                              scale: float = 1.0, weight_grad: Optional[torch.Tensor] = None,
                              bias_grad: Optional[torch.Tensor] = None, accumulate: bool = False):
    """The loss of ``linear_cross_entropy`` and its gradients, of one call:
    ``(loss, dx, dw, db)`` (``db`` is None without a bias).

    The gradients are those of ``scale * loss``.  ``dx`` has x's type; ``dw``
    and ``db`` go into ``weight_grad`` and ``bias_grad`` where these are given
    (float32 or x's type; rows may be strided, as in a packed gradient buffer, see
    ``GradientLayout.layer_view``), added to what is there with ``accumulate``,
    and have w's and the bias's type otherwise.  The probabilities are rounded
    once to x's type for the products, whatever type the results have.
    torch does not differentiate the results.
    """
    if reduction == "none":
        raise ValueError("reduction must be 'mean' or 'sum': the gradients are those of one number")
    if accumulate and weight_grad is None and bias_grad is None:
        raise ValueError("accumulate adds to weight_grad and bias_grad, and neither is given")
    with torch.no_grad():
        a, device = _loss_args(x, w, target, bias, ignore_index, reduction)
        dw = torch.empty_like(w, memory_format=torch.contiguous_format) if weight_grad is None else weight_grad
        db = None if bias is None else torch.empty_like(bias) if bias_grad is None else bias_grad
        if bias is None and bias_grad is not None:
            raise ValueError("bias_grad is given without a bias")
        if accumulate and (weight_grad is None or (db is not None and bias_grad is None)):
            raise ValueError("accumulate needs every gradient's buffer: weight_grad, and bias_grad with a bias")
        loss = torch.empty((), dtype=torch.float32, device=x.device)
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        a.scale, a.accumulate, a.loss = float(scale), bool(accumulate), loss.data_ptr()
        _gradients(a, device, x, w, bias, dx, dw, db)
        _enqueue(a, device)
        _written([t for t in (weight_grad, bias_grad) if t is not None])
    return loss, dx, dw, db


def _gradients(a, device, x, w, bias, dx, dw, db) -> None:
    """The results that are gradients, each of them or None."""
    if dx is not None:
        a.dx, a.lddx = dx.data_ptr(), dx.shape[1]
    if dw is not None:
        a.dw_dtype = _gradient_at(device, "weight_grad", dw, w.shape, w.dtype)
        a.dw, a.lddw = dw.data_ptr(), _row_stride("weight_grad", dw.shape, dw.stride())
    if db is not None:
        a.db_dtype = _gradient_at(device, "bias_grad", db, bias.shape, x.dtype)
        if not db.is_contiguous():
            raise ValueError("bias_grad must be contiguous")
        a.db = db.data_ptr()


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, target, bias, ignore_index, reduction):
        ctx.save_for_backward(x, w, target, bias)
        ctx.how = ignore_index, reduction
        return _loss(x, w, target, bias, ignore_index, reduction)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, w, target, bias = ctx.saved_tensors
        ignore_index, reduction = ctx.how
        a, device = _loss_args(x, w, target, bias, ignore_index, reduction)
        need = ctx.needs_input_grad
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need[0] else None
        dw = torch.empty_like(w, memory_format=torch.contiguous_format) if need[1] else None
        db = torch.empty_like(bias) if need[3] else None
        g = g.contiguous()
        if reduction == "none":
            a.row_scale = g.data_ptr()
        else:
            a.scale_dev = g.data_ptr()
        _gradients(a, device, x, w, bias, dx, dw, db)
        _enqueue(a, device)
        return dx, dw, None, db, None, None


def linear_cross_entropy(x: torch.Tensor, w: torch.Tensor, target: torch.Tensor, bias: Optional[torch.Tensor] = None,
                         ignore_index: int = -100, reduction: str = "mean") -> torch.Tensor:
    """Softmax cross entropy of the logits ``x @ w.T + bias`` at ``target``.

    ``x`` (rows, width) and ``w`` (vocab, width) are bfloat16 or float16,
    ``target`` (rows) int64 or int32, ``bias`` (vocab) float32 or x's type.  The
    logits are never in memory.  float32: the mean over the rows whose target is
    not ``ignore_index`` (NaN if there is none), their sum, or with "none" the
    loss of each row, 0 where it is ignored.  A target outside the vocabulary
    that is not ``ignore_index`` gives NaN, and NaN gradients.

    torch differentiates the result; the backward pass computes the logits
    again.  ``linear_cross_entropy_grad`` gives loss and gradients in one call
    and takes a quarter less.
    """
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad)):
        return _LinearCrossEntropy.apply(x, w, target, bias, ignore_index, reduction)
    return _loss(x, w, target, bias, ignore_index, reduction)
