"""The operators of a language model's training step, bound with ctypes.

* ``linear_cross_entropy`` and ``linear_cross_entropy_grad``: the softmax cross
  entropy of a linear layer over a large vocabulary, without the logits in memory,
  and its gradients, with 16 bits of each logit of a chunk of rows there.
* ``dropout``: from a counter-based generator, whose mask is never stored.
* ``rms_norm`` and ``rms_norm_grad``: the root-mean-square norm of a residual
  stream to which a branch, with dropout, is added in the same pass.

As the operators of the expert layers, every call checks its arguments,
allocates its results with torch and enqueues the library's kernels on torch's
current stream; nothing waits for the device.  A result that goes into a buffer
of the caller's must not overlap an operand (dropout in place apart).  A backward
pass may be captured into a graph, as any of torch's, while no eager graph of the
same leaves lives.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from .binding import PSGD_MAX_NORM_WIDTH, CrossEntropyArgs, _check, lib
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
    out = x.new_empty((x.shape[0],) if reduction == "none" else (), dtype=torch.float32)
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
    and have w's and the bias's type otherwise.  torch does not differentiate the
    results.

    The probabilities are rounded once to x's type for the products, whatever type
    the results have; bfloat16 calls of over 3e9 multiplications (rows x vocab x
    width) round x, times the target's probability, as well for ``dw`` and ``db``.

    A row's buffers have about 2 bytes a word and 6 a column while the call's work
    is done: 2.3 GiB for 16384 rows of 65536 x 2048.  Rows go in chunks of about
    4 GiB, 256 rows at least.
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
        loss = x.new_empty((), dtype=torch.float32)
        dx = x.new_empty(x.shape)
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
    loss keeps no logit in memory.  float32: the mean over the rows whose target is
    not ``ignore_index`` (NaN if there is none), their sum, or with "none" the
    loss of each row, 0 where it is ignored.  A target outside the vocabulary
    that is not ``ignore_index`` gives NaN, and NaN gradients.

    torch differentiates the result; the backward pass computes the logits
    again, and takes the memory of ``linear_cross_entropy_grad``, which gives loss
    and gradients in one call and takes a quarter less time.  With "none", rows of
    unequal gradients round x times theirs as well (in float16 those under 6e-8 of
    the largest are lost).
    """
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad)):
        return _LinearCrossEntropy.apply(x, w, target, bias, ignore_index, reduction)
    return _loss(x, w, target, bias, ignore_index, reduction)


# --------------------------------------------------------------------- dropout --

def dropout_state(seed: int, step: int = 0, device=None) -> torch.Tensor:
    """Where the generator stands, for ``dropout`` and ``rms_norm``: an int64
    tensor (seed, step) on the device.  ``state[1] += 1`` goes on to the next
    step's masks, also inside a captured graph."""
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda" if device is None else device)


def _state_at(state: Optional[torch.Tensor], device: int) -> int:
    if state is None:
        raise ValueError("dropout needs a state (see dropout_state)")
    if state.dtype is not torch.int64:
        raise TypeError(f"state must be int64 (got {state.dtype})")
    if state.numel() != 2 or state.dim() != 1 or state.get_device() != device or not state.is_contiguous():
        raise ValueError("state must be (seed, step), contiguous, on the operands' device")
    return state.data_ptr()


def _cut(p: float) -> int:
    """p in 65536ths, as the library rounds it."""
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be in [0, 1] (got {p})")
    return round(p * 65536.0)


def _drop(x: torch.Tensor, p: float, state: torch.Tensor, site: int, out: Optional[torch.Tensor],
          seen: Optional[torch.Tensor] = None) -> torch.Tensor:
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise TypeError(f"x must be float32, bfloat16 or float16 (got {x.dtype})")
    device = x.get_device()
    if device < 0:
        raise ValueError("x must be a CUDA tensor")
    at = _state_at(state, device)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be in [0, 1] (got {p})")
    flat = x.is_contiguous()
    if not flat and (x.dim() != 2 or x.stride(1) != 1 or x.stride(0) < 0):
        x, flat = x.contiguous(), True
    if out is None:
        y = x.new_empty(x.shape)
    else:
        y = _result_check(out, x.shape, x.dtype, device)
        if not y.is_contiguous():
            flat = False
            if y.dim() != 2 or y.stride(1) != 1 or y.stride(0) < y.shape[1]:
                raise ValueError(f"out must lie in row-major order (strides {tuple(y.stride())})")
    if flat:
        rows, cols = 1, x.numel()
        ldx = ldy = cols
    else:
        rows, cols, ldx, ldy = x.shape[0], x.shape[1], x.stride(0), y.stride(0)
    with _on(device):
        _check(lib().psgd_dropout(rows, cols, dtype, x.data_ptr(), ldx, y.data_ptr(), ldy, p, at, site,
                                  None if seen is None else seen.data_ptr(), _stream(device)))
    if out is not None:
        _written((out,))
    return y


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, p, state, site):
        seen = None if state is None else torch.empty_like(state)  # None: refused by the call
        y = _drop(x, p, state, site, None, seen)
        ctx.save_for_backward(seen)
        ctx.how = p, site
        return y

    @staticmethod
    def backward(ctx, dy):
        seen, = ctx.saved_tensors
        p, site = ctx.how
        return dropout(dy, p, seen, site), None, None, None


def dropout(x: torch.Tensor, p: float, state: torch.Tensor, site: int = 0,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``x`` with each value zeroed with probability ``p`` and the others scaled
    by ``1 / (1 - p)``; ``p`` counts in 65536ths.

    The mask is no tensor: it comes from ``state`` (``dropout_state``: seed and
    step, on the device), ``site`` (0 to 65535, one of each place that drops in a
    step) and a value's index in row-major order, whatever its type and strides.
    The same call with dy gives the gradient, which is what torch's backward pass
    does, with the state that the forward pass saw.  A zeroed value is 0 whatever
    it was.  ``out`` may be x; operands that require a gradient are refused there.
    """
    if torch.is_grad_enabled() and x.requires_grad:
        if out is not None:
            raise RuntimeError("a result in out= cannot be differentiated, and x requires a gradient: detach it, or call "
                               "under torch.no_grad()")
        return _Dropout.apply(x, p, state, site)
    return _drop(x, p, state, site, out)


# ----------------------------------------------------------------------- norm --

_NORM_CTAS = 2432  # rows of sums in the gradient's workspace, as psgd_rms_norm_workspace has it


def _rows_of(name: str, t: torch.Tensor, like: torch.Tensor, device: int) -> torch.Tensor:
    """An operand of like's type and shape that the kernels read in place, or a copy of it."""
    if t.dtype is not like.dtype:
        raise TypeError(f"{name} must have the rows' type {like.dtype} (got {t.dtype})")
    if t is not like:
        if t.shape != like.shape:
            raise ValueError(f"{name} must have shape {tuple(like.shape)} (got {tuple(t.shape)})")
        if t.get_device() != device:
            raise ValueError(f"{name} must be on the operands' device")
    if not t.is_contiguous():
        width, ld = t.shape[1], t.stride(0)
        if t.stride(1) != 1 or width % 8 or ld % 8 or ld < width:
            return t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def _norm_check(name: str, x: torch.Tensor, weight: Optional[torch.Tensor]) -> Tuple[int, int, Optional[int], int]:
    """(data type, device, the weight's address and data type)."""
    kind, shape = x.dtype, x.shape
    dtype = _DTYPES.get(kind)
    if dtype is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16 (got {kind})")
    device = x.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if len(shape) != 2:
        raise ValueError(f"{name} must have 2 dimensions (got {tuple(shape)})")
    width = shape[1]
    if not 1 <= width <= PSGD_MAX_NORM_WIDTH:
        raise ValueError(f"{name} must have 1 to {PSGD_MAX_NORM_WIDTH} columns (got {width})")
    if weight is None:
        return dtype, device, None, dtype
    wkind = weight.dtype
    if wkind is not torch.float32 and wkind is not kind:
        raise TypeError(f"weight must be float32 or {kind} (got {wkind})")
    if weight.dim() != 1 or weight.numel() != width or weight.get_device() != device or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous vector of {width} values on {name}'s device")
    return dtype, device, weight.data_ptr(), _DTYPES[wkind]


def _norm(x, weight, residual, eps, p, state, site, seen=None):
    dtype, device, w, wdt = _norm_check("x", x, weight)
    rows, width = shape = x.shape
    x = _rows_of("x", x, x, device)
    res = r = at = None
    ldres = 0
    if residual is not None:
        residual = _rows_of("residual", residual, x, device)
        res, ldres = residual.data_ptr(), residual.stride(0)
    if p and _cut(p):
        at = _state_at(state, device)
    y = x.new_empty(shape)
    if at or res is not None:
        r = x.new_empty(shape)
    with _on(device):
        _check(lib().psgd_rms_norm(rows, width, dtype, x.data_ptr(), x.stride(0), res, ldres, w, wdt, eps, p, at, site,
                                   None if seen is None else seen.data_ptr(), y.data_ptr(), width,
                                   None if r is None else r.data_ptr(), width, _stream(device)))
    return y, r


def rms_norm_grad(dy: torch.Tensor, r: torch.Tensor, weight: Optional[torch.Tensor] = None,
                  dr: Optional[torch.Tensor] = None, eps: float = 1e-6, p: float = 0.0,
                  state: Optional[torch.Tensor] = None, site: int = 0, weight_grad: Optional[torch.Tensor] = None,
                  accumulate: bool = False):
    """The gradients of ``rms_norm``: ``(dx, dresidual, dw)``, of ``dy`` in its
    first result and ``dr`` (or None) in its second, ``r``.

    ``dresidual`` is the whole gradient in r; ``dx`` is that with dropout's mask,
    the same tensor without dropout.  ``dw`` is float32 (None without a weight),
    or goes into ``weight_grad`` (float32 or r's type), added to what is there with
    ``accumulate``.  torch does not differentiate the results.
    """
    with torch.no_grad():
        return _norm_grad(dy, r, weight, dr, eps, p, state, site, weight_grad, accumulate)


def _norm_grad(dy, r, weight, dr, eps, p, state, site, weight_grad=None, accumulate=False, need_w=True):
    dtype, device, w, wdt = _norm_check("r", r, weight)
    shape, kind = r.shape, r.dtype
    rows, width = shape
    drop = bool(p) and _cut(p) != 0
    at = _state_at(state, device) if drop else None
    dw = weight_grad
    if dw is not None:
        if weight is None:
            raise ValueError("weight_grad is given without a weight")
        if dw.dtype is not torch.float32 and dw.dtype is not kind:
            raise TypeError(f"weight_grad must be float32 or {kind} (got {dw.dtype})")
        if not _result_check(dw, weight.shape, dw.dtype, device, "weight_grad").is_contiguous():
            raise ValueError("weight_grad must be contiguous")
    elif accumulate:
        raise ValueError("accumulate adds to weight_grad, which is not given")
    elif weight is not None and need_w:
        dw = r.new_empty(width, dtype=torch.float32)
    r = _rows_of("r", r, r, device)
    dy = _rows_of("dy", dy, r, device)
    if dr is not None:
        dr = _rows_of("dr", dr, r, device)
    out = r.new_empty(shape)
    dx = r.new_empty(shape) if drop else None
    size = 0 if dw is None else min(rows, _NORM_CTAS) * width * 4
    with _on(device):
        stream = _stream(device)
        ws = _workspace(device, stream, size) if size else None
        _check(lib().psgd_rms_norm_grad(rows, width, dtype, dy.data_ptr(), dy.stride(0), r.data_ptr(), r.stride(0),
                                        None if dr is None else dr.data_ptr(), 0 if dr is None else dr.stride(0), w, wdt,
                                        eps, p, at, site, None if dx is None else dx.data_ptr(), width, out.data_ptr(),
                                        width, None if dw is None else dw.data_ptr(),
                                        dtype if dw is None else _DTYPES[dw.dtype], accumulate,
                                        None if ws is None else ws.data_ptr(), size, stream))
    if weight_grad is not None:
        _written((weight_grad,))
    return (out if dx is None else dx), out, dw


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, p, state, site):
        ctx.set_materialize_grads(False)
        seen = torch.empty_like(state) if _cut(p) and state is not None else None
        y, r = _norm(x, weight, residual, eps, p, state, site, seen)
        ctx.save_for_backward(x if r is None else r, weight, seen)
        ctx.how = eps, p, site
        return y if r is None else (y, r)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dr=None):
        r, weight, seen = ctx.saved_tensors
        eps, p, site = ctx.how
        need = ctx.needs_input_grad
        if dy is None and dr is None:
            return None, None, None, None, None, None, None
        dy = torch.zeros_like(r) if dy is None else dy
        buf = torch.empty_like(weight) if weight is not None and need[1] else None
        dx, dres, dw = _norm_grad(dy, r, weight, dr, eps, p, seen, site, buf, False, False)
        return (dx if need[0] else None), dw, (dres if need[2] else None), None, None, None, None


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-6, p: float = 0.0, state: Optional[torch.Tensor] = None, site: int = 0):
    """``(y, r)``: the residual stream ``r = residual + dropout(x, p)`` and its norm
    ``y = r / sqrt(mean(r^2) + eps) * weight``, row by row, in one pass.

    ``x`` and ``residual`` (rows, width) are float32, bfloat16 or float16,
    ``weight`` (width) float32 or of x's type, or None.  r is rounded to x's type
    and y computed from that; sums are float32.  Without a residual and dropout r
    is x.  ``p``, ``state`` and ``site`` as for ``dropout``.  torch differentiates
    both results; ``rms_norm_grad`` gives the gradients directly.
    """
    if torch.is_grad_enabled() and (x.requires_grad or (weight is not None and weight.requires_grad)
                                    or (residual is not None and residual.requires_grad)):
        got = _RmsNorm.apply(x, weight, residual, eps, p, state, site)
        return got if isinstance(got, tuple) else (got, x)
    y, r = _norm(x, weight, residual, eps, p, state, site)
    return y, x if r is None else r
