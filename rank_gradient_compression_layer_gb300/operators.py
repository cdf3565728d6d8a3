"""The operators beside the compression step, bound with ctypes.

* ``experts_forward``, ``experts_grad_input``, ``experts_grad_weight`` and the
  differentiable ``experts_linear``: matrix products grouped by expert, over
  rows sorted by expert with ragged group sizes.
* ``grad_norm``, ``clip_grad_norm`` and ``GradientLayout``: the global norm of
  a set of gradients, and clipping by it.

Every call checks its arguments, allocates its results with torch and enqueues
the library's kernels on torch's current stream; nothing waits for the device.
A tensor that another stream wrote has to be ordered before the call by the
caller, as for any torch operation.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import torch

from .binding import (PSGD_BF16, PSGD_F16, PSGD_F32, PSGD_GRAD_NORM_WORKSPACE, PSGD_MAX_EXPERTS, _check, _i64,
                      lib, psgd_plan_layout)

_DTYPES = {torch.float32: PSGD_F32, torch.bfloat16: PSGD_BF16, torch.float16: PSGD_F16}
_HALF = {torch.bfloat16: PSGD_BF16, torch.float16: PSGD_F16}


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


# ------------------------------------------------------- expert products --

def _row_stride(name: str, t: torch.Tensor) -> int:
    """Row stride of the last two dimensions; their rows must be contiguous."""
    if t.size(-1) > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous (strides {tuple(t.stride())})")
    return t.stride(-2) if t.size(-2) > 1 else t.size(-1)


def _experts_check(name: str, rows: torch.Tensor, offsets: torch.Tensor) -> Tuple[int, int]:
    """Checks what the three products share; (data type, experts)."""
    dtype = _HALF.get(rows.dtype)
    if dtype is None:
        raise TypeError(f"{name} must be bfloat16 or float16 (got {rows.dtype})")
    _need(rows.is_cuda, f"{name} must be a CUDA tensor")
    _need(rows.dim() == 2, f"{name} must have 2 dimensions (got {tuple(rows.shape)})")
    if offsets.dtype != torch.int32:
        raise TypeError(f"offsets must be int32 (got {offsets.dtype})")
    _need(offsets.dim() == 1 and offsets.numel() >= 2 and offsets.is_contiguous(),
          "offsets must be a contiguous vector of experts + 1 values")
    _need(offsets.numel() - 1 <= PSGD_MAX_EXPERTS, f"at most {PSGD_MAX_EXPERTS} experts (got {offsets.numel() - 1})")
    _need(offsets.device == rows.device, "offsets must be on the operands' device")
    return dtype, offsets.numel() - 1


def _weights_check(w: torch.Tensor, rows: torch.Tensor, experts: int) -> None:
    if w.dtype != rows.dtype:
        raise TypeError(f"w must have the rows' type {rows.dtype} (got {w.dtype})")
    _need(w.dim() == 3 and w.size(0) == experts, f"w must be ({experts}, n, k) (got {tuple(w.shape)})")
    _need(w.device == rows.device, "w must be on the operands' device")


def _result(out: Optional[torch.Tensor], shape, dtype, device) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.dtype != dtype:
        raise TypeError(f"out must be {dtype} (got {out.dtype})")
    _need(tuple(out.shape) == tuple(shape), f"out must have shape {tuple(shape)} (got {tuple(out.shape)})")
    _need(out.device == device, "out must be on the operands' device")
    return out


def experts_forward(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``y[t] = w[e(t)] @ x[t]`` for rows sorted by expert.

    ``x`` (rows, k) and ``w`` (experts, n, k) are bfloat16 or float16;
    ``offsets`` (experts + 1, int32, on the device) gives each expert's rows
    ``offsets[e]:offsets[e + 1]``.  Rows of no expert give zeros.  Sums are
    float32, rounded once to the operands' type.
    """
    dtype, experts = _experts_check("x", x, offsets)
    _weights_check(w, x, experts)
    rows, k = x.shape
    n = w.size(1)
    _need(w.size(2) == k, f"w has {w.size(2)} columns, x {k}")
    y = _result(out, (rows, n), x.dtype, x.device)
    with torch.cuda.device(x.device):
        _check(lib().psgd_experts_forward(
            rows, experts, n, k, dtype, x.data_ptr(), _row_stride("x", x), w.data_ptr(), _row_stride("w", w),
            w.stride(0), offsets.data_ptr(), y.data_ptr(), _row_stride("out", y), _stream(x.device)))
    return y


def experts_grad_input(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``dx[t] = w[e(t)].T @ dy[t]``: the gradient of ``experts_forward`` in x.

    ``dy`` (rows, n), ``w`` (experts, n, k), ``offsets`` as in the forward
    product; the result is (rows, k).
    """
    dtype, experts = _experts_check("dy", dy, offsets)
    _weights_check(w, dy, experts)
    rows, n = dy.shape
    k = w.size(2)
    _need(w.size(1) == n, f"w has {w.size(1)} rows, dy {n} columns")
    dx = _result(out, (rows, k), dy.dtype, dy.device)
    with torch.cuda.device(dy.device):
        _check(lib().psgd_experts_grad_input(
            rows, experts, n, k, dtype, dy.data_ptr(), _row_stride("dy", dy), w.data_ptr(), _row_stride("w", w),
            w.stride(0), offsets.data_ptr(), dx.data_ptr(), _row_stride("out", dx), _stream(dy.device)))
    return dx


def experts_grad_weight(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``dw[e] = dy[rows of e].T @ x[rows of e]``: the gradient in w.

    The result (experts, n, k) is float32, the type the compression step
    takes; ``out`` may be a strided view of a packed gradient buffer (see
    ``GradientLayout.experts_view``), or have the operands' type.  An expert
    without rows gets zeros.
    """
    dtype, experts = _experts_check("dy", dy, offsets)
    _need(x.dim() == 2 and x.size(0) == dy.size(0), f"x must have dy's {dy.size(0)} rows (got {tuple(x.shape)})")
    if x.dtype != dy.dtype:
        raise TypeError(f"x must have dy's type {dy.dtype} (got {x.dtype})")
    _need(x.device == dy.device, "x must be on the operands' device")
    rows, n = dy.shape
    k = x.size(1)
    odt = out.dtype if out is not None and out.dtype == dy.dtype else torch.float32
    dw = _result(out, (experts, n, k), odt, dy.device)
    with torch.cuda.device(dy.device):
        _check(lib().psgd_experts_grad_weight(
            rows, experts, n, k, dtype, dy.data_ptr(), _row_stride("dy", dy), x.data_ptr(), _row_stride("x", x),
            offsets.data_ptr(), _DTYPES[odt], dw.data_ptr(), _row_stride("out", dw), dw.stride(0),
            _stream(dy.device)))
    return dw


class _ExpertsLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, weight_grad):
        ctx.save_for_backward(x, w, offsets)
        ctx.weight_grad = weight_grad
        return experts_forward(x, w, offsets)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx = experts_grad_input(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw = None
        if ctx.weight_grad is not None:
            experts_grad_weight(dy, x, offsets, out=ctx.weight_grad)
        elif ctx.needs_input_grad[1]:
            dw = experts_grad_weight(dy, x, offsets, out=torch.empty_like(w, memory_format=torch.contiguous_format))
        return dx, dw, None, None


def experts_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                   weight_grad: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``experts_forward`` that torch differentiates.

    With ``weight_grad`` (experts, n, k; float32 or w's type) the backward
    pass writes the weight gradient there -- for instance into a packed buffer
    of the compression step -- and leaves ``w.grad`` alone.
    """
    return _ExpertsLinear.apply(x, w, offsets, weight_grad)


# ------------------------------------------------------- norm and clipping --

def _two_dims(t: torch.Tensor) -> Optional[Tuple[int, int, int]]:
    """(rows, columns, row stride) of a tensor whose values lie so, in any order of its dimensions."""
    dims = sorted((st, sz) for sz, st in zip(t.shape, t.stride()) if sz != 1)
    if not dims:
        return 1, 1, 1
    cols = 1
    i = 0
    while i < len(dims) and dims[i][0] == cols:
        cols *= dims[i][1]
        i += 1
    if i == len(dims):
        return 1, cols, cols
    ld, rows = dims[i][0], 1
    if ld < cols:
        return None
    while i < len(dims) and dims[i][0] == ld * rows:
        rows *= dims[i][1]
        i += 1
    return (rows, cols, ld) if i == len(dims) else None


def _table(name: str, tensors: Sequence[torch.Tensor]):
    """Pointers, rows, columns and row strides of a list of tensors."""
    ptrs = [t.data_ptr() for t in tensors]
    if all([t.is_contiguous() for t in tensors]):
        cols = [t.numel() for t in tensors]
        return ptrs, [1] * len(cols), cols, cols
    rows, cols, lds = [], [], []
    for i, t in enumerate(tensors):
        shape = (0, 0, 0) if t.numel() == 0 else _two_dims(t)
        if shape is None:
            raise ValueError(f"{name} {i}: values must lie in equally spaced contiguous rows (shape "
                             f"{tuple(t.shape)}, strides {tuple(t.stride())})")
        rows.append(shape[0])
        cols.append(shape[1])
        lds.append(shape[2])
    return ptrs, rows, cols, lds


def _one_type(tensors: Sequence[torch.Tensor]) -> Tuple[int, torch.device]:
    if not tensors:
        raise ValueError("the list of tensors is empty")
    first = tensors[0]
    dtype, device = first.dtype, first.device
    if dtype not in _DTYPES:
        raise TypeError(f"gradients must be float32, bfloat16 or float16 (got {dtype})")
    _need(first.is_cuda, "gradients must be CUDA tensors")
    if any([t.dtype != dtype for t in tensors]):
        raise TypeError("the gradients of one call must have one type")
    _need(all([t.device == device for t in tensors]), "the gradients of one call must be on one device")
    return _DTYPES[dtype], device


def _pointers(ptrs: Sequence[int]):
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


def _workspace(device: torch.device) -> torch.Tensor:
    return torch.empty(PSGD_GRAD_NORM_WORKSPACE, dtype=torch.uint8, device=device)


def grad_norm(tensors: Sequence[torch.Tensor]) -> torch.Tensor:
    """sqrt of the sum of squares of every value of ``tensors``: a float32
    scalar on the device.  One type for all (float32, bfloat16, float16); any
    strides whose values lie in equally spaced contiguous rows."""
    tensors = list(tensors)
    dtype, device = _one_type(tensors)
    ptrs, rows, cols, lds = _table("tensor", tensors)
    with torch.cuda.device(device):
        norm = torch.empty((), dtype=torch.float32, device=device)
        ws = _workspace(device)
        _check(lib().psgd_grad_norm(len(ptrs), _pointers(ptrs), _i64(rows), _i64(cols), _i64(lds), dtype,
                                    norm.data_ptr(), ws.data_ptr(), ws.numel(), _stream(device)))
    return norm


def clip_grad_norm(tensors: Sequence[torch.Tensor], max_norm: float,
                   out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """Scales ``tensors`` by ``min(1, max_norm / (norm + 1e-6))`` and returns
    their norm before that (a float32 scalar on the device; the host does not
    wait).  In place, or into ``out``: tensors of the same shapes and order of
    dimensions, whose memory overlaps no gradient."""
    tensors = list(tensors)
    dtype, device = _one_type(tensors)
    ptrs, rows, cols, lds = _table("tensor", tensors)
    if out is None:
        optrs, old = ptrs, lds
    else:
        out = list(out)
        _need(len(out) == len(tensors), f"out has {len(out)} tensors, {len(tensors)} are needed")
        _need(all([o.shape == t.shape for o, t in zip(out, tensors)]), "out must have the gradients' shapes")
        odt, odev = _one_type(out)
        if odt != dtype:
            raise TypeError("out must have the gradients' type")
        _need(odev == device, "out must be on the gradients' device")
        optrs, orows, ocols, old = _table("out", out)
        if not (all([t.is_contiguous() for t in tensors]) and all([o.is_contiguous() for o in out])):
            optrs, rows, cols, lds, old = _pair(tensors, out)
    with torch.cuda.device(device):
        norm = torch.empty((), dtype=torch.float32, device=device)
        ws = _workspace(device)
        _check(lib().psgd_clip_grad_norm(len(ptrs), _pointers(ptrs), _pointers(optrs), _i64(rows), _i64(cols),
                                         _i64(lds), _i64(old), dtype, float(max_norm), norm.data_ptr(), ws.data_ptr(),
                                         ws.numel(), _stream(device)))
    return norm


def _pair(tensors, out):
    """The tables of gradients and outputs whose strides differ: both as the rows they share."""
    optrs, rows, cols, lds, old = [], [], [], [], []
    for i, (t, o) in enumerate(zip(tensors, out)):
        optrs.append(o.data_ptr())
        if t.numel() == 0:
            a = b = (0, 0, 0)
        else:
            order = sorted((d for d in range(t.dim()) if t.size(d) != 1), key=lambda d: (t.stride(d), d))
            a, b = _two_dims(t), _two_dims(o)
            same = order == sorted(order, key=lambda d: (o.stride(d), d))
            if a is None or b is None or not same:
                raise ValueError(f"out {i}: strides {tuple(o.stride())} do not match the gradient's "
                                 f"{tuple(t.stride())}")
            if a[:2] != b[:2]:  # one of them is contiguous: the other's rows
                r, c = max(a[0], b[0]), min(a[1], b[1])
                a = (r, c, a[2] if a[0] > 1 else c)
                b = (r, c, b[2] if b[0] > 1 else c)
        rows.append(a[0])
        cols.append(a[1])
        lds.append(a[2])
        old.append(b[2])
    return optrs, rows, cols, lds, old


class GradientLayout:
    """The packed gradient buffer of a layer set, without a compression context.

    ``shapes`` lists (n, m) per layer, m == 0 for a vector, as for
    ``PowerSGD``; ``offsets``, ``lds`` and ``total`` describe the buffer.
    """

    def __init__(self, shapes: Sequence[Tuple[int, int]]):
        self.shapes = [(int(a), int(b)) for a, b in shapes]
        self.offsets, self.lds, self.total = psgd_plan_layout(self.shapes)
        self._n, self._m = _i64([s[0] for s in self.shapes]), _i64([s[1] for s in self.shapes])

    def layer_view(self, buf: torch.Tensor, layer: int) -> torch.Tensor:
        n, m = self.shapes[layer]
        off, ld = self.offsets[layer], self.lds[layer]
        if m == 0:
            return buf[off:off + n]
        return buf[off:off + n * ld].view(n, ld)[:, :m]

    def experts_view(self, buf: torch.Tensor, first: int, experts: int) -> torch.Tensor:
        """``experts`` equal matrix layers from layer ``first`` on, as one (experts, n, m) tensor."""
        n, m = self.shapes[first]
        _need(m > 0 and all(s == (n, m) for s in self.shapes[first:first + experts])
              and first + experts <= len(self.shapes), f"layers {first}.. are not {experts} equal matrices")
        ld = self.lds[first]
        return buf[self.offsets[first]:self.offsets[first] + experts * n * ld].view(experts, n, ld)[:, :, :m]

    def _buffers(self, name: str, bufs: Sequence[torch.Tensor]):
        _need(len(bufs) >= 1, f"{name} is empty")
        for b in bufs:
            if b.dtype != torch.float32:
                raise TypeError(f"{name} must be packed float32 buffers (got {b.dtype})")
            _need(b.is_cuda and b.device == bufs[0].device and b.is_contiguous() and b.numel() >= self.total,
                  f"{name} must be contiguous CUDA buffers of {self.total} values on one device")
        return _pointers([b.data_ptr() for b in bufs])

    def grad_norm(self, grads: Sequence[torch.Tensor]) -> torch.Tensor:
        """The norm of each packed buffer (float32 vector); padding does not count."""
        ptrs = self._buffers("grads", grads)
        device = grads[0].device
        with torch.cuda.device(device):
            norms = torch.empty(len(grads), dtype=torch.float32, device=device)
            ws = _workspace(device)
            _check(lib().psgd_packed_grad_norm(len(self.shapes), self._n, self._m, len(grads), ptrs, norms.data_ptr(),
                                               ws.data_ptr(), ws.numel(), _stream(device)))
        return norms

    def clip_grad_norm(self, grads: Sequence[torch.Tensor], max_norm: float,
                       out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
        """Clips each packed buffer by its own norm, in place or into ``out``
        (padding is left alone), and returns the norms before that."""
        ptrs = self._buffers("grads", grads)
        optrs = ptrs if out is None else self._buffers("out", out)
        _need(len(optrs) == len(ptrs), f"out has {len(optrs)} buffers, {len(ptrs)} are needed")
        device = grads[0].device
        _need(out is None or out[0].device == device, "out must be on the gradients' device")
        with torch.cuda.device(device):
            norms = torch.empty(len(grads), dtype=torch.float32, device=device)
            ws = _workspace(device)
            _check(lib().psgd_packed_clip_grad_norm(len(self.shapes), self._n, self._m, len(grads), ptrs, optrs,
                                                    float(max_norm), norms.data_ptr(), ws.data_ptr(), ws.numel(),
                                                    _stream(device)))
        return norms
