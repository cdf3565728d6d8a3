"""The operators beside the compression step, bound with ctypes.

* ``experts_forward``, ``experts_grad_input``, ``experts_grad_weight`` and the
  differentiable ``experts_linear``: matrix products grouped by expert, over
  rows sorted by expert with ragged group sizes.
* ``grad_norm``, ``clip_grad_norm`` and ``GradientLayout``: the global norm of
  a set of gradients, and clipping by it.

Every call checks its arguments, allocates its results with torch and enqueues
the library's kernels on torch's current stream; nothing waits for the device.
A tensor that another stream wrote has to be ordered before the call by the
caller, as for any torch operation.  A result in ``out`` must not overlap an
operand (clipping in place apart).
"""
from __future__ import annotations

import ctypes
import operator
import threading
from array import array
from contextlib import nullcontext
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

from .binding import (PSGD_BF16, PSGD_F16, PSGD_F32, PSGD_GRAD_NORM_WORKSPACE, PSGD_MAX_EXPERTS, _check, lib,
                      psgd_plan_layout)

_DTYPES = {torch.float32: PSGD_F32, torch.bfloat16: PSGD_BF16, torch.float16: PSGD_F16}
_HALF = {torch.bfloat16: PSGD_BF16, torch.float16: PSGD_F16}


def _stream(device: int) -> int:
    """torch's current stream of a device."""
    return torch._C._cuda_getCurrentRawStream(device)


def _on(device: int):
    """The device as the current one."""
    return nullcontext() if torch._C._cuda_getDevice() == device else torch.cuda.device(device)


# Workspaces, one per host thread, device and stream: calls on one stream run in
# order, and two threads never share one.  Larger ones belong to their call, and
# so do those of a call that a graph captures, which keeps its address.
_KEPT_BYTES = 16 << 20
_kept = threading.local()


def _workspace(device: int, stream: int, size: int) -> torch.Tensor:
    where = torch.device("cuda", device)
    if size > _KEPT_BYTES or torch._C._cuda_isCurrentStreamCapturing():
        return torch.empty(size, dtype=torch.uint8, device=where)
    kept = _kept.__dict__
    ws = kept.get((device, stream))
    if ws is None or ws.numel() < size:
        if len(kept) >= 64:
            kept.clear()
        ws = kept[(device, stream)] = torch.empty(max(size, PSGD_GRAD_NORM_WORKSPACE), dtype=torch.uint8, device=where)
    return ws


def _written(tensors) -> None:
    """Tells torch that the kernels write to tensors of the caller's, so that a
    backward pass over an earlier value of one stops with an error."""
    torch.autograd.graph.increment_version(tensors)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


# ------------------------------------------------------- expert products --

def _row_stride(name: str, shape, strides) -> int:
    """Row stride of the last two dimensions; their rows must be contiguous."""
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous (strides {strides})")
    return strides[-2] if shape[-2] > 1 else shape[-1]


def _experts_check(name: str, rows: torch.Tensor, offsets: torch.Tensor, second: str, other: torch.Tensor):
    """Checks what the three products share; (data type, experts, device)."""
    kind = rows.dtype
    dtype = _HALF.get(kind)
    if dtype is None:
        raise TypeError(f"{name} must be bfloat16 or float16 (got {kind})")
    if other.dtype is not kind:
        raise TypeError(f"{second} must have {name}'s type {kind} (got {other.dtype})")
    if offsets.dtype is not torch.int32:
        raise TypeError(f"offsets must be int32 (got {offsets.dtype})")
    device = rows.get_device()
    if device < 0 or other.get_device() != device or offsets.get_device() != device:
        raise ValueError(f"{name}, {second} and offsets must be CUDA tensors on one device")
    if rows.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions (got {tuple(rows.shape)})")
    if offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous vector of experts + 1 values")
    experts = offsets.numel() - 1
    if not 1 <= experts <= PSGD_MAX_EXPERTS:
        raise ValueError(f"offsets must have experts + 1 values, for 1 to {PSGD_MAX_EXPERTS} experts (got {experts + 1})")
    return dtype, experts, device


def _result_check(out: torch.Tensor, shape, dtype, device: int, name: str = "out") -> torch.Tensor:
    if out.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {out.dtype})")
    if out.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(out.shape)})")
    if out.get_device() != device:
        raise ValueError(f"{name} must be on the operands' device")
    return out


def _plain(at: int, ld: int, stride: int, count: int, cols: int) -> bool:
    """Whether an operand's rows can be read where they are."""
    return not (at | 2 * ld | 2 * stride) & 15 and ld >= cols and (count == 1 or (stride and stride % ld == 0))


# The library's rule for contractions that it sums in parts or segments (cut_of),
# so that the common call need not ask it for a workspace's size.
_PAIRS, _PART, _LONG = 76, 16, 96         # pairs of CTAs; blocks of 64 values of a part, and of a long contraction
_MOST = {PSGD_F16: 512, PSGD_BF16: 4096}  # blocks in one piece at most
_MOST_WEIGHTS = 1024                      # the same for the weight gradient


def _rows_in_one_piece(dtype: int, rows: int, experts: int, side: int, depth: int) -> bool:
    """Whether experts_forward or experts_grad_input needs no room for sums."""
    blocks, tiles = (depth + 63) // 64, (side + 255) // 256 * (rows // 256 + min(experts, rows))
    return blocks < _LONG or (blocks <= _MOST[dtype] and tiles > _PAIRS // 2)


def _weights_in_one_piece(rows: int, experts: int, n: int, k: int) -> bool:
    """Whether experts_grad_weight needs none."""
    blocks, tiles = (rows + 63) // 64, (n + 255) // 256 * ((k + 255) // 256)
    segment = max(_PART, -(-3 * tiles * blocks // (2 * _PAIRS)))
    if blocks <= _MOST_WEIGHTS:
        return blocks <= segment or (blocks < _LONG and experts * tiles >= _PAIRS)
    exact, size = _MOST_WEIGHTS, n * ((k + 3) // 4) * 16
    room = (rows * (n + k) * 2 + experts * n * k * 4) // 4
    while exact < blocks and ((blocks + blocks // exact) // exact + blocks // exact + 1) * size > room:
        exact *= 2
    return blocks <= min(segment, exact)


def _workspace_bytes(op: int, rows, experts, n, k, a, lda, b, ldb, b_stride) -> int:
    size = ctypes.c_size_t()
    _check(lib().psgd_experts_workspace(op, rows, experts, n, k, a, lda, b, ldb, b_stride, ctypes.byref(size)))
    return size.value


def _rows_times_weights(op: int, name: str, rows: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                        out: Optional[torch.Tensor]) -> torch.Tensor:
    """experts_forward (op 0) and experts_grad_input (op 1)."""
    dtype, experts, device = _experts_check(name, rows, offsets, "w", w)
    wshape, rshape = w.shape, rows.shape
    if len(wshape) != 3 or wshape[0] != experts:
        raise ValueError(f"w must be ({experts}, n, k) (got {tuple(wshape)})")
    _, n, k = wshape
    count, depth = rshape
    if depth != (n if op else k):
        raise ValueError(f"{name} has {depth} columns, w is {n} x {k}")
    wstrides = w.stride()
    ld, ldw, stride = _row_stride(name, rshape, rows.stride()), _row_stride("w", wshape, wstrides), wstrides[0]
    shape = (count, k if op else n)
    y = rows.new_empty(shape) if out is None else _result_check(out, shape, rows.dtype, device)
    ldy = shape[1] if out is None else _row_stride("out", shape, y.stride())
    a, b = rows.data_ptr(), w.data_ptr()
    # the common case needs no workspace
    if _plain(a, ld, 0, 1, depth) and _plain(b, ldw, stride, experts, k) and _rows_in_one_piece(
            dtype, count, experts, shape[1], depth):
        size = 0
    else:
        size = _workspace_bytes(op, count, experts, n, k, a, ld, b, ldw, stride)
    f = lib().psgd_experts_grad_input if op else lib().psgd_experts_forward
    with _on(device):
        stream = _stream(device)
        ws = _workspace(device, stream, size) if size else None
        _check(f(count, experts, n, k, dtype, a, ld, b, ldw, stride, offsets.data_ptr(), y.data_ptr(), ldy,
                 ws.data_ptr() if size else None, size, stream))
    if out is not None:
        _written((out,))
    return y


def _recorded(out: Optional[torch.Tensor], a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether torch's autograd is to record a product of a and b."""
    if not (torch.is_grad_enabled() and (a.requires_grad or b.requires_grad)):
        return False
    if out is not None:
        raise RuntimeError("a result in out= cannot be differentiated, and an operand requires a gradient: detach it, "
                           "or call under torch.no_grad()")
    return True


def experts_sync() -> None:
    """Waits for the current stream; raises if a product's kernel on the device
    gave up one of its bounded waits since this thread's last call for the
    stream, or its first product there (none is expected to).  Without it, the
    next product after an abandoned one raises."""
    _check(lib().psgd_experts_sync(torch.cuda.current_stream().cuda_stream))


def experts_forward(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``y[t] = w[e(t)] @ x[t]`` for rows sorted by expert.

    ``x`` (rows, k) and ``w`` (experts, n, k) are bfloat16 or float16;
    ``offsets`` (experts + 1, int32, on the device) gives each expert's rows
    ``offsets[e]:offsets[e + 1]``.  Rows of no expert give zeros.  Sums are
    float32, rounded once to the operands' type.  torch differentiates the
    result; one that goes into ``out`` it cannot, so operands that require a
    gradient are refused there, as by torch's own functions.
    """
    if _recorded(out, x, w):
        return _ExpertsLinear.apply(x, w, offsets, None, False, None)
    return _rows_times_weights(0, "x", x, w, offsets, out)


def experts_grad_input(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``dx[t] = w[e(t)].T @ dy[t]``: the gradient of ``experts_forward`` in x.

    ``dy`` (rows, n), ``w`` (experts, n, k), ``offsets`` as in the forward
    product; the result is (rows, k), and differentiable in the same way.
    """
    if _recorded(out, dy, w):
        return _ExpertsGradInput.apply(dy, w, offsets)
    return _rows_times_weights(1, "dy", dy, w, offsets, out)


def experts_grad_weight(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``dw[e] = dy[rows of e].T @ x[rows of e]``: the gradient in w.

    The result (experts, n, k) is float32, the type the compression step
    takes; ``out`` may be a strided view of a packed gradient buffer (see
    ``GradientLayout.experts_view``), or have the operands' type.  An expert
    without rows gets zeros.  torch does not differentiate it further, whatever
    the operands require.
    """
    dtype, experts, device = _experts_check("dy", dy, offsets, "x", x)
    rows, n = dy.shape
    if x.dim() != 2 or x.shape[0] != rows:
        raise ValueError(f"x must have dy's {rows} rows (got {tuple(x.shape)})")
    k = x.shape[1]
    ldy, ldx = _row_stride("dy", dy.shape, dy.stride()), _row_stride("x", x.shape, x.stride())
    shape = (experts, n, k)
    if out is None:
        odt = PSGD_F32
        dw = dy.new_empty(shape, dtype=torch.float32)
        ldw, stride = k, n * k
    else:
        same = out.dtype is dy.dtype
        odt = dtype if same else PSGD_F32
        dw = _result_check(out, shape, dy.dtype if same else torch.float32, device)
        strides = dw.stride()
        ldw, stride = _row_stride("out", shape, strides), strides[0]
    a, b = dy.data_ptr(), x.data_ptr()
    if _plain(a, ldy, 0, 1, n) and _plain(b, ldx, 0, 1, k) and _weights_in_one_piece(rows, experts, n, k):
        size = 0  # as above
    else:
        size = _workspace_bytes(2, rows, experts, n, k, a, ldy, b, ldx, 0)
    with _on(device):
        on = _stream(device)
        ws = _workspace(device, on, size) if size else None
        _check(lib().psgd_experts_grad_weight(rows, experts, n, k, dtype, a, ldy, b, ldx, offsets.data_ptr(), odt,
                                              dw.data_ptr(), ldw, stride, ws.data_ptr() if size else None, size, on))
    if out is not None:
        _written((out,))
    return dw


# The weight gradients that the running backward passes have written: pass ->
# address -> (layout, stream).  The engine tells of a pass's end.
_passes = {}
_passes_lock = threading.Lock()


def _torch_stream(device: torch.device) -> torch.cuda.Stream:
    return torch.cuda.current_stream(device)


def _written_before(buf: torch.Tensor) -> bool:
    """Notes a write of the running backward pass; whether the buffer had one
    before, behind which the current stream then is."""
    task, stream = torch._C._current_graph_task_id(), _torch_stream(buf.device)
    layout = (buf.shape, buf.stride(), buf.dtype)
    with _passes_lock:
        if task not in _passes:
            while len(_passes) >= 64:  # of passes that ended in an exception
                _passes.pop(next(iter(_passes)))
            _passes[task] = {}
            torch.autograd.Variable._execution_engine.queue_callback(lambda: _end_of_pass(task))
        written = _passes[task]
        before = written.get(buf.data_ptr())
        written[buf.data_ptr()] = layout, stream
    if before is None:
        return False
    if before[0] != layout:
        raise ValueError("weight_grad: one backward pass writes matrices of unlike layouts to one address")
    if before[1] != stream:
        stream.wait_stream(before[1])
    return True


def _end_of_pass(task: int) -> None:
    """What the pass wrote on other streams is there for the caller's."""
    with _passes_lock:
        written = _passes.pop(task, {})
    for _, stream in written.values():
        caller = _torch_stream(stream.device)
        if caller != stream:
            caller.wait_stream(stream)


class _ExpertsLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, weight_grad, accumulate, anchor):
        ctx.save_for_backward(x, w, offsets)
        ctx.weight_grad = weight_grad
        ctx.accumulate = accumulate
        return experts_forward(x, w, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx = experts_grad_input(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw, buf = None, ctx.weight_grad
        if buf is not None:
            if _written_before(buf) or ctx.accumulate:
                buf.add_(experts_grad_weight(dy, x, offsets))  # float32, rounded once more to a 16-bit buffer
            else:
                experts_grad_weight(dy, x, offsets, out=buf)
        elif ctx.needs_input_grad[1]:
            dw = experts_grad_weight(dy, x, offsets, out=torch.empty_like(w, memory_format=torch.contiguous_format))
        return dx, dw, None, None, None, None


class _ExpertsGradInput(torch.autograd.Function):
    @staticmethod
    def forward(ctx, dy, w, offsets):
        ctx.save_for_backward(dy, w, offsets)
        return experts_grad_input(dy, w, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        dy, w, offsets = ctx.saved_tensors
        g = g.contiguous()
        ddy = experts_forward(g, w, offsets) if ctx.needs_input_grad[0] else None
        dw = None
        if ctx.needs_input_grad[1]:
            dw = experts_grad_weight(dy, g, offsets, out=torch.empty_like(w, memory_format=torch.contiguous_format))
        return ddy, dw, None


def experts_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                   weight_grad: Optional[torch.Tensor] = None, accumulate: bool = False) -> torch.Tensor:
    """``experts_forward`` whose weight gradient may go where the caller wants it.

    With ``weight_grad`` (experts, n, k; float32 or w's type) the backward
    pass writes the weight gradient there -- for instance into a packed buffer
    of the compression step -- and leaves ``w.grad`` alone.  It does so whether
    or not x or w require a gradient: the result then does.

    A backward pass gives the buffer its whole gradient: the first use of the
    buffer overwrites what was there, further uses of it (a weight that the
    graph uses twice) add to that.  With ``accumulate`` every use adds, for
    several backward passes into a buffer that the caller clears.  (A backward
    pass inside another, as of a reentrant checkpoint, is one of its own.)
    """
    anchor = None
    if weight_grad is not None and torch.is_grad_enabled():
        dtype = weight_grad.dtype if weight_grad.dtype is w.dtype else torch.float32
        _result_check(weight_grad, w.shape, dtype, w.get_device(), "weight_grad")
        if not (x.requires_grad or w.requires_grad):  # else torch would leave the backward pass out
            anchor = torch.empty(0, requires_grad=True)
    return _ExpertsLinear.apply(x, w, offsets, weight_grad, accumulate, anchor)


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


def _rows_table(name: str, tensors: Sequence[torch.Tensor]):
    """Rows, columns and row strides of tensors that are not all contiguous."""
    rows, cols, lds = [], [], []
    for i, t in enumerate(tensors):
        shape = (0, 0, 0) if t.numel() == 0 else _two_dims(t)
        if shape is None:
            raise ValueError(f"{name} {i}: values must lie in equally spaced contiguous rows (shape "
                             f"{tuple(t.shape)}, strides {tuple(t.stride())})")
        rows.append(shape[0])
        cols.append(shape[1])
        lds.append(shape[2])
    return rows, cols, lds


# per-tensor lookups of a list, without a Python frame or bytecode for each
_dtype_of = operator.attrgetter("dtype")
_device_of = torch.Tensor.get_device
_address_of = torch.Tensor.data_ptr
_length_of = torch.Tensor.numel
_contiguous = torch.Tensor.is_contiguous


def _one_type(tensors: Sequence[torch.Tensor]) -> Tuple[int, int]:
    """Data type and device that all tensors share."""
    if not tensors:
        raise ValueError("the list of tensors is empty")
    types = set(map(_dtype_of, tensors))
    if len(types) > 1:
        raise TypeError("the gradients of one call must have one type")
    first = types.pop()
    if first not in _DTYPES:
        raise TypeError(f"gradients must be float32, bfloat16 or float16 (got {first})")
    devices = set(map(_device_of, tensors))
    device = devices.pop()
    if devices or device < 0:
        raise ValueError("the gradients of one call must be CUDA tensors on one device")
    return _DTYPES[first], device


# the C entries' tables: int64 (addresses too), passed by address
def _ints(values) -> array:
    return array("q", list(values))  # a list first: an array grows slower


def _at(table: Optional[array]) -> Optional[int]:
    return None if table is None else table.buffer_info()[0]


def _once(name: str, tensors: Sequence[torch.Tensor], ptrs: list) -> None:
    """Refuses memory that clipping would scale twice: in its second read, a
    tile of one tensor may or may not be scaled by the other already."""
    if len(set(ptrs)) < len(ptrs):
        first = {}
        for i, t in enumerate(tensors):
            if t.numel() and first.setdefault(ptrs[i], i) != i:
                raise ValueError(f"{name} {first[ptrs[i]]} and {i} are the same memory")


def grad_norm(tensors: Sequence[torch.Tensor]) -> torch.Tensor:
    """sqrt of the sum of squares of every value of ``tensors``: a float32
    scalar on the device.  One type for all (float32, bfloat16, float16); any
    strides whose values lie in equally spaced contiguous rows."""
    tensors = list(tensors)
    dtype, device = _one_type(tensors)
    if all(map(_contiguous, tensors)):
        rows = lds = None
        cols = _ints(map(_length_of, tensors))
    else:
        rows, cols, lds = map(_ints, _rows_table("tensor", tensors))
    ptrs = _ints(map(_address_of, tensors))
    with _on(device):
        norm = torch.empty((), dtype=torch.float32, device=tensors[0].device)
        stream = _stream(device)
        ws = _workspace(device, stream, PSGD_GRAD_NORM_WORKSPACE)
        _check(lib().psgd_grad_norm(len(tensors), _at(ptrs), _at(rows), _at(cols), _at(lds), dtype, norm.data_ptr(),
                                    ws.data_ptr(), PSGD_GRAD_NORM_WORKSPACE, stream))
    return norm


def clip_grad_norm(tensors: Sequence[torch.Tensor], max_norm: float,
                   out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """Scales ``tensors`` by ``min(1, max_norm / (norm + 1e-6))`` and returns
    their norm before that (a float32 scalar on the device; the host does not
    wait).  In place, or into ``out``: tensors of the same shapes and order of
    dimensions (where all are contiguous, of the same lengths), whose memory
    overlaps no gradient.  No two of the tensors written may overlap."""
    tensors = list(tensors)
    dtype, device = _one_type(tensors)
    flat = all(map(_contiguous, tensors))
    ptrs = list(map(_address_of, tensors))
    if out is None:
        outs, optrs = tensors, ptrs
    else:
        outs = list(out)
        _need(len(outs) == len(tensors), f"out has {len(outs)} tensors, {len(tensors)} are needed")
        odt, odev = _one_type(outs)
        if odt != dtype:
            raise TypeError("out must have the gradients' type")
        _need(odev == device, "out must be on the gradients' device")
        optrs = list(map(_address_of, outs))
        flat = flat and all(map(_contiguous, outs))
        if not flat or list(map(_length_of, outs)) != list(map(_length_of, tensors)):
            _need([o.shape for o in outs] == [t.shape for t in tensors], "out must have the gradients' shapes")
    _once("tensors" if out is None else "out tensors", outs, optrs)
    ptrs = array("q", ptrs)
    optrs = ptrs if out is None else array("q", optrs)
    if flat:
        rows = lds = old = None
        cols = _ints(map(_length_of, tensors))
    elif out is None:
        rows, cols, lds = map(_ints, _rows_table("tensor", tensors))
        old = lds
    else:
        rows, cols, lds, old = map(_ints, _pair(tensors, outs))
    with _on(device):
        norm = torch.empty((), dtype=torch.float32, device=tensors[0].device)
        stream = _stream(device)
        ws = _workspace(device, stream, PSGD_GRAD_NORM_WORKSPACE)
        _check(lib().psgd_clip_grad_norm(len(tensors), _at(ptrs), _at(optrs), _at(rows), _at(cols), _at(lds), _at(old),
                                         dtype, float(max_norm), norm.data_ptr(), ws.data_ptr(),
                                         PSGD_GRAD_NORM_WORKSPACE, stream))
    _written(outs)
    return norm


def _pair(tensors, out):
    """The tables of gradients and outputs whose strides differ: both as the rows they share."""
    rows, cols, lds, old = [], [], [], []
    for i, (t, o) in enumerate(zip(tensors, out)):
        if t.numel() == 0:
            a = b = (0, 0, 0)
        else:
            order = sorted((d for d in range(t.dim()) if t.size(d) != 1), key=lambda d: (t.stride(d), d))
            a, b = _two_dims(t), _two_dims(o)
            same = order == sorted(order, key=lambda d: (o.stride(d), d))
            if a is None or b is None or not same:
                raise ValueError(f"out {i}: strides {tuple(o.stride())} do not match the gradient's "
                                 f"{tuple(t.stride())}")
            if a[:2] != b[:2]:  # where one of them is contiguous, the other's rows
                if a[0] > 1 and b[0] > 1:
                    raise ValueError(f"out {i}: strides {tuple(o.stride())} do not match the gradient's "
                                     f"{tuple(t.stride())}")
                r, c = max(a[0], b[0]), min(a[1], b[1])
                a = (r, c, a[2] if a[0] > 1 else c)
                b = (r, c, b[2] if b[0] > 1 else c)
        rows.append(a[0])
        cols.append(a[1])
        lds.append(a[2])
        old.append(b[2])
    return rows, cols, lds, old


class GradientLayout:
    """The packed gradient buffer of a layer set, without a compression context.

    ``shapes`` lists (n, m) per layer, m == 0 for a vector, as for
    ``PowerSGD``; ``offsets``, ``lds`` and ``total`` describe the buffer.
    """

    def __init__(self, shapes: Sequence[Tuple[int, int]]):
        self.shapes = [(int(a), int(b)) for a, b in shapes]
        self.offsets, self.lds, self.total = psgd_plan_layout(self.shapes)
        self._n, self._m = _ints([s[0] for s in self.shapes]), _ints([s[1] for s in self.shapes])

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

    def _buffers(self, name: str, bufs: Sequence[torch.Tensor], device: int = -1) -> list:
        """The addresses of packed buffers that pass the checks."""
        if not bufs:
            raise ValueError(f"{name} is empty")
        device = bufs[0].get_device() if device < 0 else device
        for b in bufs:
            if b.dtype is not torch.float32:
                raise TypeError(f"{name} must be packed float32 buffers (got {b.dtype})")
            if b.get_device() != device or device < 0 or not b.is_contiguous() or b.numel() < self.total:
                raise ValueError(f"{name} must be contiguous CUDA buffers of {self.total} values on one device")
        return [b.data_ptr() for b in bufs]

    def grad_norm(self, grads: Sequence[torch.Tensor]) -> torch.Tensor:
        """The norm of each packed buffer (float32 vector); padding does not count."""
        return self._run(grads, None, None)

    def clip_grad_norm(self, grads: Sequence[torch.Tensor], max_norm: float,
                       out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
        """Clips each packed buffer by its own norm, in place or into ``out``
        (padding is left alone), and returns the norms before that."""
        return self._run(grads, float(max_norm), out)

    def _run(self, grads, max_norm: Optional[float], out) -> torch.Tensor:
        ptrs = optrs = self._buffers("grads", grads)
        count, device = len(grads), grads[0].get_device()
        if out is not None:
            optrs = self._buffers("out", out, device)
            _need(len(optrs) == count, f"out has {len(optrs)} buffers, {count} are needed")
        src, dst = array("q", ptrs), array("q", optrs)
        with _on(device):
            norms = torch.empty(count, dtype=torch.float32, device=grads[0].device)
            stream = _stream(device)
            ws = _workspace(device, stream, PSGD_GRAD_NORM_WORKSPACE)
            if max_norm is None:
                _check(lib().psgd_packed_grad_norm(len(self.shapes), _at(self._n), _at(self._m), count, _at(src),
                                                   norms.data_ptr(), ws.data_ptr(), PSGD_GRAD_NORM_WORKSPACE,
                                                   stream))
            else:
                written = grads if out is None else out
                _once("grads" if out is None else "out buffers", written, optrs)
                _check(lib().psgd_packed_clip_grad_norm(len(self.shapes), _at(self._n), _at(self._m), count, _at(src),
                                                        _at(dst), max_norm, norms.data_ptr(), ws.data_ptr(),
                                                        PSGD_GRAD_NORM_WORKSPACE, stream))
                _written(written)
        return norms
