"""Products with packed weights: the tensor forms of the uzip_weight_* and
uzip_*linear* entry points (include/uzip.h).

A bf16 weight that arrived compressed is packed once with ``pack_weight`` and
then multiplied from its packed form: ``linear`` (bias, activation, gate and
residual in its epilogue), ``grouped_linear`` (rows grouped by expert, ragged)
and ``linear_cross_entropy`` (the loss over a large vocabulary, the logits
never stored), each with its gradients.  Shapes, types and the rounding of
each result are those the header states; argument errors raise ValueError or
TypeError before anything is launched.

A call with ``stream=`` runs there, and what it allocates is that stream's
memory.  The caller orders the streams: the arguments have to be ready for
``stream``, and be kept until its work is done, and the results are not ready
for the current stream until that waits for it.

Nothing is recorded for autograd.  Where it would be expected to be (an
argument requires grad and gradients are enabled) the forward calls raise
ValueError: wrap the pair of calls in a ``torch.autograd.Function``, or call
them under ``torch.no_grad()``.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import (UZIP_BF16, UZIP_FP32, UZIP_OK, _check, lib, workspace)

_vp, _sz, _u32, _i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_int64

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5}


class uzip_weight(ctypes.Structure):
    _fields_ = [("data", _vp), ("bytes", _sz), ("matrices", _sz), ("rows", _sz), ("cols", _sz), ("gated", _u32),
                ("reserved", _u32)]


class uzip_linear_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_stride", _sz), ("tokens", _sz), ("offsets", _vp), ("bias", _vp), ("residual", _vp),
                ("residual_stride", _sz), ("y", _vp), ("y_stride", _sz), ("preact", _vp), ("preact_stride", _sz),
                ("bias_dtype", _u32), ("y_dtype", _u32), ("act", _u32), ("preact_dtype", _u32), ("clear_rest", _u32),
                ("reserved", _u32)]


class uzip_linear_backward_args(ctypes.Structure):
    _fields_ = [("dy", _vp), ("dy_stride", _sz), ("x", _vp), ("x_stride", _sz), ("preact", _vp), ("preact_stride", _sz),
                ("tokens", _sz), ("offsets", _vp), ("dx", _vp), ("dx_stride", _sz), ("dw", _vp), ("dbias", _vp),
                ("dy_dtype", _u32), ("dbias_dtype", _u32), ("act", _u32), ("preact_dtype", _u32), ("clear_rest", _u32),
                ("reserved", _u32)]


class uzip_loss_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_stride", _sz), ("tokens", _sz), ("target", _vp), ("ignore_index", _i64), ("loss", _vp),
                ("lse", _vp), ("dloss", _vp), ("dx", _vp), ("dx_stride", _sz), ("dw", _vp)]


def _declare(L):
    i32, W = ctypes.c_int, ctypes.POINTER(uzip_weight)
    F, B, S = (ctypes.POINTER(t) for t in (uzip_linear_args, uzip_linear_backward_args, uzip_loss_args))
    for name in ("uzip_weight_max_size", "uzip_weight_workspace_size"):
        getattr(L, name).restype = _sz
        getattr(L, name).argtypes = [_sz, _sz, _sz, _u32]
    L.uzip_weight_pack.restype = i32
    L.uzip_weight_pack.argtypes = [_vp, _sz, _sz, _sz, _sz, _sz, _u32, _vp, _sz, _vp, _vp, _sz, _vp]
    L.uzip_weight_unpack.restype = i32
    L.uzip_weight_unpack.argtypes = [W, _vp, _sz, _sz, _vp]
    for name, args in (("uzip_linear", F), ("uzip_linear_backward", B), ("uzip_linear_cross_entropy", S),
                       ("uzip_linear_cross_entropy_backward", S), ("uzip_grouped_linear", F),
                       ("uzip_grouped_linear_backward", B)):
        getattr(L, name).restype = i32
        getattr(L, name).argtypes = [W, args, _vp, _sz, _vp]
        size = name + "_workspace_size"
        if "grouped" not in name:
            getattr(L, size).restype = _sz
            getattr(L, size).argtypes = [W, args]
    L._weights_declared = True
    return L


def _lib():
    L = lib()
    return L if getattr(L, "_weights_declared", False) else _declare(L)


# ---- the C entry points, same names and arguments ----------------------------
def uzip_weight_max_size(matrices, rows, cols, gated=0) -> int:
    return _lib().uzip_weight_max_size(matrices, rows, cols, gated)


def uzip_weight_workspace_size(matrices, rows, cols, gated=0) -> int:
    return _lib().uzip_weight_workspace_size(matrices, rows, cols, gated)


def uzip_weight_pack(d_in, matrices, rows, cols, row_stride, matrix_stride, gated, d_out, out_capacity, d_out_size,
                     d_workspace, workspace_bytes, stream) -> int:
    return _lib().uzip_weight_pack(d_in, matrices, rows, cols, row_stride, matrix_stride, gated, d_out, out_capacity,
                                   d_out_size, d_workspace, workspace_bytes, stream)


def uzip_weight_unpack(weight, d_out, row_stride, matrix_stride, stream) -> int:
    return _lib().uzip_weight_unpack(ctypes.byref(weight), d_out, row_stride, matrix_stride, stream)


def _ref(s):
    return None if s is None else ctypes.byref(s)


def uzip_linear_workspace_size(weight, args) -> int:
    return _lib().uzip_linear_workspace_size(_ref(weight), _ref(args))


def uzip_linear(weight, args, d_workspace, workspace_bytes, stream) -> int:
    return _lib().uzip_linear(_ref(weight), _ref(args), d_workspace, workspace_bytes, stream)


def uzip_grouped_linear(weight, args, d_workspace, workspace_bytes, stream) -> int:
    return _lib().uzip_grouped_linear(_ref(weight), _ref(args), d_workspace, workspace_bytes, stream)


def uzip_linear_backward_workspace_size(weight, args) -> int:
    return _lib().uzip_linear_backward_workspace_size(_ref(weight), _ref(args))


def uzip_linear_backward(weight, args, d_workspace, workspace_bytes, stream) -> int:
    return _lib().uzip_linear_backward(_ref(weight), _ref(args), d_workspace, workspace_bytes, stream)


def uzip_grouped_linear_backward(weight, args, d_workspace, workspace_bytes, stream) -> int:
    return _lib().uzip_grouped_linear_backward(_ref(weight), _ref(args), d_workspace, workspace_bytes, stream)


def uzip_linear_cross_entropy_workspace_size(weight, args) -> int:
    return _lib().uzip_linear_cross_entropy_workspace_size(_ref(weight), _ref(args))


def uzip_linear_cross_entropy(weight, args, d_workspace, workspace_bytes, stream) -> int:
    return _lib().uzip_linear_cross_entropy(_ref(weight), _ref(args), d_workspace, workspace_bytes, stream)


def uzip_linear_cross_entropy_backward_workspace_size(weight, args) -> int:
    return _lib().uzip_linear_cross_entropy_backward_workspace_size(_ref(weight), _ref(args))


def uzip_linear_cross_entropy_backward(weight, args, d_workspace, workspace_bytes, stream) -> int:
    return _lib().uzip_linear_cross_entropy_backward(_ref(weight), _ref(args), d_workspace, workspace_bytes, stream)


# ---- tensors --------------------------------------------------------------------
class PackedWeight:
    """A losslessly packed bf16 weight (or stack of them) in device memory.
    ``data`` is the packed buffer, ``shape`` the weight's: [rows, cols] or
    [matrices, rows, cols]."""

    def __init__(self, data: torch.Tensor, shape, gated: bool):
        if not isinstance(data, torch.Tensor) or data.dtype is not torch.uint8 or not data.is_contiguous():
            raise TypeError("a PackedWeight's data is a contiguous uint8 tensor")
        self.data = data
        self.shape = torch.Size(shape)
        self.gated = bool(gated)
        self.device = data.device
        matrices = self.shape[0] if len(self.shape) == 3 else 1
        self._c = uzip_weight(data.data_ptr(), data.numel(), matrices, self.shape[-2], self.shape[-1], int(gated), 0)
        self._ref = ctypes.byref(self._c)

    @property
    def nbytes(self) -> int:
        return self.data.numel()

    def __repr__(self):
        return "PackedWeight(shape=%s, gated=%s, nbytes=%d, device=%s)" % (tuple(self.shape), self.gated, self.nbytes,
                                                                          self.device)


_here = contextlib.nullcontext()


def _on(device, stream=None):
    """Makes `device` current for a launch when it is not already, and `stream`
    if there is one: what is allocated meanwhile comes from that stream's
    memory, so that no work of another stream can still be using it."""
    if stream is not None:
        if stream.device != device:
            raise ValueError("stream is on %s, the weight on %s" % (stream.device, device))
        return torch.cuda.stream(stream)
    return _here if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _caller(device, stream):
    """The stream that results made on `stream` are handed to."""
    return None if stream is None else torch.cuda.current_stream(device)


def _share(stream, caller, new=(), given=()):
    """Tells the allocator of tensors that two streams use: `new` ones of
    `stream` that the caller gets, and `given` ones that `stream` works on."""
    if stream is None or stream == caller:
        return
    for t in new:
        if t is not None:
            t.record_stream(caller)
    for t in given:
        if t is not None:
            t.record_stream(stream)


def _stream_of(stream, device) -> int:
    """The stream's handle; without one that of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else int(stream.cuda_stream)


def _code(t: torch.dtype, what: str) -> int:
    if t is torch.bfloat16:
        return UZIP_BF16
    if t is torch.float32:
        return UZIP_FP32
    raise TypeError("%s must be bfloat16 or float32, not %s" % (what, t))


def _matrix(t: torch.Tensor, what: str, rows: int, cols: int, device, dtype=torch.bfloat16):
    """Checks a [rows, cols] argument with contiguous rows and returns its stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor, not %s" % (what, type(t).__name__))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, not %s" % (what, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, the weight on %s" % (what, t.device, device))
    if t.shape != (rows, cols):
        raise ValueError("%s must have shape [%d, %d], not %s" % (what, rows, cols, list(t.shape)))
    if rows == 0:
        return cols
    s0, s1 = t.stride()
    if (s1 != 1 and cols > 1) or (rows > 1 and s0 < cols):
        raise ValueError("%s needs contiguous rows that do not overlap (stride(-1) == 1, stride(0) >= %d)" % (what, cols))
    return s0 if rows > 1 else max(s0, cols)


def _weight(w, what: str, dims: int):
    if not isinstance(w, PackedWeight):
        raise TypeError("%s takes a PackedWeight (see pack_weight), not %s" % (what, type(w).__name__))
    if len(w.shape) != dims:
        raise ValueError("%s takes a %s, not one of shape %s" % (
            what, "single packed matrix" if dims == 2 else "packed stack [matrices, rows, cols]", tuple(w.shape)))
    return w


def _act(act: str, w: PackedWeight) -> int:
    if act not in ACTIVATIONS:
        raise ValueError("act must be one of %s, not %r" % (", ".join(sorted(ACTIVATIONS)), act))
    if (act == "swiglu") != w.gated:
        raise ValueError("swiglu takes a weight packed with gated=True, and such a weight takes no other activation")
    return ACTIVATIONS[act]


def _offsets(offsets, w: PackedWeight):
    if not isinstance(offsets, torch.Tensor) or offsets.dtype is not torch.int32:
        raise TypeError("offsets must be an int32 tensor")
    if offsets.device != w.device or offsets.dim() != 1 or offsets.numel() != w.shape[0] + 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be %d contiguous values on %s" % (w.shape[0] + 1, w.device))
    return offsets.data_ptr()


def _overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two matrices with contiguous rows share memory."""
    if 0 in (a.numel(), b.numel()) or a.device != b.device:
        return False
    wide = [t.shape[1] * t.element_size() for t in (a, b)]
    step = [t.stride(0) * t.element_size() if t.shape[0] > 1 else w for t, w in zip((a, b), wide)]
    first = [t.data_ptr() for t in (a, b)]
    end = [f + (t.shape[0] - 1) * s + w for f, t, s, w in zip(first, (a, b), step, wide)]
    if first[0] >= end[1] or first[1] >= end[0]:
        return False
    if step[0] == step[1] and a.shape[0] > 1 and b.shape[0] > 1:  # two slices of columns
        at = (first[0] - first[1]) % step[0]
        return not (at >= wide[1] and at + wide[0] <= step[0])
    return True


def _tokens(x, what: str) -> int:
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a tensor, not %s" % (what, type(x).__name__))
    if x.dim() != 2:
        raise ValueError("%s must be a matrix [tokens, cols], not of shape %s" % (what, list(x.shape)))
    return x.shape[0]


def _no_history(what: str, *tensors):
    """Refuses arguments whose gradient autograd is to record: the result would
    have no history, and the gradient would be missing without a word."""
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError("%s records nothing for autograd, and an argument requires grad: call it under torch.no_grad() "
                             "or from a torch.autograd.Function, and take the gradients from %s_backward" % (what, what))


def _call(name: str, fn, size, w, a, ws, stream):
    """Calls `fn` with the caller's workspace or a new one (made under
    `_on(device, stream)`): nothing is shared between calls."""
    ref, device = ctypes.byref(a), w.device
    if ws is None:
        need = size(w._ref, ref)
        ws = workspace(need, device) if need else None
    elif ws.dtype is not torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on %s" % device)
    st = fn(w._ref, ref, ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
            _stream_of(stream, device))
    if st != UZIP_OK:
        _check(st, "uzip_" + name)


def pack_weight(w: torch.Tensor, gated: bool = False, trim: bool = True, stream=None) -> PackedWeight:
    """Pack a bf16 device weight [rows, cols] or stack [matrices, rows, cols]
    without loss.  gated=True is for swiglu: the first half of each matrix's
    rows is the gate.  trim=True waits for the packed size and keeps only that
    many bytes; trim=False neither waits nor trims (the buffer then has the
    size of the worst case)."""
    if not isinstance(w, torch.Tensor) or w.dtype is not torch.bfloat16:
        raise TypeError("pack_weight packs bfloat16 tensors")
    if not w.is_cuda or w.dim() not in (2, 3):
        raise ValueError("pack_weight needs a device tensor [rows, cols] or [matrices, rows, cols]")
    if w.stride(-1) != 1 and w.shape[-1] > 1 or w.shape[-2] > 1 and w.stride(-2) < w.shape[-1]:
        raise ValueError("pack_weight needs contiguous rows that do not overlap")
    matrices = w.shape[0] if w.dim() == 3 else 1
    rows, cols = w.shape[-2:]
    cap = uzip_weight_max_size(matrices, rows, cols, int(gated))
    if cap == 0:
        raise ValueError("a weight of shape %s%s cannot be packed" % (list(w.shape), " (gated)" if gated else ""))
    caller = _caller(w.device, stream)
    with _on(w.device, stream):
        out = torch.empty(cap, dtype=torch.uint8, device=w.device)
        size = torch.empty(1, dtype=torch.int64, device=w.device)
        ws = workspace(uzip_weight_workspace_size(matrices, rows, cols, int(gated)), w.device)
        st = uzip_weight_pack(w.data_ptr(), matrices, rows, cols, max(w.stride(-2), cols), w.stride(0) if w.dim() == 3 else 0,
                              int(gated), out.data_ptr(), cap, size.data_ptr(), ws.data_ptr(), ws.numel(), _stream_of(stream, w.device))
        _check(st, "uzip_weight_pack")
        if trim:
            out = out[:int(size.item())].clone()
    if trim and stream is not None:
        caller.wait_stream(stream)
    _share(stream, caller, new=(out,))
    return PackedWeight(out, w.shape, gated)


def unpack_weight(w: PackedWeight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The bf16 weight back, bit for bit."""
    if not isinstance(w, PackedWeight):
        raise TypeError("unpack_weight takes a PackedWeight, not %s" % type(w).__name__)
    caller, given = _caller(w.device, stream), out
    with _on(w.device, stream):
        if out is None:
            out = torch.empty(tuple(w.shape), dtype=torch.bfloat16, device=w.device)
        elif out.dtype is not torch.bfloat16 or out.shape != w.shape or out.device != w.device or not out.is_contiguous():
            raise ValueError("out must be a contiguous bfloat16 tensor of shape %s on %s" % (tuple(w.shape), w.device))
        st = uzip_weight_unpack(w._c, out.data_ptr(), w.shape[-1], w.shape[-2] * w.shape[-1], _stream_of(stream, w.device))
        _check(st, "uzip_weight_unpack")
    _share(stream, caller, new=(out,) if given is None else (), given=(given,))
    return out


def _forward(what, w, x, offsets, bias, act, residual, out_dtype, return_preact, preact_dtype, out, ws, stream):
    grouped = what == "grouped_linear"
    w = _weight(w, what, 3 if grouped else 2)
    L = _lib()
    device, (rows, cols) = w.device, w.shape[-2:]
    tokens = _tokens(x, "x")
    x_stride = _matrix(x, "x", tokens, cols, device)
    act = _act(act, w)
    off = _offsets(offsets, w) if grouped else None
    width = rows // 2 if w.gated else rows
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    y_code = _code(out_dtype, "out_dtype")
    b = b_code = r = r_stride = 0
    if bias is not None:
        if not isinstance(bias, torch.Tensor):
            raise TypeError("bias must be a tensor, not %s" % type(bias).__name__)
        b_code = _code(bias.dtype, "bias")
        if bias.shape != ((w.shape[0], rows) if grouped else (rows,)) or bias.device != device or not bias.is_contiguous():
            raise ValueError("bias must be contiguous of shape %s on %s" % ([w.shape[0], rows] if grouped else [rows], device))
        b = bias.data_ptr()
    if residual is not None:
        r_stride = _matrix(residual, "residual", tokens, width, device, out_dtype)
        r = residual.data_ptr()
    z_code = _code(preact_dtype, "preact_dtype") if return_preact else 0
    clear = int(grouped and out is None)
    if out is not None:
        y_stride = _matrix(out, "out", tokens, width, device, out_dtype)
        if _overlap(out, x):
            raise ValueError("out must not overlap x")
        if residual is not None and _overlap(out, residual) and (
                out.data_ptr() != residual.data_ptr() or y_stride != r_stride):
            raise ValueError("out must be the residual itself or not overlap it")
    _no_history(what, x, bias, residual, out)
    caller, given = _caller(device, stream), out
    with _on(device, stream):
        if out is None:
            out = torch.empty((tokens, width), dtype=out_dtype, device=device)
            y_stride = width
        z = None
        if return_preact:  # (rows of no group: zero; the call itself clears them only together with a new output's)
            z = (torch.zeros if grouped and not clear else torch.empty)((tokens, rows), dtype=preact_dtype, device=device)
        if tokens:
            a = uzip_linear_args(x.data_ptr(), x_stride, tokens, off, b, r, r_stride, out.data_ptr(), y_stride,
                                 z.data_ptr() if return_preact else 0, rows, b_code, y_code, act, z_code, clear)
            _call(what, L.uzip_grouped_linear if grouped else L.uzip_linear, L.uzip_linear_workspace_size, w, a, ws, stream)
    _share(stream, caller, new=(out if given is None else None, z), given=(given, ws))
    return (out, z) if return_preact else out


def linear(x, weight: PackedWeight, bias=None, act: str = "none", residual=None, out_dtype=None,
           return_preact: bool = False, preact_dtype=torch.float32, out=None, ws=None, stream=None):
    """act(x W^T + bias) + residual for x [tokens, cols] bf16 and a packed
    weight [rows, cols]; the result [tokens, rows] ([tokens, rows / 2] for
    swiglu) is bf16, or out_dtype.  residual has the result's shape and type;
    out (the result's place) may be the residual, and must not overlap x.
    return_preact=True also returns x W^T + bias [tokens, rows], which
    linear_backward takes, in preact_dtype (in bf16 it takes half the memory and
    the gradients lose about as much as dz's own rounding costs them)."""
    return _forward("linear", weight, x, None, bias, act, residual, out_dtype, return_preact, preact_dtype, out, ws,
                    stream)


def grouped_linear(x, offsets, weight: PackedWeight, bias=None, act: str = "none", out_dtype=None,
                   return_preact: bool = False, preact_dtype=torch.float32, out=None, ws=None, stream=None):
    """`linear` for rows grouped by matrix: rows offsets[g] .. offsets[g + 1] - 1
    of x [tokens, cols] are multiplied with matrix g of a packed stack
    [matrices, rows, cols].  offsets: matrices + 1 ascending int32 values on
    the device.  bias: [matrices, rows].  Rows of no group are not written:
    zero in a new output and in the pre-activation, unchanged in `out`."""
    return _forward("grouped_linear", weight, x, offsets, bias, act, None, out_dtype, return_preact, preact_dtype, out, ws,
                    stream)


def _backward(what, w, dy, x, offsets, preact, act, need_x, need_weight, need_bias, bias_dtype, ws, stream):
    grouped = what == "grouped_linear_backward"
    w = _weight(w, what, 3 if grouped else 2)
    L = _lib()
    device, (rows, cols) = w.device, w.shape[-2:]
    tokens = _tokens(dy, "dy")
    a = uzip_linear_backward_args()
    a.act, a.tokens, a.dy_dtype = _act(act, w), tokens, _code(dy.dtype, "dy")
    a.dy_stride, a.dy = _matrix(dy, "dy", tokens, rows // 2 if w.gated else rows, device, dy.dtype), dy.data_ptr()
    if act != "none":
        if preact is None:
            raise ValueError("%s needs the pre-activation for %s (return_preact=True)" % (what, act))
        a.preact_dtype = _code(getattr(preact, "dtype", None), "preact")
        a.preact_stride, a.preact = _matrix(preact, "preact", tokens, rows, device, preact.dtype), preact.data_ptr()
    if need_weight:
        a.x_stride, a.x = _matrix(x, "x", tokens, cols, device), x.data_ptr()
    if grouped:
        a.offsets = _offsets(offsets, w)
    code = _code(bias_dtype, "bias_dtype")
    caller = _caller(device, stream)
    with _on(device, stream):
        dx = dw = db = None
        if need_x:
            dx = torch.empty((tokens, cols), dtype=torch.bfloat16, device=device)
            a.dx, a.dx_stride, a.clear_rest = dx.data_ptr(), cols, int(grouped)
        if need_weight:
            dw = torch.empty(w.shape, dtype=torch.bfloat16, device=device)
            a.dw = dw.data_ptr()
        if need_bias:
            db = torch.empty((w.shape[0], rows) if grouped else (rows,), dtype=bias_dtype, device=device)
            a.dbias, a.dbias_dtype = db.data_ptr(), code
        _call(what, L.uzip_grouped_linear_backward if grouped else L.uzip_linear_backward,
              L.uzip_linear_backward_workspace_size, w, a, ws, stream)
    _share(stream, caller, new=(dx, dw, db), given=(ws,))
    return dx, dw, db


def linear_backward(dy, x, weight: PackedWeight, preact=None, act: str = "none", need_x: bool = True,
                    need_weight: bool = True, need_bias: bool = False, bias_dtype=torch.bfloat16, ws=None, stream=None):
    """The gradients (dx, dw, dbias) of `linear`, None for those not needed;
    the residual's gradient is dy itself.  preact is what linear returned with
    return_preact=True (not needed for act "none"); x is needed for dw only."""
    return _backward("linear_backward", weight, dy, x, None, preact, act, need_x, need_weight, need_bias, bias_dtype, ws,
                     stream)


def grouped_linear_backward(dy, x, offsets, weight: PackedWeight, preact=None, act: str = "none", need_x: bool = True,
                            need_weight: bool = True, need_bias: bool = False, bias_dtype=torch.bfloat16, ws=None,
                            stream=None):
    """The gradients (dx, dw, dbias) of `grouped_linear`.  A group without rows
    has zero dw and dbias; dx of rows of no group is zero."""
    return _backward("grouped_linear_backward", weight, dy, x, offsets, preact, act, need_x, need_weight, need_bias,
                     bias_dtype, ws, stream)


def _vector(t, what: str, n: int, device, dtype) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError("%s must be a %s tensor" % (what, dtype))
    if t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be %d contiguous values on %s" % (what, n, device))
    return t.data_ptr()


def _loss_args(what, x, w, target, ignore_index):
    w = _weight(w, what, 2)
    if w.gated:
        raise ValueError("%s takes a weight that is not gated" % what)
    tokens = _tokens(x, "x")
    a = uzip_loss_args()
    a.x_stride, a.x, a.tokens = _matrix(x, "x", tokens, w.shape[1], w.device), x.data_ptr(), tokens
    a.target, a.ignore_index = _vector(target, "target", tokens, w.device, torch.int64), ignore_index
    return w, tokens, a


def linear_cross_entropy(x, weight: PackedWeight, target, ignore_index: int = -100, ws=None, stream=None):
    """(loss, lse), both fp32 [tokens]: the softmax cross entropy of the logits
    x W^T against int64 targets, and the logits' log-sum-exp, which the
    gradient takes.  The logits are not stored.  A token with ignore_index has
    loss 0; a target outside the vocabulary gives NaN."""
    w, tokens, a = _loss_args("linear_cross_entropy", x, weight, target, ignore_index)
    _no_history("linear_cross_entropy", x)
    L, device = _lib(), w.device
    caller = _caller(device, stream)
    with _on(device, stream):
        loss = torch.empty(tokens, dtype=torch.float32, device=device)
        lse = torch.empty(tokens, dtype=torch.float32, device=device)
        if tokens:
            a.loss, a.lse = loss.data_ptr(), lse.data_ptr()
            _call("linear_cross_entropy", L.uzip_linear_cross_entropy, L.uzip_linear_cross_entropy_workspace_size, w, a, ws,
                  stream)
    _share(stream, caller, new=(loss, lse), given=(ws,))
    return loss, lse


def linear_cross_entropy_backward(dloss, x, weight: PackedWeight, target, lse, ignore_index: int = -100,
                                  need_x: bool = True, need_weight: bool = True, ws=None, stream=None):
    """(dx, dw) of `linear_cross_entropy`, bf16, None for one not needed, given
    the losses' gradients dloss (fp32 [tokens]) and its lse.  Tokens that are
    ignored or have no such target leave no trace, whatever their x holds."""
    w, tokens, a = _loss_args("linear_cross_entropy_backward", x, weight, target, ignore_index)
    L, device = _lib(), w.device
    a.dloss = _vector(dloss, "dloss", tokens, device, torch.float32)
    a.lse = _vector(lse, "lse", tokens, device, torch.float32)
    caller = _caller(device, stream)
    with _on(device, stream):
        dx = dw = None
        if need_x:
            dx = torch.empty((tokens, w.shape[1]), dtype=torch.bfloat16, device=device)
            a.dx, a.dx_stride = dx.data_ptr(), w.shape[1]
        if need_weight:
            dw = torch.empty(w.shape, dtype=torch.bfloat16, device=device)
            a.dw = dw.data_ptr()
        _call("linear_cross_entropy_backward", L.uzip_linear_cross_entropy_backward,
              L.uzip_linear_cross_entropy_backward_workspace_size, w, a, ws, stream)
    _share(stream, caller, new=(dx, dw), given=(ws,))
    return dx, dw
