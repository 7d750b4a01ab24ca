"""The router and the expert layer on packed weights: the tensor forms of the
uzip_moe* entry points (include/uzip.h).

``moe_route`` turns a router's logits into a ``Routing``: the experts of each
token, their weights, and the rows grouped by expert.  ``moe`` is the layer
from packed experts; ``grouped_linear`` takes a routing's rows too
(``x[r.order // k]`` with ``r.offsets``).  ``moe_route_backward`` is the
router's gradient.  Streams, workspaces, errors and autograd are as for the
products with packed weights.
"""
from __future__ import annotations

import ctypes

import torch

from . import UZIP_OK, _check, lib, workspace
from .weights import (PackedWeight, _act, _caller, _code, _matrix, _no_history, _on, _overlap, _ref, _share, _stream_of,
                      _tokens, _weight, uzip_weight)

_vp, _sz, _u32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32

SCORES = {"softmax": 0, "sigmoid": 1}
MAX_EXPERTS = 1024
MAX_CHOSEN = 64


class uzip_moe_route_args(ctypes.Structure):
    _fields_ = [("logits", _vp), ("logits_stride", _sz), ("tokens", _sz), ("bias", _vp), ("experts", _vp), ("weights", _vp),
                ("order", _vp), ("offsets", _vp), ("dweights", _vp), ("dlogits", _vp), ("dlogits_stride", _sz),
                ("num_experts", _u32), ("k", _u32), ("logits_dtype", _u32), ("scores", _u32), ("renormalize", _u32),
                ("scale", ctypes.c_float)]


class uzip_moe_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_stride", _sz), ("tokens", _sz), ("weights", _vp), ("order", _vp), ("offsets", _vp),
                ("up_bias", _vp), ("down_bias", _vp), ("residual", _vp), ("residual_stride", _sz), ("y", _vp),
                ("y_stride", _sz), ("k", _u32), ("act", _u32), ("bias_dtype", _u32), ("y_dtype", _u32)]


def _lib():
    L = lib()
    if getattr(L, "_moe_declared", False):
        return L
    i32, W = ctypes.c_int, ctypes.POINTER(uzip_weight)
    R, M = ctypes.POINTER(uzip_moe_route_args), ctypes.POINTER(uzip_moe_args)
    L.uzip_moe_route_workspace_size.restype = _sz
    L.uzip_moe_route_workspace_size.argtypes = [R]
    L.uzip_moe_route.restype = i32
    L.uzip_moe_route.argtypes = [R, _vp, _sz, _vp]
    L.uzip_moe_route_backward.restype = i32
    L.uzip_moe_route_backward.argtypes = [R, _vp]
    L.uzip_moe_workspace_size.restype = _sz
    L.uzip_moe_workspace_size.argtypes = [W, W, M]
    L.uzip_moe.restype = i32
    L.uzip_moe.argtypes = [W, W, M, _vp, _sz, _vp]
    L._moe_declared = True
    return L


# ---- the C entry points, same names and arguments ----------------------------
def uzip_moe_route_workspace_size(args) -> int:
    return _lib().uzip_moe_route_workspace_size(_ref(args))


def uzip_moe_route(args, d_workspace, workspace_bytes, stream) -> int:
    return _lib().uzip_moe_route(_ref(args), d_workspace, workspace_bytes, stream)


def uzip_moe_route_backward(args, stream) -> int:
    return _lib().uzip_moe_route_backward(_ref(args), stream)


def uzip_moe_workspace_size(up, down, args) -> int:
    return _lib().uzip_moe_workspace_size(_ref(up), _ref(down), _ref(args))


def uzip_moe(up, down, args, d_workspace, workspace_bytes, stream) -> int:
    return _lib().uzip_moe(_ref(up), _ref(down), _ref(args), d_workspace, workspace_bytes, stream)


# ---- tensors --------------------------------------------------------------------
class Routing:
    """What a router decided for [tokens] of `num_experts` experts: ``experts``
    int32 and ``weights`` fp32 [tokens, k]; ``order`` int32 [tokens * k], the
    pairs token * k + place grouped by expert, each at most once; ``offsets``
    int32 [num_experts + 1], where each expert's begin.  A program may make one
    of its own tensors; where a token names an expert again ``moe`` adds both
    (``moe_route_backward`` is for routings of ``moe_route``)."""

    def __init__(self, experts, weights, order, offsets, scores="softmax", renormalize=True, scale=1.0):
        if experts.dim() != 2 or not 1 <= experts.shape[1] <= MAX_CHOSEN or not 2 <= offsets.numel() <= MAX_EXPERTS + 1:
            raise ValueError("a Routing is of up to %d experts, of which each token has 1 to %d, not of %s and %s" % (
                MAX_EXPERTS, MAX_CHOSEN, list(experts.shape), list(offsets.shape)))
        if scores not in SCORES:
            raise ValueError("scores must be softmax or sigmoid, not %r" % (scores,))
        for what, t, shape, dtype in (("experts", experts, experts.shape, torch.int32), ("weights", weights, experts.shape, torch.float32),
                                      ("order", order, (experts.numel(),), torch.int32), ("offsets", offsets, (offsets.numel(),), torch.int32)):
            if t.dtype is not dtype:
                raise TypeError("a Routing's %s must be %s, not %s" % (what, dtype, t.dtype))
            if t.shape != shape or t.device != experts.device or not t.is_contiguous():
                raise ValueError("a Routing's %s must be contiguous of shape %s on %s" % (what, list(shape), experts.device))
        self.experts, self.weights, self.order, self.offsets = experts, weights, order, offsets
        self.scores, self.renormalize, self.scale = scores, renormalize, scale
        self.tokens, self.k = experts.shape
        self.num_experts = offsets.shape[0] - 1
        self.device = experts.device

    def __repr__(self):
        return "Routing(tokens=%d, k=%d, num_experts=%d, device=%s)" % (self.tokens, self.k, self.num_experts, self.device)


def _workspace(need: int, ws, device):
    if ws is None:
        return workspace(need, device) if need else None
    if not isinstance(ws, torch.Tensor) or ws.dtype is not torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on %s" % device)
    return ws


def _place(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel())


def _logits(logits, what: str):
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a tensor, not %s" % type(logits).__name__)
    code = _code(logits.dtype, "logits")
    if logits.dim() != 2 or not 0 < logits.shape[1] <= MAX_EXPERTS:
        raise ValueError("%s takes logits [tokens, experts] of up to %d experts, not of shape %s" % (
            what, MAX_EXPERTS, list(logits.shape)))
    return code, _matrix(logits, "logits", logits.shape[0], logits.shape[1], logits.device, logits.dtype)


def _device(t, what: str):
    if not t.is_cuda:
        raise ValueError("%s needs device tensors" % what)
    return t.device


def _route(a, k, num_experts, device, ws, stream, how=("softmax", True, 1.0), given=None):
    tokens = a.tokens
    pairs = tokens * k
    caller = _caller(device, stream)
    with _on(device, stream):
        # one allocation for the four results
        room = torch.empty(3 * pairs + num_experts + 1, dtype=torch.int32, device=device)
        weights, experts, order, offsets = room.split_with_sizes((pairs, pairs, pairs, num_experts + 1))
        weights, experts = weights.view(torch.float32).view(tokens, k), experts.view(tokens, k)
        if given is not None:
            experts.copy_(given[0])
            weights.copy_(given[1])
        at, step = room.data_ptr(), 4 * pairs
        a.weights, a.experts, a.order, a.offsets = at, at + step, at + 2 * step, at + 3 * step
        a.num_experts, a.k = num_experts, k
        L, ref = _lib(), ctypes.byref(a)
        ws = _workspace(L.uzip_moe_route_workspace_size(ref), ws, device)
        st = L.uzip_moe_route(ref, *_place(ws), _stream_of(stream, device))
        if st != UZIP_OK:
            _check(st, "uzip_moe_route")
    _share(stream, caller, new=(experts, weights, order, offsets), given=(ws,))
    r = Routing.__new__(Routing)
    r.experts, r.weights, r.order, r.offsets = experts, weights, order, offsets
    r.scores, r.renormalize, r.scale = how
    r.tokens, r.k, r.num_experts, r.device = tokens, k, num_experts, device
    return r


def moe_route(logits, k: int, scores: str = "softmax", bias=None, renormalize: bool = True, scale: float = 1.0, ws=None,
              stream=None) -> Routing:
    """The k best experts of each token from logits [tokens, experts] (bf16 or
    fp32), best first, of equal ones the lowest, and their weights: scale times
    the softmax over all experts, or the sigmoid, of the logit; with
    renormalize over the sum of the chosen.  bias (fp32 [experts], sigmoid
    only) is added to the scores for the choice, not for the weights.  An
    expert whose logit is -inf is never chosen; where none is left the expert
    is -1 and the weight 0."""
    code, stride = _logits(logits, "moe_route")
    tokens, num = logits.shape
    if isinstance(k, bool) or not isinstance(k, int) or not 1 <= k <= min(num, MAX_CHOSEN):
        raise ValueError("k must be a whole number from 1 to %d, not %r" % (min(num, MAX_CHOSEN), k))
    if scores not in SCORES:
        raise ValueError("scores must be softmax or sigmoid, not %r" % (scores,))
    device = _device(logits, "moe_route")
    a = uzip_moe_route_args(logits.data_ptr(), stride, tokens, logits_dtype=code, scores=SCORES[scores],
                            renormalize=int(bool(renormalize)), scale=float(scale))
    if bias is not None:
        if scores != "sigmoid":
            raise ValueError("a bias goes with sigmoid scores")
        if not isinstance(bias, torch.Tensor) or bias.dtype is not torch.float32:
            raise TypeError("bias must be a float32 tensor")
        if bias.shape != (num,) or bias.device != device or not bias.is_contiguous():
            raise ValueError("bias must be %d contiguous values on %s" % (num, device))
        a.bias = bias.data_ptr()
    _no_history("moe_route", logits)
    return _route(a, k, num, device, ws, stream, (scores, bool(renormalize), float(scale)))


def moe_group(experts, weights, num_experts: int, ws=None, stream=None) -> Routing:
    """A Routing from experts (int32 [tokens, k]) and weights (fp32 [tokens,
    k]) that another router chose.  An expert outside [0, num_experts) becomes
    -1 with weight 0; so does one that a token names again, its weight added
    to the first."""
    if not isinstance(experts, torch.Tensor) or experts.dtype is not torch.int32:
        raise TypeError("experts must be an int32 tensor")
    if not isinstance(weights, torch.Tensor) or weights.dtype is not torch.float32:
        raise TypeError("weights must be a float32 tensor")
    if experts.dim() != 2 or not 1 <= experts.shape[1] <= MAX_CHOSEN or weights.shape != experts.shape:
        raise ValueError("experts and weights must both have shape [tokens, k], k from 1 to %d, not %s and %s" % (
            MAX_CHOSEN, list(experts.shape), list(weights.shape)))
    if isinstance(num_experts, bool) or not isinstance(num_experts, int) or not 1 <= num_experts <= MAX_EXPERTS:
        raise ValueError("num_experts must be a whole number from 1 to %d, not %r" % (MAX_EXPERTS, num_experts))
    if weights.device != experts.device:
        raise ValueError("weights is on %s, experts on %s" % (weights.device, experts.device))
    device = _device(experts, "moe_group")
    _no_history("moe_group", weights)
    a = uzip_moe_route_args(tokens=experts.shape[0], scale=1.0)
    return _route(a, experts.shape[1], num_experts, device, ws, stream, given=(experts, weights))


def _routing(r, what: str) -> Routing:
    if not isinstance(r, Routing):
        raise TypeError("%s takes a Routing (see moe_route), not %s" % (what, type(r).__name__))
    return r


def moe_route_backward(dweights, logits, routing: Routing, stream=None):
    """The gradient of moe_route's logits, in their type, from the weights'
    (fp32 [tokens, k]); the choice is held fixed.  A place without an expert
    has none."""
    r = _routing(routing, "moe_route_backward")
    code, stride = _logits(logits, "moe_route_backward")
    device = _device(logits, "moe_route_backward")
    if logits.shape != (r.tokens, r.num_experts) or r.device != device:
        raise ValueError("logits must have shape [%d, %d] on %s" % (r.tokens, r.num_experts, r.device))
    if not isinstance(dweights, torch.Tensor) or dweights.dtype is not torch.float32:
        raise TypeError("dweights must be a float32 tensor")
    if dweights.shape != (r.tokens, r.k) or dweights.device != device or not dweights.is_contiguous():
        raise ValueError("dweights must be contiguous of shape [%d, %d] on %s" % (r.tokens, r.k, device))
    caller = _caller(device, stream)
    with _on(device, stream):
        out = torch.empty(logits.shape, dtype=logits.dtype, device=device)
        a = uzip_moe_route_args(logits.data_ptr(), stride, r.tokens, None, r.experts.data_ptr(), dweights=dweights.data_ptr(),
                                dlogits=out.data_ptr(), dlogits_stride=r.num_experts, num_experts=r.num_experts, k=r.k,
                                logits_dtype=code, scores=SCORES[r.scores], renormalize=int(r.renormalize), scale=r.scale)
        st = _lib().uzip_moe_route_backward(ctypes.byref(a), _stream_of(stream, device))
        if st != UZIP_OK:
            _check(st, "uzip_moe_route_backward")
    _share(stream, caller, new=(out,))
    return out


def _bias(b, what: str, matrices: int, rows: int, device) -> int:
    if not isinstance(b, torch.Tensor):
        raise TypeError("%s must be a tensor, not %s" % (what, type(b).__name__))
    if b.shape != (matrices, rows) or b.device != device or not b.is_contiguous():
        raise ValueError("%s must be contiguous of shape [%d, %d] on %s" % (what, matrices, rows, device))
    return b.data_ptr()


def moe(x, routing: Routing, up: PackedWeight, down: PackedWeight, act: str = "swiglu", up_bias=None, down_bias=None,
        residual=None, out_dtype=None, out=None, ws=None, stream=None):
    """The expert layer: of each token of x [tokens, cols] (bf16) the sum over
    its experts e of weight times (D_e act(U_e x + up_bias_e) + down_bias_e),
    plus the residual.  up: packed stack [experts, rows, cols] of U, packed
    with gated=True for swiglu; down: packed stack of D, [experts, out_cols,
    rows], for swiglu [experts, out_cols, rows / 2].  The result is bf16, or
    out_dtype; residual has its shape and type; out may be the residual, and
    must not overlap x.  The biases have one type, bf16 or fp32.

    Up to 256 tokens (4,096 pairs, 16 an expert on average) take two kernels
    and keep the activations between the products to 2^-17 of themselves; more
    go through gathered rows and ``grouped_linear``, with activations in bf16
    (a result off by 0.0023 of the whole instead of 0.0017, its own rounding)."""
    r = _routing(routing, "moe")
    _weight(up, "moe", 3)
    _weight(down, "moe", 3)
    device = up.device
    act = _act(act, up)
    if down.gated:
        raise ValueError("down must not be gated")
    if down.device != device or r.device != device:
        raise ValueError("up is on %s, down on %s, the routing on %s" % (device, down.device, r.device))
    matrices, rows, cols = up.shape
    if down.shape[0] != matrices or down.shape[2] != (rows // 2 if up.gated else rows):
        raise ValueError("down must have shape [%d, out_cols, %d] to follow up, not %s" % (
            matrices, rows // 2 if up.gated else rows, list(down.shape)))
    tokens, width = _tokens(x, "x"), down.shape[1]
    if r.tokens != tokens or r.num_experts != matrices:
        raise ValueError("the routing is of %d tokens and %d experts, x has %d tokens and up %d experts" % (
            r.tokens, r.num_experts, tokens, matrices))
    a = uzip_moe_args()
    a.x_stride, a.x, a.tokens, a.k, a.act = _matrix(x, "x", tokens, cols, device), x.data_ptr(), tokens, r.k, act
    a.weights, a.order, a.offsets = r.weights.data_ptr(), r.order.data_ptr(), r.offsets.data_ptr()
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    a.y_dtype = _code(out_dtype, "out_dtype")
    if up_bias is not None:
        a.up_bias, a.bias_dtype = _bias(up_bias, "up_bias", matrices, rows, device), _code(up_bias.dtype, "up_bias")
    if down_bias is not None:
        a.down_bias, a.bias_dtype = _bias(down_bias, "down_bias", matrices, width, device), _code(down_bias.dtype, "down_bias")
        if up_bias is not None and up_bias.dtype is not down_bias.dtype:
            raise TypeError("up_bias is %s, down_bias %s: both must have one type" % (up_bias.dtype, down_bias.dtype))
    if residual is not None:
        a.residual_stride, a.residual = _matrix(residual, "residual", tokens, width, device, out_dtype), residual.data_ptr()
    if out is not None:
        a.y_stride = _matrix(out, "out", tokens, width, device, out_dtype)
        if _overlap(out, x):
            raise ValueError("out must not overlap x")
        if residual is not None and _overlap(out, residual) and (
                out.data_ptr() != residual.data_ptr() or a.y_stride != a.residual_stride):
            raise ValueError("out must be the residual itself or not overlap it")
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, r.weights, up_bias, down_bias, residual, out)):
        raise ValueError("moe records nothing for autograd, and an argument requires grad: call it under torch.no_grad(); for "
                         "training multiply by grouped_linear, which has its gradients, in a torch.autograd.Function")
    caller, given = _caller(device, stream), out
    with _on(device, stream):
        if out is None:
            out = torch.empty((tokens, width), dtype=out_dtype, device=device)
            a.y_stride = width
        if tokens:
            a.y = out.data_ptr()
            L, ref = _lib(), ctypes.byref(a)
            ws = _workspace(L.uzip_moe_workspace_size(up._ref, down._ref, ref), ws, device)
            st = L.uzip_moe(up._ref, down._ref, ref, *_place(ws), _stream_of(stream, device))
            if st != UZIP_OK:
                _check(st, "uzip_moe")
    _share(stream, caller, new=(out,) if given is None else (), given=(given, ws))
    return out
