"""Sampling of tokens from logits: the tensor form of uzip_sample
(include/uzip.h), for the logits that ``linear`` makes of a packed output
head.  Streams, workspaces and errors are as for the products with packed
weights; a sampled token has no gradient (that of its log-probability is
``linear_cross_entropy_backward``'s).
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import UZIP_OK, _check, lib, workspace
from .weights import _caller, _code, _matrix, _on, _ref, _share, _stream_of

_vp, _sz, _u32, _f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_float


class uzip_sample_args(ctypes.Structure):
    _fields_ = [("logits", _vp), ("logits_stride", _sz), ("rows", _sz), ("vocab", _sz), ("u", _vp), ("temperature", _vp),
                ("top_k", _vp), ("top_p", _vp), ("min_p", _vp), ("token", _vp), ("logprob", _vp), ("temperature_all", _f32),
                ("top_k_all", ctypes.c_int32), ("top_p_all", _f32), ("min_p_all", _f32), ("logits_dtype", _u32),
                ("u_double", _u32)]


def _lib():
    L = lib()
    if not getattr(L, "_sample_declared", False):
        S = ctypes.POINTER(uzip_sample_args)
        L.uzip_sample_workspace_size.restype = _sz
        L.uzip_sample_workspace_size.argtypes = [S]
        L.uzip_sample.restype = ctypes.c_int
        L.uzip_sample.argtypes = [S, _vp, _sz, _vp]
        L._sample_declared = True
    return L


# ---- the C entry points, same names and arguments ----------------------------
def uzip_sample_workspace_size(args) -> int:
    return _lib().uzip_sample_workspace_size(_ref(args))


def uzip_sample(args, d_workspace, workspace_bytes, stream) -> int:
    return _lib().uzip_sample(_ref(args), d_workspace, workspace_bytes, stream)


# ---- tensors --------------------------------------------------------------------
def _row(v, what: str, rows: int, device, dtype) -> int:
    if v.dtype is not dtype:
        raise TypeError("%s must be a number or a %s tensor, not %s" % (what, dtype, v.dtype))
    if v.shape != (rows,) or v.device != device or not v.is_contiguous():
        raise ValueError("%s must be a number or %d contiguous values on %s" % (what, rows, device))
    return v.data_ptr()


def _device(t):
    if not t.is_cuda:
        raise ValueError("sample needs device tensors")
    return t.device


def _number(v, what: str) -> float:
    if isinstance(v, bool) or not isinstance(v, (int, float)) or v != v:
        raise TypeError("%s must be a number or a tensor, not %r" % (what, v))
    return float(v)


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, ws=None, stream=None):
    """(token int64 [rows], logprob fp32 [rows]) drawn from logits [rows,
    vocab], bf16 or fp32, with the random numbers u [rows] in [0, 1), fp32 or
    fp64.

    With e = exp((z - max) / temperature) and the tokens ordered by (z
    descending, index ascending): of the first top_k (0: all) those are kept
    before which less than top_p of their sum has passed, and of these the ones
    with e >= min_p; the first is always kept.  The token is the first kept
    one, by index, at which the running sum of e exceeds u times the sum of the
    kept.  temperature 0 takes the largest logit, of equal ones the first.
    logprob is the token's log-softmax over all logits / temperature (by 1
    where it is 0), whatever the filters.  Each parameter is a number (taken as
    fp32) or a tensor with one value a row: fp32, top_k int32.

    -inf is never drawn; a row with a NaN or with nothing above -inf, or with a
    negative or infinite temperature or a NaN among its parameters, gives token
    -1 and logprob NaN."""
    if not isinstance(logits, torch.Tensor) or not isinstance(u, torch.Tensor):
        raise TypeError("logits and u must be tensors")
    code = _code(logits.dtype, "logits")
    if logits.dim() != 2 or logits.shape[1] == 0:
        raise ValueError("logits must have shape [rows, vocab], not %s" % list(logits.shape))
    device, (rows, vocab) = _device(logits), logits.shape
    if u.dtype not in (torch.float32, torch.float64):
        raise TypeError("u must be float32 or float64, not %s" % u.dtype)
    if u.shape != (rows,) or u.device != device or not u.is_contiguous():
        raise ValueError("u must be %d contiguous values on %s" % (rows, device))
    a = uzip_sample_args(logits.data_ptr(), _matrix(logits, "logits", rows, vocab, device, logits.dtype), rows, vocab,
                         u.data_ptr(), logits_dtype=code, u_double=int(u.dtype is torch.float64))
    if isinstance(temperature, torch.Tensor):
        a.temperature = _row(temperature, "temperature", rows, device, torch.float32)
    else:
        a.temperature_all = _number(temperature, "temperature")
        if a.temperature_all < 0 or math.isinf(a.temperature_all):
            raise ValueError("temperature must be at least 0 and finite, not %r" % temperature)
    if isinstance(top_k, torch.Tensor):
        a.top_k = _row(top_k, "top_k", rows, device, torch.int32)
    elif isinstance(top_k, bool) or not isinstance(top_k, int) or top_k < 0:
        raise ValueError("top_k must be a whole number of at least 0 or a tensor, not %r" % (top_k,))
    else:
        a.top_k_all = min(top_k, vocab)
    for name, v in (("top_p", top_p), ("min_p", min_p)):
        if isinstance(v, torch.Tensor):
            setattr(a, name, _row(v, name, rows, device, torch.float32))
        else:
            v = _number(v, name)
            if not 0 <= v <= 1:
                raise ValueError("%s must be from 0 to 1, not %r" % (name, v))
            setattr(a, name + "_all", v)
    if logits.requires_grad and torch.is_grad_enabled():
        raise ValueError("sample records nothing for autograd, and logits requires grad: call it under torch.no_grad()")
    caller = _caller(device, stream)
    with _on(device, stream):
        token = torch.empty(rows, dtype=torch.int64, device=device)
        logprob = torch.empty(rows, dtype=torch.float32, device=device)
        if rows:
            a.token, a.logprob = token.data_ptr(), logprob.data_ptr()
            L, ref = _lib(), ctypes.byref(a)
            need = L.uzip_sample_workspace_size(ref)
            if ws is None:
                ws = workspace(need, device) if need else None
            elif not isinstance(ws, torch.Tensor) or ws.dtype is not torch.uint8 or ws.device != device or not ws.is_contiguous():
                raise ValueError("ws must be a contiguous uint8 tensor on %s" % device)
            st = L.uzip_sample(ref, ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
                               _stream_of(stream, device))
            if st != UZIP_OK:
                _check(st, "uzip_sample")
    _share(stream, caller, new=(token, logprob), given=(ws,))
    return token, logprob
