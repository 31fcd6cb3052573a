"""Binding of the gradient-norm operators (include/tbe_grads.h)."""
from __future__ import annotations

import ctypes

import torch

from .experts import _ROW_DT, _On, _lib, _ok

__all__ = ["tbe_grad_norm", "tbe_grad_clip", "TBE_GRAD_WORKSPACE_BYTES"]

TBE_GRAD_WORKSPACE_BYTES = 16384


class tbe_grad_tensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def configure(lib):
    P, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    lib.tbe_grad_norm.argtypes = [P, i64, P, P, sz, P]
    lib.tbe_grad_clip.argtypes = [P, i64, ctypes.c_float, P, P, sz, P]
    lib.tbe_grad_norm.restype = lib.tbe_grad_clip.restype = ctypes.c_int


def _filled(t):
    """Whether the elements fill one block of memory, in any order of dimensions."""
    if t.is_contiguous():
        return True
    want = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size == 1:
            continue
        if stride != want:
            return False
        want *= size
    return True


def _table(grads, outs):
    rows = []
    for i, g in enumerate(grads):
        if g.dtype not in _ROW_DT:
            raise TypeError("gradients must be float16, bfloat16 or float32")
        if not g.is_cuda:
            raise ValueError("gradients must be CUDA tensors")
        if not _filled(g):
            raise ValueError("every gradient must fill one block of memory")
        at = g.data_ptr()
        to = at
        if outs is not None:
            o = outs[i]
            if o.dtype != g.dtype or o.shape != g.shape or not o.is_cuda:
                raise ValueError("out must hold a CUDA tensor of each gradient's type and shape")
            if o.stride() != g.stride() and not (o.is_contiguous() and g.is_contiguous()):
                raise ValueError("out must have each gradient's strides")
            to = o.data_ptr()
        rows.append((at, to, g.numel(), _ROW_DT[g.dtype], 0))
    return (tbe_grad_tensor * len(rows))(*rows)


def _scratch(on, grads, norm, ws):
    if norm is None:
        norm = on.empty((), torch.float32, grads[0])
    elif norm.dtype != torch.float32 or norm.numel() != 1 or not norm.is_cuda:
        raise ValueError("norm must be a float32 CUDA tensor with one entry")
    if ws is None:
        ws = on.empty(TBE_GRAD_WORKSPACE_BYTES, torch.uint8, grads[0])
    elif ws.dtype != torch.uint8 or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 CUDA tensor")
    return norm, ws


def tbe_grad_norm(grads, norm=None, ws=None, stream=None):
    """Global 2-norm of a sequence of gradients (float16, bfloat16 or float32,
    mixed as they come), as a float32 tensor with one entry.  ws: uint8
    scratch of TBE_GRAD_WORKSPACE_BYTES, allocated when not given."""
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    table = _table(grads, None)
    on = _On(stream)
    norm, ws = _scratch(on, grads, norm, ws)
    _ok("tbe_grad_norm", _lib().tbe_grad_norm(
        table, len(grads), norm.data_ptr(), ws.data_ptr(), ws.numel(), on.ptr))
    return norm


def tbe_grad_clip(grads, max_norm, out=None, norm=None, ws=None, stream=None):
    """Multiplies every gradient by min(1, max_norm / (norm + 1e-6)), in place or
    into the tensors of `out`, and returns the norm before clipping."""
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError("out must hold one tensor for each gradient")
    table = _table(grads, out)
    on = _On(stream)
    norm, ws = _scratch(on, grads, norm, ws)
    _ok("tbe_grad_clip", _lib().tbe_grad_clip(
        table, len(grads), float(max_norm), norm.data_ptr(), ws.data_ptr(), ws.numel(), on.ptr))
    return norm
