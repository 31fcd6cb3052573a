"""Binding of the gradient-norm operators (include/tbe_grads.h).

Autograd is not involved: the norm requires no gradient, and clipping in place
moves no version counter.
"""
from __future__ import annotations

import ctypes
import operator

import numpy as np
import torch

from .experts import _ROW_DT, _empty, _lib, _ok, _refuse_device, _stream_of

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


_ROW = np.dtype([("grad", np.uint64), ("out", np.uint64), ("numel", np.int64),
                 ("dtype", np.int32), ("reserved", np.int32)])
assert _ROW.itemsize == ctypes.sizeof(tbe_grad_tensor)


def _filled(t):
    """Whether the elements fill one block of memory, in any order of dimensions."""
    want = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size == 1:
            continue
        if stride != want:
            return False
        want *= size
    return True


_dtype_of = operator.attrgetter("dtype")
_Tensor = torch.Tensor


def _table(grads, outs):
    """The tensors' table for the C call.  Attributes are read a list at a time
    (40 ns a tensor each): hundreds of gradients are an ordinary step, and
    their checks must not take longer than their clipping."""
    dtypes = list(map(_dtype_of, grads))
    if not all(d in _ROW_DT for d in set(dtypes)):
        raise TypeError("gradients must be float16, bfloat16 or float32")
    devices = set(map(_Tensor.get_device, grads))
    if -1 in devices:
        raise ValueError("gradients must be CUDA tensors")
    if len(devices) > 1:
        raise ValueError("the gradients must be on one device")
    dense = all(map(_Tensor.is_contiguous, grads))
    if not dense and not all(g.is_contiguous() or _filled(g) for g in grads):
        raise ValueError("every gradient must fill one block of memory")
    numel = list(map(_Tensor.numel, grads))
    at = to = list(map(_Tensor.data_ptr, grads))
    if outs is not None:
        if list(map(_dtype_of, outs)) != dtypes or list(map(_Tensor.numel, outs)) != numel or \
                set(map(_Tensor.get_device, outs)) != devices:
            raise ValueError("out must hold a tensor of each gradient's type, size and device")
        if not (dense and all(map(_Tensor.is_contiguous, outs))) and \
                not all(o.shape == g.shape and o.stride() == g.stride() or
                        o.is_contiguous() and g.is_contiguous() for o, g in zip(outs, grads)):
            raise ValueError("out must have each gradient's strides")
        to = list(map(_Tensor.data_ptr, outs))
    table = np.empty(len(grads), _ROW)
    table["grad"], table["out"], table["numel"] = at, to, numel
    table["dtype"] = list(map(_ROW_DT.__getitem__, dtypes))
    return table


def _scratch(stream, grads, norm, ws):
    device = grads[0].get_device()
    if norm is None:
        norm = _empty(stream, (), torch.float32, grads[0])
    else:
        if norm.dtype != torch.float32 or norm.numel() != 1:
            raise ValueError("norm must be a float32 tensor with one entry")
        if norm.get_device() != device:
            _refuse_device(norm, "norm", device)
    if ws is None:
        ws = _empty(stream, TBE_GRAD_WORKSPACE_BYTES, torch.uint8, grads[0])
    else:
        if ws.dtype != torch.uint8 or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous uint8 tensor")
        if ws.get_device() != device:
            _refuse_device(ws, "ws", device)
    return device, norm, ws


def tbe_grad_norm(grads, norm=None, ws=None, stream=None):
    """Global 2-norm of a sequence of gradients (float16, bfloat16 or float32,
    mixed as they come, on one device), as a float32 tensor with one entry.  ws: uint8
    scratch of TBE_GRAD_WORKSPACE_BYTES, allocated when not given."""
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    table = _table(grads, None)
    device, norm, ws = _scratch(stream, grads, norm, ws)
    _ok("tbe_grad_norm", _lib(device).tbe_grad_norm(
        table.ctypes.data, len(grads), norm.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream_of(stream, device)))
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
    device, norm, ws = _scratch(stream, grads, norm, ws)
    _ok("tbe_grad_clip", _lib(device).tbe_grad_clip(
        table.ctypes.data, len(grads), float(max_norm), norm.data_ptr(), ws.data_ptr(),
        ws.numel(), _stream_of(stream, device)))
    return norm
