"""Binding of the root-mean-square norm (include/tbe_norm.h): with the residual's
addition, in the rows' type or in 8 bits for a tbe_expert_product of all rows with one
expert, and its gradients.

As in the rest of the package the functions only check and marshal their
arguments; outputs that are not given are allocated on the stream the call runs on,
and results carry no autograd graph.
"""
from __future__ import annotations

import ctypes

import torch

from .experts import (_ROW_DT, _dense, _empty, _fp8_out, _lib, _matrix, _ok, _refuse_device,
                      _stream_of, _workspace)

__all__ = ["tbe_rms_norm", "tbe_rms_norm_fp8", "tbe_rms_norm_backward",
           "tbe_rms_norm_workspace_size", "TBE_MAX_NORM_WIDTH"]

TBE_MAX_NORM_WIDTH = 16384


def configure(lib):
    P, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                            ctypes.c_size_t)
    lib.tbe_rms_norm.argtypes = [P, P, P, i32, i32, i64, i64, i64, i64, f32, P, i64, P, i64, P]
    lib.tbe_rms_norm_fp8.argtypes = [P, P, P, i32, i32, i64, i64, i64, i64, f32, P, i64, P, i64,
                                     P, P]
    lib.tbe_rms_norm_workspace_size.argtypes = [i64, i64, ctypes.POINTER(sz)]
    lib.tbe_rms_norm_backward.argtypes = [P, P, P, P, i32, i32, i64, i64, i64, i64, i64, f32, P,
                                          i64, P, P, sz, P]
    for f in ("tbe_rms_norm", "tbe_rms_norm_fp8", "tbe_rms_norm_workspace_size",
              "tbe_rms_norm_backward"):
        getattr(lib, f).restype = ctypes.c_int


def _weight(weight, x, width, device):
    """Address and type of the weight."""
    if weight is None:
        return None, 0
    if weight.dtype not in (x.dtype, torch.float32):
        raise TypeError("weight must be of the rows' type or float32")
    if weight.dim() != 1 or weight.shape[0] != width or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous tensor of shape ({width},)")
    if weight.get_device() != device:
        _refuse_device(weight, "weight", device)
    return weight.data_ptr(), _ROW_DT[weight.dtype]


def _inputs(x, weight, residual, h, stream):
    device = x.get_device()
    xs = _matrix(x, "x", device, _ROW_DT)
    rows, width = x.shape
    w, wt = _weight(weight, x, width, device)
    rs = hs = width
    if residual is not None:
        rs = _matrix(residual, "residual", device, (x.dtype,), width, rows)
        if h is None:
            h = _empty(stream, (rows, width), x.dtype, x)
        else:
            hs = _matrix(h, "h", device, (x.dtype,), width, rows)
    elif h is not None:
        raise ValueError("h is the sum with a residual: it needs one")
    return device, xs, w, wt, rs, h, hs


def _at(t):
    return None if t is None else t.data_ptr()


def tbe_rms_norm(x, weight=None, residual=None, eps=1e-6, out=None, h=None, stream=None):
    """Rows x [rows, width] over their root mean square, times weight [width] (x's type or
    float32; None: ones).  With a residual the norm is of h = x + residual, rounded to
    their type, and (out, h) is returned; without one, out."""
    device, xs, w, wt, rs, h, hs = _inputs(x, weight, residual, h, stream)
    rows, width = x.shape
    os_ = width
    if out is None:
        out = _empty(stream, (rows, width), x.dtype, x)
    else:
        os_ = _matrix(out, "out", device, (x.dtype,), width, rows)
    _ok("tbe_rms_norm", _lib(device).tbe_rms_norm(
        x.data_ptr(), _at(residual), w, _ROW_DT[x.dtype], wt, rows, width, xs, rs, float(eps),
        _at(h), hs, out.data_ptr(), os_, _stream_of(stream, device)))
    return out if h is None else (out, h)


def tbe_rms_norm_fp8(x, weight=None, residual=None, eps=1e-6, out=None, scale=None, h=None,
                     stream=None):
    """tbe_rms_norm with the result quantised to e4m3, one fp32 scale for each 128 columns, as
    tbe_expert_product takes it of one expert for all rows: (q, scale), or (q, scale, h) with a
    residual.  Routed experts take their rows from tbe_rms_norm by tbe_expert_dispatch_fp8."""
    device, xs, w, wt, rs, h, hs = _inputs(x, weight, residual, h, stream)
    rows, width = x.shape
    out, qs, scale = _fp8_out(stream, device, x, rows, out, scale)
    _ok("tbe_rms_norm_fp8", _lib(device).tbe_rms_norm_fp8(
        x.data_ptr(), _at(residual), w, _ROW_DT[x.dtype], wt, rows, width, xs, rs, float(eps),
        _at(h), hs, out.data_ptr(), qs, scale.data_ptr(), _stream_of(stream, device)))
    return (out, scale) if h is None else (out, scale, h)


def tbe_rms_norm_workspace_size(rows, width):
    """Bytes of scratch tbe_rms_norm_backward needs for the weight's gradient."""
    import table_embedding_bag_gb300 as tbe
    n = ctypes.c_size_t(0)
    _ok("tbe_rms_norm_workspace_size", tbe._load().tbe_rms_norm_workspace_size(
        int(rows), int(width), ctypes.byref(n)))
    return n.value


def tbe_rms_norm_backward(grad_out, h, weight=None, grad_h=None, eps=1e-6, grad_x=None,
                          grad_weight=None, need_weight=True, ws=None, stream=None):
    """Gradients of tbe_rms_norm: (grad_x [rows, width], which is the gradient of x and
    of the residual alike, and grad_weight [width] fp32, or None unless need_weight).  h:
    the rows that were normalised (tbe_rms_norm's h, or x where it had no residual); grad_h:
    the gradient that arrives at h from behind, added to grad_x.  ws: uint8 scratch of
    tbe_rms_norm_workspace_size(rows, width) bytes, allocated when not given."""
    device = grad_out.get_device()
    gs = _matrix(grad_out, "grad_out", device, _ROW_DT)
    rows, width = grad_out.shape
    hs = _matrix(h, "h", device, (grad_out.dtype,), width, rows)
    w, wt = _weight(weight, grad_out, width, device)
    ghs = gxs = width
    if grad_h is not None:
        ghs = _matrix(grad_h, "grad_h", device, (grad_out.dtype,), width, rows)
    if grad_x is None:
        grad_x = _empty(stream, (rows, width), grad_out.dtype, grad_out)
    else:
        gxs = _matrix(grad_x, "grad_x", device, (grad_out.dtype,), width, rows)
    lib = _lib(device)
    if not need_weight:
        if grad_weight is not None:
            raise ValueError("grad_weight is given and not needed")
    else:
        if grad_weight is None:
            grad_weight = _empty(stream, (width,), torch.float32, grad_out)
        else:
            _dense(grad_weight, "grad_weight", device, torch.float32, (width,))
        ws = _workspace(lib, "tbe_rms_norm_workspace_size", (rows, width), ws, stream, grad_out)
    _ok("tbe_rms_norm_backward", lib.tbe_rms_norm_backward(
        grad_out.data_ptr(), h.data_ptr(), w, _at(grad_h), _ROW_DT[grad_out.dtype], wt, rows,
        width, gs, hs, ghs, float(eps), grad_x.data_ptr(), gxs, _at(grad_weight), _at(ws),
        0 if ws is None else ws.numel(), _stream_of(stream, device)))
    return grad_x, grad_weight
