"""Binding of the expert-layer operators (include/tbe_experts.h): sort, dispatch
and combine with their gradients, 8-bit quantising, and the experts' products.

As in the rest of the package the functions only check and marshal their
arguments.  A call runs on the device of its tensors, which must all be on one,
whichever device is current.  Outputs that are not given are allocated on the
stream the call runs on.  A matrix may have any row stride; its columns must be
contiguous.  An output must not share memory with an input (no call works in
place).  Autograd is not involved: results require no gradient, and the
gradients are calls of their own.
"""
from __future__ import annotations

import ctypes

import torch

__all__ = [
    "tbe_expert_sort", "tbe_expert_dispatch", "tbe_expert_dispatch_fp8", "tbe_expert_combine",
    "tbe_expert_combine_backward", "tbe_expert_dispatch_backward", "tbe_quantize_rows",
    "tbe_quantize_weights", "tbe_expert_product", "TBE_MAX_EXPERTS", "TBE_SCALE_BLOCK",
]

TBE_MAX_EXPERTS = 1024
TBE_SCALE_BLOCK = 128
_ROW_DT = {torch.float16: 1, torch.bfloat16: 4, torch.float32: 5}
_ID_DT = {torch.int32: 2, torch.int64: 3}


def configure(lib):
    P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.tbe_expert_sort.argtypes = [P, i32, i64, i32, i32, P, P, P, P]
    lib.tbe_expert_dispatch.argtypes = [P, i32, i64, i32, i64, i64, P, i32, P, P, i64, P]
    lib.tbe_expert_dispatch_fp8.argtypes = [P, i32, i64, i32, i64, i64, P, i32, P, P, i64, P, P]
    lib.tbe_expert_combine.argtypes = [P, i32, i64, i32, i64, i64, P, P, P, i64, P]
    lib.tbe_expert_combine_backward.argtypes = [P, P, i32, i64, i32, i64, i64, i64, P, i32, P, P,
                                                P, i64, P, P]
    lib.tbe_quantize_weights.argtypes = [P, i32, i64, i64, i64, P, P, P]
    lib.tbe_expert_product.argtypes = [P, i64, P, P, P, P, i64, i64, i64, i32, P, i32, i64, P, P]
    for f in ("sort", "dispatch", "dispatch_fp8", "combine", "combine_backward", "product"):
        getattr(lib, f"tbe_expert_{f}").restype = ctypes.c_int
    lib.tbe_quantize_weights.restype = ctypes.c_int


_lib_ = None


_current_device = torch._C._cuda_getDevice
_on_device = torch.cuda.device


def _lib(device):
    """The library, whose calls launch on the current device, for a call on `device`."""
    global _lib_
    if _lib_ is None:
        import table_embedding_bag_gb300 as tbe
        _lib_ = tbe._load()
    return _lib_ if device == _current_device() else _OnDevice(_lib_, device)


class _OnDevice:
    """The library with `device` made current during each call."""

    def __init__(self, lib, device):
        self.lib, self.device = lib, device

    def __getattr__(self, name):
        def call(*args):
            with _on_device(self.device):
                return getattr(self.lib, name)(*args)
        return call


def _ok(call, code):
    if code:
        import table_embedding_bag_gb300 as tbe
        raise tbe.TBEError(call, code)


# The calls below take microseconds on the GPU, so their checks are written to
# take few on the host: no torch.cuda.current_stream() object (2.8 us), no check
# of what was just allocated.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream_of(stream, device):
    """The cudaStream_t a call on `device` runs on."""
    if stream is None:
        return _raw_stream(device)
    if stream.device_index != device:
        raise ValueError("the stream must be one of the tensors' device")
    return stream.cuda_stream


def _empty(stream, shape, dtype, like):
    """An output that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _refuse_device(t, name, device):
    if device < 0 or t.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} must be on the device of the other tensors")


def _matrix(t, name, device, dtypes, cols=None, rows=None):
    """A 2-d tensor on `device` with contiguous columns; returns its row stride."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(str(d) for d in dtypes)}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    if t.get_device() != device or device < 0:
        _refuse_device(t, name, device)
    r, c = t.shape
    if (cols is not None and c != cols) or (rows is not None and r != rows):
        raise ValueError(f"{name} must have the shape [{rows if rows is not None else '*'}, "
                         f"{cols if cols is not None else '*'}]")
    if t.is_contiguous():
        return c
    s0, s1 = t.stride()
    if c > 1 and s1 != 1:
        raise ValueError(f"{name} must have contiguous columns")
    if r <= 1:
        return c
    if s0 < c:
        raise ValueError(f"{name} must not have overlapping rows")
    return s0


def _dense(t, name, device, dtype, shape):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}")
    if t.get_device() != device or device < 0:
        _refuse_device(t, name, device)


def _positions(position, device):
    if position.dtype != torch.int32:
        raise TypeError("position must be torch.int32")
    shape = position.shape
    if len(shape) != 2 or shape[1] < 1 or not position.is_contiguous():
        raise ValueError("position must be a contiguous tensor [tokens, k], k >= 1")
    if position.get_device() != device or device < 0:
        _refuse_device(position, "position", device)
    return shape


def _experts(offsets, device):
    if offsets.dtype != torch.int32:
        raise TypeError("offsets must be torch.int32")
    n = offsets.numel() - 1
    if n < 1 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous tensor [num_experts + 1]")
    if offsets.get_device() != device or device < 0:
        _refuse_device(offsets, "offsets", device)
    return n


def tbe_expert_sort(ids, num_experts, offsets=None, source=None, position=None, stream=None):
    """Sorts the assignments ids [tokens, k] (int32 or int64; an id outside
    [0, num_experts) drops its assignment) by expert.  Returns (offsets
    [num_experts + 1], source [tokens * k], position [tokens, k]), all int32;
    see tbe_expert_sort in include/tbe_experts.h."""
    if ids.dtype not in _ID_DT:
        raise TypeError("ids must be int32 or int64")
    if ids.dim() != 2 or ids.shape[1] < 1:
        raise ValueError("ids must have the shape [tokens, k], k >= 1")
    device = ids.get_device()
    _dense(ids, "ids", device, ids.dtype, ids.shape)
    if not 1 <= num_experts <= TBE_MAX_EXPERTS:
        raise ValueError(f"num_experts must lie in [1, {TBE_MAX_EXPERTS}]")
    tokens, k = ids.shape
    if offsets is None:
        offsets = _empty(stream, num_experts + 1, torch.int32, ids)
    else:
        _dense(offsets, "offsets", device, torch.int32, (num_experts + 1,))
    if source is None:
        source = _empty(stream, tokens * k, torch.int32, ids)
    else:
        _dense(source, "source", device, torch.int32, (tokens * k,))
    if position is None:
        position = _empty(stream, (tokens, k), torch.int32, ids)
    else:
        _dense(position, "position", device, torch.int32, (tokens, k))
    _ok("tbe_expert_sort", _lib(device).tbe_expert_sort(
        ids.data_ptr(), _ID_DT[ids.dtype], tokens, k, num_experts, offsets.data_ptr(),
        source.data_ptr(), position.data_ptr(), _stream_of(stream, device)))
    return offsets, source, position


def tbe_expert_dispatch(x, offsets, position, out=None, stream=None):
    """rows [tokens * k, width]: x's rows at their sorted places, zeros after the
    last kept one."""
    device = x.get_device()
    experts = _experts(offsets, device)
    tokens, k = _positions(position, device)
    xs = _matrix(x, "x", device, _ROW_DT, rows=tokens)
    width = os_ = x.shape[1]
    if out is None:
        out = _empty(stream, (tokens * k, width), x.dtype, x)
    else:
        os_ = _matrix(out, "out", device, (x.dtype,), width, tokens * k)
    _ok("tbe_expert_dispatch", _lib(device).tbe_expert_dispatch(
        x.data_ptr(), _ROW_DT[x.dtype], tokens, k, width, xs, offsets.data_ptr(), experts,
        position.data_ptr(), out.data_ptr(), os_, _stream_of(stream, device)))
    return out


def _fp8_out(stream, device, x, rows, out, scale):
    width = qs = x.shape[1]
    blocks = -(-width // TBE_SCALE_BLOCK)
    if out is None:
        out = _empty(stream, (rows, width), torch.float8_e4m3fn, x)
    else:
        qs = _matrix(out, "out", device, (torch.float8_e4m3fn,), width, rows)
    if scale is None:
        scale = _empty(stream, (rows, blocks), torch.float32, x)
    else:
        _dense(scale, "scale", device, torch.float32, (rows, blocks))
    return out, qs, scale


def tbe_expert_dispatch_fp8(x, offsets, position, out=None, scale=None, stream=None):
    """The dispatch with the rows quantised to e4m3 on the way: (q [tokens * k,
    width], scale [tokens * k, ceil(width / 128)])."""
    device = x.get_device()
    experts = _experts(offsets, device)
    tokens, k = _positions(position, device)
    xs = _matrix(x, "x", device, _ROW_DT, rows=tokens)
    out, qs, scale = _fp8_out(stream, device, x, tokens * k, out, scale)
    _ok("tbe_expert_dispatch_fp8", _lib(device).tbe_expert_dispatch_fp8(
        x.data_ptr(), _ROW_DT[x.dtype], tokens, k, x.shape[1], xs, offsets.data_ptr(), experts,
        position.data_ptr(), out.data_ptr(), qs, scale.data_ptr(), _stream_of(stream, device)))
    return out, scale


def tbe_quantize_rows(x, out=None, scale=None, stream=None):
    """Rows to e4m3 with an fp32 scale for each 128 columns: (q, scale)."""
    device = x.get_device()
    xs = _matrix(x, "x", device, _ROW_DT)
    out, qs, scale = _fp8_out(stream, device, x, x.shape[0], out, scale)
    _ok("tbe_quantize_rows", _lib(device).tbe_expert_dispatch_fp8(
        x.data_ptr(), _ROW_DT[x.dtype], x.shape[0], 1, x.shape[1], xs, None, 0, None,
        out.data_ptr(), qs, scale.data_ptr(), _stream_of(stream, device)))
    return out, scale


def tbe_quantize_weights(w, out=None, scale=None, stream=None):
    """Weights [experts, n, k] to e4m3 with an fp32 scale for each 128 x 128
    block: (q, scale [experts, ceil(n / 128), ceil(k / 128)])."""
    if w.dtype not in _ROW_DT:
        raise TypeError("w must be float16, bfloat16 or float32")
    if w.dim() != 3:
        raise ValueError("w must have the shape [experts, n, k]")
    device = w.get_device()
    _dense(w, "w", device, w.dtype, w.shape)
    e, n, k = w.shape
    grid = (e, -(-n // TBE_SCALE_BLOCK), -(-k // TBE_SCALE_BLOCK))
    if out is None:
        out = _empty(stream, (e, n, k), torch.float8_e4m3fn, w)
    else:
        _dense(out, "out", device, torch.float8_e4m3fn, (e, n, k))
    if scale is None:
        scale = _empty(stream, grid, torch.float32, w)
    else:
        _dense(scale, "scale", device, torch.float32, grid)
    _ok("tbe_quantize_weights", _lib(device).tbe_quantize_weights(
        w.data_ptr(), _ROW_DT[w.dtype], e, n, k, out.data_ptr(), scale.data_ptr(),
        _stream_of(stream, device)))
    return out, scale


def tbe_expert_combine(y, position, weights=None, out=None, stream=None):
    """out [tokens, width]: the experts' rows y [tokens * k, width] weighted (fp32
    weights [tokens, k], or None for ones) and summed per token."""
    device = y.get_device()
    tokens, k = _positions(position, device)
    ys = _matrix(y, "y", device, _ROW_DT, rows=tokens * k)
    width = os_ = y.shape[1]
    if weights is not None:
        _dense(weights, "weights", device, torch.float32, (tokens, k))
    if out is None:
        out = _empty(stream, (tokens, width), y.dtype, y)
    else:
        os_ = _matrix(out, "out", device, (y.dtype,), width, tokens)
    _ok("tbe_expert_combine", _lib(device).tbe_expert_combine(
        y.data_ptr(), _ROW_DT[y.dtype], tokens, k, width, ys, position.data_ptr(),
        None if weights is None else weights.data_ptr(), out.data_ptr(), os_,
        _stream_of(stream, device)))
    return out


def tbe_expert_dispatch_backward(grad_rows, position, out=None, stream=None):
    """Gradient of tbe_expert_dispatch's x: each token's rows of grad_rows summed."""
    return tbe_expert_combine(grad_rows, position, None, out, stream)


def tbe_expert_combine_backward(grad_out, y, offsets, position, weights=None, grad_y=None,
                                grad_weights=None, stream=None):
    """Gradients of tbe_expert_combine: (grad_y [tokens * k, width], grad_weights
    [tokens, k] fp32)."""
    device = grad_out.get_device()
    experts = _experts(offsets, device)
    tokens, k = _positions(position, device)
    gs = _matrix(grad_out, "grad_out", device, _ROW_DT, rows=tokens)
    width = gys = grad_out.shape[1]
    ys = _matrix(y, "y", device, (grad_out.dtype,), width, tokens * k)
    if weights is not None:
        _dense(weights, "weights", device, torch.float32, (tokens, k))
    if grad_y is None:
        grad_y = _empty(stream, (tokens * k, width), grad_out.dtype, grad_out)
    else:
        gys = _matrix(grad_y, "grad_y", device, (grad_out.dtype,), width, tokens * k)
    if grad_weights is None:
        grad_weights = _empty(stream, (tokens, k), torch.float32, grad_out)
    else:
        _dense(grad_weights, "grad_weights", device, torch.float32, (tokens, k))
    _ok("tbe_expert_combine_backward", _lib(device).tbe_expert_combine_backward(
        grad_out.data_ptr(), y.data_ptr(), _ROW_DT[grad_out.dtype], tokens, k, width, gs, ys,
        offsets.data_ptr(), experts, position.data_ptr(),
        None if weights is None else weights.data_ptr(), grad_y.data_ptr(), gys,
        grad_weights.data_ptr(), _stream_of(stream, device)))
    return grad_y, grad_weights


def tbe_expert_product(a, a_scale, w, w_scale, offsets=None, out=None, out_dtype=torch.bfloat16,
                       status=None, stream=None):
    """out [rows, n]: rows a [rows, k] (e4m3, scales a_scale from
    tbe_quantize_rows or tbe_expert_dispatch_fp8) of expert e, offsets[e] <= row
    < offsets[e + 1], times the transpose of w[e] (w [experts, n, k] e4m3 with
    w_scale from tbe_quantize_weights).  offsets None: one expert takes all
    rows.  Rows before offsets[0] and from offsets[-1] on are zeros, so w, w_scale
    and offsets may be those of a run of the experts.  status: an int32 CUDA tensor that
    receives TBE_ERR_* bits, or None; what a device wait that gave up may have
    lost is NaN either way."""
    fp8, device = torch.float8_e4m3fn, a.get_device()
    as_ = _matrix(a, "a", device, (fp8,))
    rows, k = a.shape
    if w.dim() != 3 or w.shape[2] != k:
        raise ValueError(f"w must have the shape [experts, n, {k}]")
    e, n, _ = shape = w.shape
    _dense(w, "w", device, fp8, shape)
    kb = -(-k // TBE_SCALE_BLOCK)
    _dense(a_scale, "a_scale", device, torch.float32, (rows, kb))
    _dense(w_scale, "w_scale", device, torch.float32, (e, -(-n // TBE_SCALE_BLOCK), kb))
    if offsets is not None:
        _dense(offsets, "offsets", device, torch.int32, (e + 1,))
    elif e != 1:
        raise ValueError("offsets may be None with one expert only")
    if status is not None:
        if status.dtype != torch.int32 or status.numel() < 1:
            raise ValueError("status must be an int32 tensor with an entry")
        if status.get_device() != device:
            _refuse_device(status, "status", device)
    os_ = n
    if out is None:
        if out_dtype not in _ROW_DT:
            raise TypeError("out_dtype must be float16, bfloat16 or float32")
        out = _empty(stream, (rows, n), out_dtype, a)
    else:
        os_ = _matrix(out, "out", device, _ROW_DT, n, rows)
    _ok("tbe_expert_product", _lib(device).tbe_expert_product(
        a.data_ptr(), as_, a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
        None if offsets is None else offsets.data_ptr(), rows, n, k, e, out.data_ptr(),
        _ROW_DT[out.dtype], os_, None if status is None else status.data_ptr(),
        _stream_of(stream, device)))
    return out
