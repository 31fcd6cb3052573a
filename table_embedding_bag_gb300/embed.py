"""Binding of the token embedding (include/tbe_embed.h): rows of a table by token,
and the table's gradient by sorted tokens.

As in the rest of the package the functions only check and marshal their
arguments; outputs that are not given are allocated on the stream the call runs on,
and results carry no autograd graph.
"""
from __future__ import annotations

import ctypes

import torch

from .experts import (_ID_DT, _ROW_DT, _empty, _lib, _matrix, _ok, _refuse_device, _stream_of,
                      _workspace)

__all__ = ["tbe_embed", "tbe_embed_backward", "tbe_embed_workspace_size"]


def configure(lib):
    P, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float,
                            ctypes.c_size_t)
    lib.tbe_embed.argtypes = [P, i32, i64, i64, i64, P, i32, i64, f32, P, i64, P]
    lib.tbe_embed_workspace_size.argtypes = [i64, i64, i64, ctypes.POINTER(sz)]
    lib.tbe_embed_backward.argtypes = [P, i32, i64, i64, i64, P, i32, i64, f32, i32, P, i32, i64,
                                       P, sz, P]
    for f in ("tbe_embed", "tbe_embed_workspace_size", "tbe_embed_backward"):
        getattr(lib, f).restype = ctypes.c_int


def _token_ids(ids, device):
    if ids.dtype not in _ID_DT:
        raise TypeError("ids must be int32 or int64")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    if ids.get_device() != device or device < 0:
        _refuse_device(ids, "ids", device)
    return ids.numel()


def tbe_embed(table, ids, scale=1.0, out=None, stream=None):
    """scale * table[ids]: rows of table [rows, width] by ids (int32 or int64, any
    shape), rounded once; zeros where an id is no row.  Returns [*ids.shape, width], or
    out [ids.numel(), width] if that is given."""
    device = table.get_device()
    ts = _matrix(table, "table", device, _ROW_DT)
    rows, width = table.shape
    n = _token_ids(ids, device)
    os_ = width
    if out is None:
        out = _empty(stream, (*ids.shape, width), table.dtype, table)
    else:
        os_ = _matrix(out, "out", device, (table.dtype,), width, n)
    _ok("tbe_embed", _lib(device).tbe_embed(
        table.data_ptr(), _ROW_DT[table.dtype], rows, width, ts, ids.data_ptr(),
        _ID_DT[ids.dtype], n, float(scale), out.data_ptr(), os_, _stream_of(stream, device)))
    return out


def tbe_embed_workspace_size(tokens, rows, width):
    """Bytes of scratch tbe_embed_backward needs."""
    import table_embedding_bag_gb300 as tbe
    n = ctypes.c_size_t(0)
    _ok("tbe_embed_workspace_size", tbe._load().tbe_embed_workspace_size(
        int(tokens), int(rows), int(width), ctypes.byref(n)))
    return n.value


def tbe_embed_backward(grad_out, ids, rows, scale=1.0, out=None, out_dtype=None, accumulate=False,
                       ws=None, stream=None):
    """Gradient of tbe_embed's table: [rows, width] of out_dtype (grad_out's type, or
    float32), each row scale times the sum of its tokens' rows of grad_out.  grad_out is
    [ids.numel(), width], or [*ids.shape, width] if contiguous.  accumulate: adds to
    out, leaving rows without tokens as they are.  ws: uint8 scratch of
    tbe_embed_workspace_size(tokens, rows, width) bytes, allocated when not given."""
    device = grad_out.get_device()
    if grad_out.dim() != 2 and grad_out.dim() >= 1 and grad_out.is_contiguous() and \
            grad_out.shape[:-1] == ids.shape:
        grad_out = grad_out.view(ids.numel(), grad_out.shape[-1])
    n = _token_ids(ids, device)
    gs = _matrix(grad_out, "grad_out", device, _ROW_DT, rows=n)
    width = os_ = grad_out.shape[1]
    rows = int(rows)
    if rows < 0:
        raise ValueError("rows must not be negative")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an out to add to")
        out_dtype = grad_out.dtype if out_dtype is None else out_dtype
        if out_dtype not in (grad_out.dtype, torch.float32):
            raise TypeError("out_dtype must be grad_out's type or float32")
        out = _empty(stream, (rows, width), out_dtype, grad_out)
    else:
        if out_dtype is not None and out_dtype != out.dtype:
            raise TypeError("out must be of out_dtype")
        os_ = _matrix(out, "out", device, (grad_out.dtype, torch.float32), width, rows)
    lib = _lib(device)
    ws = _workspace(lib, "tbe_embed_workspace_size", (n, rows, width), ws, stream, grad_out)
    _ok("tbe_embed_backward", lib.tbe_embed_backward(
        grad_out.data_ptr(), _ROW_DT[grad_out.dtype], n, width, gs, ids.data_ptr(),
        _ID_DT[ids.dtype], rows, float(scale), bool(accumulate), out.data_ptr(),
        _ROW_DT[out.dtype], os_, None if ws is None else ws.data_ptr(),
        0 if ws is None else ws.numel(), _stream_of(stream, device)))
    return out
