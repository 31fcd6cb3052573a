"""A launch that the runtime refuses is reported by the call that asked for it, once, and
by none that follows.  The refusal is made on the host: a stream whose capture has become
invalid takes no launches."""
import contextlib
import ctypes

import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu

CAPTURE_THREAD_LOCAL, UNSUPPORTED, INVALIDATED = 1, 900, 901


@contextlib.contextmanager
def stream_that_takes_no_launches():
    cudart = ctypes.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cudart.cudaStreamCreateWithFlags(ctypes.byref(stream), 1) == 0
    try:
        assert cudart.cudaStreamBeginCapture(stream, CAPTURE_THREAD_LOCAL) == 0
        # waiting for a stream that is captured is refused, and ends the capture's validity
        assert cudart.cudaStreamSynchronize(stream) == UNSUPPORTED
        yield torch.cuda.ExternalStream(stream.value)
        assert cudart.cudaStreamEndCapture(stream, ctypes.byref(graph)) == INVALIDATED
    finally:
        cudart.cudaStreamDestroy(stream)
        cudart.cudaGetLastError()  # of the runtime that torch shares


def embed_gradient(n):
    grad, ids = torch.ones(n, 16, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda")
    out = torch.empty(5, 16, device="cuda")
    ws = torch.empty(max(tbe.tbe_embed_workspace_size(n, 5, 16), 1), dtype=torch.uint8,
                     device="cuda")
    return lambda stream: tbe.tbe_embed_backward(grad, ids, 5, out=out, ws=ws, stream=stream)


def sort(n):
    ids = torch.zeros(n, 1, dtype=torch.int32, device="cuda")
    out = tbe.tbe_expert_sort(ids, 4)
    return lambda stream: tbe.tbe_expert_sort(ids, 4, *out, stream=stream)


def product():
    a = torch.ones(128, 256, device="cuda")
    q, s = tbe.tbe_quantize_rows(a)
    w = tbe.tbe_quantize_weights(torch.ones(1, 128, 256, device="cuda"))
    out = tbe.tbe_expert_product(q, s, *w)
    return lambda stream: tbe.tbe_expert_product(q, s, *w, out=out, stream=stream)


def norm():
    x = torch.ones(8, 8192, device="cuda")
    y = torch.empty_like(x)
    return lambda stream: tbe.tbe_rms_norm(x, out=y, stream=stream)


@pytest.mark.parametrize("make", [
    lambda: embed_gradient(100), lambda: embed_gradient(2000), lambda: embed_gradient(200_000),
    lambda: sort(100), lambda: sort(200_000), product, norm])
def test_a_refused_launch_is_reported_once(make):
    call = make()
    table = torch.ones(4, 16, device="cuda")
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    with stream_that_takes_no_launches() as bad:
        with pytest.raises(tbe.TBEError) as e:
            call(bad)
        assert e.value.code == tbe.TBE_ECUDA
    assert torch.equal(tbe.tbe_embed(table, ids), torch.ones(3, 16, device="cuda"))
    call(torch.cuda.current_stream())
    torch.cuda.synchronize()
