"""The same kernel launched with different amounts of shared memory by several host threads
at once, and between the capture of a graph and its replay."""
import ctypes
import threading

import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu


BF16, I64 = 4, 3


def at_once(calls, rounds=12000):
    """Runs each of the calls in a thread of its own, on a stream of its own, and returns the
    statuses they gave."""
    seen, start = [], threading.Barrier(len(calls))

    def run(call):
        stream = torch.cuda.Stream()
        to = ctypes.c_void_p(stream.cuda_stream)
        start.wait()
        seen.append({call(to) for _ in range(rounds)})
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return set().union(*seen)


def randn(*shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(shape))
    return torch.randn(*shape, generator=g, device="cuda")


def bound(name, *args):
    """The C call with its arguments converted once, so that threads meet in it."""
    call = getattr(tbe._load(), name)
    given = [t(a) for t, a in zip(call.argtypes, args)]
    return lambda stream: call(*given, stream)


def norm_gradient(width):
    # 74 to 98 KB of shared memory, of one kernel: two vectors a thread
    gy, h, gh, gx = (randn(8, width).bfloat16() for _ in range(4))
    want, _ = tbe.tbe_rms_norm_backward(gy, h, grad_h=gh, eps=1e-6, need_weight=False)
    call = bound("tbe_rms_norm_backward", gy.data_ptr(), h.data_ptr(), None, gh.data_ptr(), BF16, 0,
                 8, width, width, width, width, 1e-6, gx.data_ptr(), width, None, None, 0)
    return call, gx, want, (gy, h, gh)


def norm(width):
    # 66 to 131 KB, four vectors a thread
    x, res = randn(700, width).bfloat16(), randn(700, width).bfloat16()
    y, h = torch.empty_like(x), torch.empty_like(x)
    want = tbe.tbe_rms_norm(x, residual=res, eps=1e-6)[0]
    call = bound("tbe_rms_norm", x.data_ptr(), res.data_ptr(), None, BF16, 0, 700, width, width,
                 width, 1e-6, h.data_ptr(), width, y.data_ptr(), width)
    return call, y, want, (x, res, h)


def embedding_gradient(width):
    # 41 and 49 KB: a ring, and the items of as many pieces as a CTA has groups of threads
    n, rows = 2000, 300
    grad, ids = randn(n, width).bfloat16(), torch.arange(n, device="cuda") * 7919 % rows
    out = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(tbe.tbe_embed_workspace_size(n, rows, width), dtype=torch.uint8, device="cuda")
    want = tbe.tbe_embed_backward(grad, ids, rows)
    call = bound("tbe_embed_backward", grad.data_ptr(), BF16, n, width, width, ids.data_ptr(), I64,
                 rows, 1.0, 0, out.data_ptr(), BF16, width, ws.data_ptr(), ws.numel())
    return call, out, want, (grad, ids, ws)


@pytest.mark.parametrize("make,widths", [
    (norm_gradient, (8192, 6144)), (norm, (16384, 8192)), (embedding_gradient, (8, 16))])
def test_calls_of_two_sizes_at_once(make, widths):
    made = [make(w) for w in widths]
    assert at_once([m[0] for m in made]) == {tbe.TBE_OK}
    assert all(torch.equal(got, want) for _, got, want, _ in made)


@pytest.mark.parametrize("make,large,small", [
    (norm_gradient, 8192, 6144), (norm, 16384, 8192), (embedding_gradient, 8, 16)])
def test_a_graph_outlives_smaller_calls(make, large, small):
    big, little = make(large), make(small)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        assert big[0](ctypes.c_void_p(stream.cuda_stream)) == tbe.TBE_OK
    for _ in range(2):
        assert little[0](None) == tbe.TBE_OK
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got, want) for _, got, want, _ in (big, little))
