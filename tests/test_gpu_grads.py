"""Global gradient norm and clipping on the GPU, against 64-bit forms.

Tolerance of the norm: each thread sums at most 128 squares in fp32 before
fp64 takes over, so the sum is off by at most 129 * 2^-24 of itself and the
norm by half of that, 2^-18 with the last roundings."""
import math

import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu

NORM_TOL = 2.0 ** -18
HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}


def norm64(grads):
    return math.sqrt(sum(float(g.double().pow(2).sum()) for g in grads))


def check(grads, max_norm, got_norm, got):
    want = norm64(grads)
    assert abs(float(got_norm) - want) <= NORM_TOL * want
    c = min(1.0, max_norm / (want + 1e-6))
    for g, o in zip(grads, got):
        ref = g.double() * c
        bound = (NORM_TOL + 2.0 ** -22 + HALF_ULP[g.dtype]) * ref.abs() + SMALLEST[g.dtype]
        assert bool(((o.double() - ref).abs() <= bound).all())


def make(sizes, dtypes, seed=0, loud=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * loud).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


ALL = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("sizes", [
    [1], [0, 3], [7, 1, 31, 8191, 8192, 8193], [100_003], [5_000_001, 17], [33] * 700,
    list(range(1, 400)), [1 << 22] * 3])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip_in_place_and_out_of_place(sizes, max_norm):
    grads = make(sizes, ALL, seed=len(sizes))
    out = [torch.full_like(g, 3.0) for g in grads]
    kept = [g.clone() for g in grads]
    norm = tbe.tbe_grad_clip(grads, max_norm, out=out)
    check(kept, max_norm, norm, out)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))  # the gradients are left alone
    assert torch.equal(tbe.tbe_grad_norm(grads), norm)
    norm2 = tbe.tbe_grad_clip(grads, max_norm)
    assert torch.equal(norm2, norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, out))


def test_the_same_bits_each_time():
    grads = make([1_000_003, 77, 65_536], ALL, seed=1)
    first = tbe.tbe_grad_norm(grads)
    assert all(torch.equal(tbe.tbe_grad_norm(grads), first) for _ in range(5))


@pytest.mark.parametrize("loud", [1e-44, 1e-30, 1e-19, 1e-10, 1e10, 1e19, 1e30, 1e36])
def test_norm_over_the_whole_range_of_fp32(loud):
    grads = make([50_000, 33], [torch.float32], seed=2, loud=loud)
    want = norm64(grads)
    got = float(tbe.tbe_grad_norm(grads))
    assert abs(got - want) <= NORM_TOL * want + 2.0 ** -149


def test_loud_and_quiet_tensors_together():
    grads = make([4096] * 3, [torch.float32], seed=4)
    grads[0] *= 1e25
    grads[2] *= 1e-25
    want = norm64(grads)
    assert abs(float(tbe.tbe_grad_norm(grads)) - want) <= NORM_TOL * want


def test_zeros_infinities_and_nan():
    z = [torch.zeros(10_000, device="cuda"), torch.zeros(3, device="cuda", dtype=torch.float16)]
    assert float(tbe.tbe_grad_clip(z, 1.0)) == 0.0
    assert not z[0].any()
    g = make([1000, 50], [torch.float32])
    g[1][7] = float("inf")
    out = [torch.empty_like(t) for t in g]
    assert float(tbe.tbe_grad_clip(g, 1.0, out=out)) == float("inf")
    assert not out[0].any() and out[1][7].isnan()  # 0 * inf
    g[0][3] = float("nan")
    assert torch.isnan(tbe.tbe_grad_clip(g, 1.0, out=out))
    assert bool(out[0].isnan().all())


def test_max_norm_zero_clears():
    g = make([5000], [torch.bfloat16])
    tbe.tbe_grad_clip(g, 0.0)
    assert not g[0].any()


def test_addresses_off_every_boundary_and_other_orders_of_dimensions():
    base = torch.randn(100_100, device="cuda")
    for dtype in ALL:
        flat = base.to(dtype)
        grads = [flat[1:1 + n] if n < 9000 else flat[n % 7:n] for n in (5, 8195, 100_001)]
        grads = [g.clone()[:] if i == 0 else g for i, g in enumerate(grads)]
        out_flat = torch.zeros(300_000, dtype=dtype, device="cuda")
        at, out = 3, []
        for g in grads:
            out.append(out_flat[at:at + g.numel()])
            at += g.numel() + 5
        check(grads, 1.0, tbe.tbe_grad_clip(grads, 1.0, out=out), out)
        # nothing outside the tensors was written
        mask = torch.ones_like(out_flat, dtype=torch.bool)
        at = 3
        for g in grads:
            mask[at:at + g.numel()] = False
            at += g.numel() + 5
        assert not out_flat[mask].any()
    t = torch.randn(40, 30, device="cuda").t()
    cl = torch.randn(2, 8, 5, 5, device="cuda").to(memory_format=torch.channels_last)
    kept = [t.clone(), cl.clone()]
    norm = tbe.tbe_grad_clip([t, cl], 0.25)
    check(kept, 0.25, norm, [t, cl])


def test_more_than_2_31_elements():
    n = (1 << 31) + 12_345
    g = torch.empty(n, dtype=torch.float16, device="cuda").fill_(0.5)
    g[-1] = 3.0
    norm = tbe.tbe_grad_clip([g], 1.0)
    want = math.sqrt((n - 1) * 0.25 + 9.0)
    assert abs(float(norm) - want) <= NORM_TOL * want
    c = torch.tensor(0.5 / want, dtype=torch.float64)
    for i in (0, n // 2, n - 2):
        assert abs(float(g[i]) - float(c)) <= 2.0 ** -24


def test_another_stream_and_a_graph():
    grads = make([70_000, 11], [torch.float32, torch.bfloat16], seed=6)
    out = [torch.empty_like(g) for g in grads]
    want = tbe.tbe_grad_clip(grads, 1.0, out=out).clone()
    kept = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm = tbe.tbe_grad_clip(grads, 1.0, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, kept))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = tbe.tbe_grad_clip(grads, 1.0, out=out)
    grads[0].mul_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    check(grads, 1.0, held, out)


def test_refusals_on_the_gpu():
    g = torch.zeros(8, 8, device="cuda")
    for error, call in [
            (ValueError, lambda: tbe.tbe_grad_norm([g[:, :4]])),
            (ValueError, lambda: tbe.tbe_grad_norm([g[0].expand(8, 8)])),
            (TypeError, lambda: tbe.tbe_grad_norm([g.double()])),
            (ValueError, lambda: tbe.tbe_grad_norm([g], norm=torch.zeros(2, device="cuda"))),
            (ValueError, lambda: tbe.tbe_grad_clip([g], 1.0, out=[g.half()])),
            (ValueError, lambda: tbe.tbe_grad_clip([g], 1.0, out=[torch.zeros(8, 8).cuda().t()])),
            (tbe.TBEError, lambda: tbe.tbe_grad_clip([g], -1.0)),
            (tbe.TBEError, lambda: tbe.tbe_grad_clip([g], float("nan"))),
            (tbe.TBEError, lambda: tbe.tbe_grad_norm([g], ws=torch.zeros(64, dtype=torch.uint8).cuda()))]:
        with pytest.raises(error):
            call()
