"""8-bit rows, weights and the experts' products on the GPU.

Quantising is compared value by value with the same fp32 operations in torch
(scale: one multiplication; value: one division and one conversion).  The
products are compared with 64-bit ones of the same 8-bit values: a block's 128
exact products are summed in fp32 (128 roundings of at most 2^-23 of the sum
of |terms|, truncation allowed), the blocks' sums are scaled (three roundings
a block) and added, and the result is rounded to its type."""
import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]
HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FP8 = torch.float8_e4m3fn
TINY = 2.0 ** -126


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def quantize_rows_plain(x):
    rows, cols = x.shape
    pad = torch.nn.functional.pad(x.float(), (0, -cols % 128)).view(rows, -1, 128)
    inv = torch.tensor(1.0, device="cuda") / torch.tensor(448.0, device="cuda")
    s = (pad.abs().amax(2) * inv).clamp_min(TINY)
    return (pad / s[..., None]).view(rows, -1)[:, :cols].to(FP8), s


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 128), (17, 130), (64, 1024), (5, 4111)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_rows(rows, cols, dtype):
    x = (torch.randn(rows, cols, generator=gen(cols), device="cuda") *
         torch.exp(3 * torch.randn(rows, 1, generator=gen(1), device="cuda"))).to(dtype)
    x[0] = 0
    q, s = tbe.tbe_quantize_rows(x)
    wq, ws = quantize_rows_plain(x)
    assert torch.equal(s, ws)
    assert torch.equal(bits(q), bits(wq))
    # rows apart, and off every boundary
    buf = torch.zeros(rows * (cols + 5) + 1, dtype=dtype, device="cuda")
    view = buf[1:].view(rows, cols + 5)[:, :cols]
    view.copy_(x)
    out = torch.zeros(rows, cols + 3, dtype=torch.uint8, device="cuda")[:, :cols].view(FP8)
    q2, s2 = tbe.tbe_quantize_rows(view, out=out)
    assert torch.equal(s2, ws) and torch.equal(bits(q2), bits(wq))


def test_quantize_values_at_the_ends_of_the_range():
    x = torch.zeros(6, 128, device="cuda")
    x[0, 0], x[0, 1] = 3.4e38, 1e-30
    x[1, 3] = 1e-44                      # its scale would be zero
    x[2, 5], x[2, 6] = float("nan"), 2.0  # a NaN takes no part in the maximum
    x[3, 7], x[3, 8] = float("inf"), 2.0
    x[4] = torch.linspace(-1, 1, 128)
    q, s = tbe.tbe_quantize_rows(x)
    v = q.float() * s.repeat_interleave(128, 1)
    assert abs(float(v[0, 0]) / 3.4e38 - 1) < 1e-6 and float(v[0, 1]) == 0
    assert float(s[1, 0]) == TINY and float(v[1].abs().max()) <= 1e-42
    assert v[2, 5].isnan() and abs(float(v[2, 6]) - 2.0) < 1e-6 and int(v[2].isnan().sum()) == 1
    assert s[3, 0] == float("inf") and bool(v[3].isnan().all())  # its block is lost
    assert float((v[4] - x[4]).abs().max()) <= 2.0 ** -4
    assert not v[5].any() and float(s[5, 0]) == TINY


def quantize_weights_plain(w):
    e, n, k = w.shape
    pad = torch.nn.functional.pad(w.float(), (0, -k % 128, 0, -n % 128))
    t = pad.view(e, pad.shape[1] // 128, 128, pad.shape[2] // 128, 128)
    inv = torch.tensor(1.0, device="cuda") / torch.tensor(448.0, device="cuda")
    s = (t.abs().amax((2, 4)) * inv).clamp_min(TINY)
    q = (t / s[:, :, None, :, None]).view(pad.shape)[:, :n, :k].to(FP8)
    return q.contiguous(), s.contiguous()


@pytest.mark.parametrize("e,n,k", [(1, 1, 16), (3, 130, 144), (2, 256, 128), (5, 100, 1008)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_weights(e, n, k, dtype):
    w = torch.randn(e, n, k, generator=gen(n), device="cuda").to(dtype)
    q, s = tbe.tbe_quantize_weights(w)
    wq, ws = quantize_weights_plain(w)
    assert torch.equal(s, ws) and torch.equal(bits(q), bits(wq))
    # the transposed weights hold the same values
    qt, st = tbe.tbe_quantize_weights(w.transpose(1, 2).contiguous())
    assert torch.equal(bits(qt), bits(q.transpose(1, 2)))
    assert torch.equal(st, s.transpose(1, 2))


@pytest.mark.parametrize("tokens,k,experts,width", [
    (1, 2, 4, 128), (37, 3, 5, 200), (300, 2, 8, 1024), (64, 4, 6, 57)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_dispatch_fp8_is_dispatch_then_quantize(tokens, k, experts, width, dtype):
    ids = torch.randint(-1, experts, (tokens, k), generator=gen(2), device="cuda")
    o, src, p = tbe.tbe_expert_sort(ids, experts)
    x = torch.randn(tokens, width, generator=gen(3), device="cuda").to(dtype)
    q, s = tbe.tbe_expert_dispatch_fp8(x, o, p)
    wq, ws = quantize_rows_plain(tbe.tbe_expert_dispatch(x, o, p))
    assert torch.equal(s, ws) and torch.equal(bits(q), bits(wq))


def product64(a, sa, w, sw, offsets):
    """(result, sum of |terms|) in 64 bits."""
    K, n = a.shape[1], w.shape[1]
    col = torch.arange(K, device="cuda") // 128
    row = torch.arange(n, device="cuda") // 128
    out = torch.zeros(a.shape[0], n, dtype=torch.float64, device="cuda")
    terms = torch.zeros_like(out)
    av = a.double() * sa.double()[:, col]
    for e in range(w.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            wv = w[e].double() * sw[e].double()[row][:, col]
            out[lo:hi] = av[lo:hi] @ wv.T
            terms[lo:hi] = av[lo:hi].abs() @ wv.abs().T
    return out, terms


def check_product(sizes, n, k, dtype=torch.float32, rest=0, seed=0, a_pad=0, out_pad=0):
    rows, e = sum(sizes) + rest, len(sizes)
    x = torch.randn(rows, k, generator=gen(seed), device="cuda") * \
        torch.exp(torch.randn(rows, 1, generator=gen(seed + 1), device="cuda"))
    w = torch.randn(e, n, k, generator=gen(seed + 2), device="cuda") / k ** 0.5
    offsets = [0]
    for s in sizes:
        offsets.append(offsets[-1] + s)
    buf = torch.zeros(rows, k + a_pad, dtype=torch.uint8, device="cuda").view(FP8)[:, :k]
    a, sa = tbe.tbe_quantize_rows(x, out=buf)
    wq, sw = tbe.tbe_quantize_weights(w)
    out = torch.full((rows, n + out_pad), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = tbe.tbe_expert_product(a, sa, wq, sw, torch.tensor(offsets, dtype=torch.int32).cuda(),
                                 out=out[:, :n], status=status)
    assert int(status) == 0
    ref, terms = product64(a, sa, wq, sw, offsets)
    blocks = -(-k // 128)
    fp32 = (128 + 2 * blocks + 2) * 2.0 ** -23 * terms
    bound = fp32 + HALF_ULP[dtype] * (ref.abs() + fp32) + 1e-7 * (dtype == torch.float16) + TINY
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    assert not got[offsets[-1]:].any()
    if out_pad:
        assert bool(out[:, n:].isnan().all())  # nothing outside the columns was written
    return got


@pytest.mark.parametrize("sizes", [
    [1], [5], [128], [129], [300], [0, 3, 0, 0, 17], [1] * 40, [64, 0, 200, 1, 257], [1000, 31]])
@pytest.mark.parametrize("n,k", [(1, 16), (64, 128), (130, 144), (256, 512), (200, 1008)])
def test_product(sizes, n, k):
    check_product(sizes, n, k, seed=n + k)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [7, 96, 136, 1000])
def test_product_types_strides_and_unused_rows(dtype, n):
    check_product([40, 0, 170], n, 272, dtype, rest=37, a_pad=48, out_pad=5)
    check_product([40, 0, 170], n, 272, dtype, rest=300, out_pad=8)
    check_product([0, 0, 0], n, 64, dtype, rest=50)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,k", [(1000, 400), (1001, 128), (2048, 1200)])
def test_product_of_many_rows(n, k, dtype):
    # enough tiles for pairs of CTAs; experts of one row, of a part of a tile, of none
    check_product([9000, 0, 1, 257, 129, 200, 10613], n, k, dtype, rest=70, seed=k)
    check_product([20000], n, k, dtype, out_pad=8)


@pytest.mark.parametrize("rows,n,k", [(1, 4096, 7168), (16, 512, 4096), (2000, 384, 2048)])
def test_product_long_sums(rows, n, k):
    check_product([rows], n, k, torch.bfloat16)
    check_product([rows], n, k)


def test_product_many_experts_and_the_largest_number():
    sizes = [(i * 7) % 5 for i in range(1024)]
    check_product(sizes, 48, 64)


def test_product_past_32_bit_element_offsets():
    rows, n, k = 70_000, 32_768, 32  # 2.3e9 outputs
    a, sa = tbe.tbe_quantize_rows(torch.randn(rows, k, generator=gen(1), device="cuda"))
    w, sw = tbe.tbe_quantize_weights(torch.randn(1, n, k, generator=gen(2), device="cuda"))
    got = tbe.tbe_expert_product(a, sa, w, sw)
    for r in (0, 65_535, rows - 300):
        part = tbe.tbe_expert_product(a[r:r + 300], sa[r:r + 300].contiguous(), w, sw)
        assert torch.equal(got[r:r + 300], part)


def test_rows_do_not_depend_on_their_neighbours():
    # other rows and experts may hold NaN; a result may not
    sizes, n, k = [30, 70, 40], 200, 256
    x = torch.randn(140, k, generator=gen(5), device="cuda")
    w = torch.randn(3, n, k, generator=gen(6), device="cuda")
    offsets = torch.tensor([0, 30, 100, 140], dtype=torch.int32, device="cuda")
    w8, sw = tbe.tbe_quantize_weights(w)
    a8, sa = tbe.tbe_quantize_rows(x)
    want = tbe.tbe_expert_product(a8, sa, w8, sw, offsets)
    x2, w2 = x.clone(), w.clone()
    x2[30:100, 7], w2[1] = float("nan"), float("inf")
    a9, sa9 = tbe.tbe_quantize_rows(x2)
    w9, sw9 = tbe.tbe_quantize_weights(w2)
    got = tbe.tbe_expert_product(a9, sa9, w9, sw9, offsets)
    assert torch.equal(got[:30], want[:30]) and torch.equal(got[100:], want[100:])
    assert bool(got[30:100].isnan().all())


def test_input_gradient_is_the_product_with_transposed_weights():
    sizes, n, k = [50, 0, 77], 144, 272
    rows = sum(sizes)
    offsets = torch.tensor([0, 50, 50, 127], dtype=torch.int32, device="cuda")
    w = torch.randn(3, n, k, generator=gen(1), device="cuda") / n ** 0.5
    wt8, swt = tbe.tbe_quantize_weights(w.transpose(1, 2).contiguous())
    w8, sw = tbe.tbe_quantize_weights(w)
    g8, sg = tbe.tbe_quantize_rows(torch.randn(rows, n, generator=gen(2), device="cuda"))
    dx = tbe.tbe_expert_product(g8, sg, wt8, swt, offsets, out_dtype=torch.float32)
    # differences of sum(out * g) over the inputs, with the forward's own weight values
    col, row = torch.arange(k, device="cuda") // 128, torch.arange(n, device="cuda") // 128
    g = g8.double() * sg.double()[:, torch.arange(n, device="cuda") // 128]
    for r, e in [(0, 0), (49, 0), (50, 2), (126, 2)]:
        wv = w8[e].double() * sw[e].double()[row][:, col]

        def loss(v):
            return float((wv @ v) @ g[r])

        for c in (0, 127, 128, 271):
            up = torch.zeros(k, dtype=torch.float64, device="cuda")
            up[c] = 0.5
            assert abs((loss(up) - loss(-up)) - float(dx[r, c])) < 1e-4 * float(
                (wv[:, c].abs() * g[r].abs()).sum())


def test_malformed_offsets_stay_in_the_buffers():
    a, sa = tbe.tbe_quantize_rows(torch.randn(20, 32, device="cuda"))
    w, sw = tbe.tbe_quantize_weights(torch.randn(3, 16, 32, device="cuda"))
    for off in ([0, 1 << 30, 5, 20], [-4, 10, -1, 99], [30, 40, 50, 60], [0, 0, 0, -9]):
        out = torch.full((22, 16), 7.0, device="cuda")
        tbe.tbe_expert_product(a, sa, w, sw, torch.tensor(off, dtype=torch.int32).cuda(),
                               out=out[1:21])
        assert bool((out[0] == 7).all()) and bool((out[21] == 7).all())


def test_another_stream_and_a_graph():
    offsets = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    x = torch.randn(64, 256, generator=gen(1), device="cuda")
    w8, sw = tbe.tbe_quantize_weights(torch.randn(2, 128, 256, generator=gen(2), device="cuda"))

    def step(stream=None):
        q, s = tbe.tbe_quantize_rows(x, stream=stream)
        return tbe.tbe_expert_product(q, s, w8, sw, offsets, stream=stream)

    want = step().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x.mul_(-2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, -2.0 * want)


def test_refusals_on_the_gpu():
    a, sa = tbe.tbe_quantize_rows(torch.zeros(8, 32, device="cuda"))
    w, sw = tbe.tbe_quantize_weights(torch.zeros(2, 16, 32, device="cuda"))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    odd, sodd = tbe.tbe_quantize_rows(torch.zeros(8, 24, device="cuda"))
    wodd, swodd = tbe.tbe_quantize_weights(torch.zeros(2, 16, 24, device="cuda"))
    for error, call in [
            (ValueError, lambda: tbe.tbe_expert_product(a, sa, w, sw)),  # two experts, no offsets
            (ValueError, lambda: tbe.tbe_expert_product(a, sa, w, sw, off[:2])),
            (ValueError, lambda: tbe.tbe_expert_product(a, sa[:4], w, sw, off)),
            (ValueError, lambda: tbe.tbe_expert_product(a, sa, w, sw[:1], off)),
            (ValueError, lambda: tbe.tbe_expert_product(a, sa, w.transpose(1, 2), sw, off)),
            (TypeError, lambda: tbe.tbe_expert_product(a.float(), sa, w, sw, off)),
            (TypeError, lambda: tbe.tbe_expert_product(a, sa, w, sw, off, out_dtype=torch.int8)),
            (tbe.TBEError, lambda: tbe.tbe_expert_product(odd, sodd, wodd, swodd, off))]:
        with pytest.raises(error):
            call()
