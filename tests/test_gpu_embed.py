"""Token embedding and its table's gradient on the GPU, against plain 64-bit forms
written here.

Tolerances: scale * row is one fp32 product rounded to the type, so it equals
the same two roundings in torch.  A sum of t rows in fp32 has t - 1 additions, the scale
and, when it is added to a table, one more: off by at most (t + 1) 2^-24 of scale times
the sum of |terms| (plus 2^-24 of the table's entry), and by half a unit in the last
place of its type (half the smallest subnormal below its normals)."""
import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def make_ids(n, rows, kind, dtype, g):
    if kind == "uniform":
        ids = torch.randint(0, max(rows, 1), (n,), generator=g, device="cuda")
    elif kind == "one":
        ids = torch.full((n,), rows - 1, device="cuda")
    elif kind == "none":
        ids = torch.full((n,), -3, device="cuda")
    elif kind == "few":  # long runs, and padding
        ids = torch.randint(-1, min(rows, 3), (n,), generator=g, device="cuda")
    else:  # far: ids that are rows in their low 32 bits only, and the type's ends
        ids = torch.randint(-2, rows + 2, (n,), generator=g, device="cuda")
        if dtype == torch.int64 and n > 4:
            ids[0], ids[1] = 1 << 32, -(1 << 32)
        if n > 4:
            ids[2], ids[3] = torch.iinfo(dtype).max, torch.iinfo(dtype).min
    return ids.to(dtype)


def plain(table, ids, scale):
    rows = table.shape[0]
    on = (ids >= 0) & (ids < rows)
    if rows == 0:
        return torch.zeros(ids.numel(), table.shape[1], dtype=table.dtype, device="cuda")
    out = table[ids.clamp(0, rows - 1).long()].float() * torch.tensor(scale, device="cuda")
    return torch.where(on[:, None], out, 0.0).to(table.dtype)


@pytest.mark.parametrize("n,rows,width", [
    (0, 5, 8), (1, 1, 1), (3, 7, 5), (4, 100, 1024), (33, 50, 8), (257, 1000, 1001),
    (1000, 3, 24), (70, 9, 4099), (5000, 300, 136), (2, 0, 16), (3, 4, 0)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_lookup(n, rows, width, dtype):
    g = gen(n + width)
    table = randn(g, rows, width).to(dtype)
    for kind, id_type, scale in (("uniform", torch.int64, 1.0), ("far", torch.int32, 0.37),
                                 ("far", torch.int64, -45.25)):
        if rows == 0 and kind == "uniform":
            kind = "none"
        ids = make_ids(n, rows, kind, id_type, g)
        assert torch.equal(tbe.tbe_embed(table, ids, scale), plain(table, ids, scale))


def test_lookup_of_ids_of_any_shape():
    g = gen(0)
    table = randn(g, 20, 16)
    ids = torch.randint(0, 20, (2, 3, 5), generator=g, device="cuda")
    assert torch.equal(tbe.tbe_embed(table, ids), table[ids])
    one = torch.tensor(7, device="cuda")
    assert torch.equal(tbe.tbe_embed(table, one), table[7])


def test_lookup_keeps_every_value_at_scale_one():
    table = torch.tensor([[float("inf"), -0.0, float("-inf"), 2.0 ** -149, 3.4e38, 1.0, 2.0, 3.0]],
                         device="cuda")
    got = tbe.tbe_embed(table, torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert torch.equal(got.view(torch.int32), table.expand(2, -1).contiguous().view(torch.int32))
    nan = torch.full((1, 8), float("nan"), device="cuda")
    assert bool(tbe.tbe_embed(nan, torch.zeros(1, dtype=torch.int32, device="cuda")).isnan().all())
    # a row that is not looked up is not touched
    table = torch.cat([nan, torch.ones(1, 8, device="cuda")])
    assert torch.equal(tbe.tbe_embed(table, torch.tensor([1, -1, 2], device="cuda")),
                       torch.tensor([[1.0], [0.0], [0.0]], device="cuda").expand(3, 8))


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 3), (5, 1)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_lookup_and_gradient_of_strided_rows(dtype, pad, shift):
    g = gen(pad)
    wide = randn(g, 40, 136 + pad).to(dtype)
    table = wide[:, shift:shift + 136]
    ids = make_ids(333, 40, "far", torch.int64, g)
    room = torch.full((333, 140), 7.0, dtype=dtype, device="cuda")
    got = tbe.tbe_embed(table, ids, 2.0, out=room[:, 2:138])
    assert torch.equal(got, plain(table, ids, 2.0))
    assert bool((room[:, :2] == 7).all()) and bool((room[:, 138:] == 7).all())
    grad = randn(g, 333, 136 + pad).to(dtype)[:, shift:shift + 136]
    into = torch.full((40, 140), 7.0, dtype=dtype, device="cuda")
    tbe.tbe_embed_backward(grad, ids, 40, 2.0, out=into[:, 2:138])
    check_gradient(into[:, 2:138], grad, ids, 40, 2.0)
    assert bool((into[:, :2] == 7).all()) and bool((into[:, 138:] == 7).all())


def test_rows_past_32_bits():
    rows, width = (1 << 31) // 512 + 10, 1024  # 4.3 billion elements
    table = torch.zeros(rows, width, dtype=torch.float16, device="cuda")
    ids = torch.tensor([rows - 1, 0, rows // 2 + 1, -1], device="cuda")
    table[ids[:3]] = torch.arange(1, 4, device="cuda", dtype=torch.float16)[:, None]
    got = tbe.tbe_embed(table, ids)
    assert got[:, 0].tolist() == [1, 2, 3, 0] and torch.equal(got, got[:, :1].expand(-1, width))
    grad = torch.ones(4, width, dtype=torch.float16, device="cuda")
    tbe.tbe_embed_backward(grad, ids, rows, out=table)
    assert bool((table[ids[:3]] == 1).all())
    assert float(table.sum(dtype=torch.float32)) == 3 * width


def check_gradient(got, grad, ids, rows, scale, before=None):
    ids = ids.reshape(-1).long()
    kept = (ids >= 0) & (ids < rows)
    to, terms = ids[kept], grad[kept].double()
    width = grad.shape[1]
    ref = torch.zeros(rows, width, dtype=torch.float64, device="cuda")
    size, count = ref.clone(), torch.zeros(rows, 1, dtype=torch.float64, device="cuda")
    ref.index_add_(0, to, terms)
    size.index_add_(0, to, terms.abs())
    count.index_add_(0, to, torch.ones(to.numel(), 1, dtype=torch.float64, device="cuda"))
    ref, size = ref * scale, size * abs(scale)
    bound = (count + 1) * 2.0 ** -24 * size
    if before is not None:
        ref = ref + before.double()
        bound += 2.0 ** -24 * before.double().abs()
    half = torch.finfo(got.dtype).eps / 2
    bound += half * (ref.abs() + bound) + SMALLEST[got.dtype] / 2
    if before is None:
        bound[count[:, 0] == 0] = 0
    assert bool(((got.double() - ref).abs() <= bound).all())
    untouched = count[:, 0] == 0
    if before is not None:
        assert torch.equal(got[untouched], before[untouched])


@pytest.mark.parametrize("n,rows,width", [
    (1, 1, 1), (1, 5, 8), (31, 4, 3), (33, 1000, 64), (64, 2, 1001), (700, 513, 128),
    (4097, 1023, 40), (6000, 70_000, 17), (2050, 5, 2056), (3000, 1 << 20, 8)])
@pytest.mark.parametrize("kind", ["uniform", "few", "far"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient(n, rows, width, kind, dtype):
    g = gen(n)
    ids = make_ids(n, rows, kind, torch.int64, g)
    grad = randn(g, n, width).to(dtype)
    for out in {dtype, torch.float32}:
        got = tbe.tbe_embed_backward(grad, ids, rows, 0.7, out_dtype=out)
        assert got.dtype == out
        check_gradient(got, grad, ids, rows, 0.7)
        again = tbe.tbe_embed_backward(grad, ids.int() if kind != "far" else ids, rows, 0.7,
                                       out_dtype=out)
        assert torch.equal(got, again)


@pytest.mark.parametrize("n", [5, 100, 3000, 20_000])
@pytest.mark.parametrize("kind", ["one", "none"])
def test_gradient_of_one_row_and_of_none(n, kind):
    ids = make_ids(n, 37, kind, torch.int32, None)
    grad = randn(gen(1), n, 264).bfloat16()
    check_gradient(tbe.tbe_embed_backward(grad, ids, 37), grad, ids, 37, 1.0)


def test_gradient_without_tokens():
    out = torch.full((6, 9), 3.0, device="cuda")
    none = torch.zeros(0, 9, device="cuda")
    ids = torch.zeros(0, dtype=torch.int64, device="cuda")
    tbe.tbe_embed_backward(none, ids, 6, out=out, accumulate=True)
    assert bool((out == 3).all())
    tbe.tbe_embed_backward(none, ids, 6, out=out)
    assert bool((out == 0).all())
    assert tbe.tbe_embed_backward(none, ids, 0).shape == (0, 9)


@pytest.mark.parametrize("n,rows,width", [(7, 5, 24), (5000, 300, 129), (9000, 40, 256)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_is_added(n, rows, width, dtype):
    g = gen(rows)
    ids = make_ids(n, rows, "far", torch.int64, g)
    ids[ids == 4] = 3  # a row without tokens
    grad = randn(g, n, width).to(dtype)
    for out in {dtype, torch.float32}:
        before = randn(g, rows, width).to(out)
        got = before.clone()
        assert tbe.tbe_embed_backward(grad, ids, rows, 1.5, out=got, accumulate=True) is got
        check_gradient(got, grad, ids, rows, 1.5, before)


def test_gradient_of_many_tokens():
    # past what one cluster sorts: three launches a pass, two and three passes
    n, width = 300_001, 24
    g = gen(5)
    grad = randn(g, n, width)
    for rows, kind in ((1000, "uniform"), (1 << 21, "uniform"), (50_000, "few")):
        ids = make_ids(n, rows, kind, torch.int32, g)
        check_gradient(tbe.tbe_embed_backward(grad, ids, rows), grad, ids, rows, 1.0)


@pytest.mark.parametrize("n", [98_304, 98_305, 163_840, 163_841])
def test_gradient_around_the_limits_of_one_launch(n):
    rows, width = 40_000, 24
    g = gen(n)
    ids, grad = make_ids(n, rows, "far", torch.int64, g), randn(g, n, width).half()
    check_gradient(tbe.tbe_embed_backward(grad, ids, rows, 0.5), grad, ids, rows, 0.5)
    before = randn(g, rows, width)
    got = before.clone()
    tbe.tbe_embed_backward(grad, ids, rows, 0.5, out=got, accumulate=True)
    check_gradient(got, grad, ids, rows, 0.5, before)


@pytest.mark.parametrize("rows,width,pad", [
    (110_000, 2000, 0), (52_000, 2048, 8), (60_001, 4097, 3)])
def test_gradient_into_large_results(rows, width, pad):
    # cleared in more CTAs above 400 MB; rows side by side and apart
    n = 3000
    g = gen(rows)
    room = torch.full((rows, width + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    ids = make_ids(n, rows, "far", torch.int64, g)
    grad = torch.randint(-8, 9, (n, width), generator=g, device="cuda").bfloat16()
    got = tbe.tbe_embed_backward(grad, ids, rows, out=room[:, :width])
    kept = ids[(ids >= 0) & (ids < rows)]
    some = kept.unique()
    for row in some[:20].tolist():
        assert torch.equal(got[row], grad[ids == row].sum(0, dtype=torch.float32).bfloat16())
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[some] = False
    assert not bool(got[others].any()) and bool((room[:, width:] == 7).all())


@pytest.mark.parametrize("lengths", [
    [8], [16], [24], [9], [7, 8, 9], [1, 15], [15, 1], [64, 65, 130, 1, 2, 17, 8, 8, 16, 7],
    [3, 1000, 5], [1200], [31, 33, 32]])
@pytest.mark.parametrize("width", [3, 40, 264])
def test_gradient_of_runs_that_end_at_every_place(lengths, width):
    # of the sorted tokens: at the pieces' boundaries, before and behind them
    ids, row = [], 0
    while len(ids) < 1500:
        ids += [row] * lengths[row % len(lengths)]
        row += 1
    for lead in (0, 1, 5):
        g = gen(lead)
        t = torch.tensor([row + 1] * lead + ids, device="cuda")
        t = t[torch.randperm(t.numel(), generator=g, device="cuda")]
        grad = randn(g, t.numel(), width)
        check_gradient(tbe.tbe_embed_backward(grad, t, row + 2), grad, t, row + 2, 1.0)
        half = grad.half()
        check_gradient(tbe.tbe_embed_backward(half, t, row + 2), half, t, row + 2, 1.0)


def test_two_gradients_at_once():
    n, rows, width = 30_000, 900, 128
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [(make_ids(n, rows, "far", torch.int64, gen(i)), randn(gen(i + 5), n, width))
            for i in range(2)]
    want = [tbe.tbe_embed_backward(grad, ids, rows) for ids, grad in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [tbe.tbe_embed_backward(grad, ids, rows, stream=s)
               for (ids, grad), s in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_many_gradients_are_added():
    # past what one cluster sorts, into what an output layer has left
    n, rows, width = 120_001, 3000, 40
    g = gen(12)
    ids, grad = make_ids(n, rows, "far", torch.int32, g), randn(g, n, width).bfloat16()
    ids[ids == 7] = 8
    before = randn(g, rows, width)
    got = before.clone()
    tbe.tbe_embed_backward(grad, ids, rows, 0.5, out=got, accumulate=True)
    check_gradient(got, grad, ids, rows, 0.5, before)


def test_a_padding_rows_gradient_is_not_used():
    ids = torch.tensor([2, -1, 2, 9], device="cuda")
    grad = torch.ones(4, 16, device="cuda")
    grad[1], grad[3] = float("nan"), float("inf")
    got = tbe.tbe_embed_backward(grad, ids, 4)
    assert got[:, 0].tolist() == [0, 0, 2, 0] and bool(got.isfinite().all())


def test_gradient_against_differences():
    # of the 64-bit plain lookup: linear in the table, so a difference is exact
    g = gen(8)
    rows, width, n = 6, 5, 40
    ids = torch.randint(-1, rows, (n,), generator=g, device="cuda")
    grad = randn(g, n, width)
    got = tbe.tbe_embed_backward(grad, ids, rows, 1.25)

    def loss(table):
        out = torch.where((ids >= 0)[:, None], table[ids.clamp_min(0)] * 1.25, 0.0)
        return (out * grad.double()).sum()

    for r in range(rows):
        for c in range(width):
            d = torch.zeros(rows, width, dtype=torch.float64, device="cuda")
            d[r, c] = 1.0
            assert abs(float(loss(d) - loss(-d)) / 2 - float(got[r, c])) < 40 * 2.0 ** -24 * 40 * 4


def test_in_a_graph_on_a_stream_with_a_workspace():
    n, rows, width = 5000, 700, 96
    g = gen(3)
    ids, grad = make_ids(n, rows, "far", torch.int64, g), randn(g, n, width)
    table = randn(g, rows, width)
    ws = torch.empty(tbe.tbe_embed_workspace_size(n, rows, width), dtype=torch.uint8,
                     device="cuda")
    out, got = torch.empty(n, width, device="cuda"), torch.empty(rows, width, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tbe.tbe_embed(table, ids, out=out, stream=side)
    tbe.tbe_embed_backward(grad, ids, rows, out=got, ws=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, plain(table, ids, 1.0))
    check_gradient(got, grad, ids, rows, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tbe.tbe_embed(table, ids, 3.0, out=out)
        tbe.tbe_embed_backward(grad, ids, rows, 3.0, out=got, ws=ws)
    for seed in (10, 11):
        ids.copy_(make_ids(n, rows, "few", torch.int64, gen(seed)))
        grad.copy_(randn(gen(seed), n, width))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, plain(table, ids, 3.0))
        check_gradient(got, grad, ids, rows, 3.0)
