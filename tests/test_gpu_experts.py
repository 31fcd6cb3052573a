"""Expert sort, dispatch, combine and their gradients on the GPU, against plain
64-bit forms written here.

Tolerances: a result summed in fp32 from t terms is off by at most t 2^-24
of the sum of |terms| for every rounding of a product or a partial sum (two a
term), and by half a unit in the last place of its type."""
import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]
HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def plan64(ids, experts):
    """The sort by counting, on the host."""
    flat = ids.reshape(-1).tolist()
    count = [0] * experts
    for e in flat:
        if 0 <= e < experts:
            count[e] += 1
    offsets = [0]
    for c in count:
        offsets.append(offsets[-1] + c)
    at, source, position = offsets[:-1].copy(), [-1] * len(flat), []
    for a, e in enumerate(flat):
        if 0 <= e < experts:
            position.append(at[e])
            source[at[e]] = a
            at[e] += 1
        else:
            position.append(-1)
    return offsets, source, position


def make_ids(tokens, k, experts, kind, dtype, seed=0):
    g = gen(seed)
    ids = torch.randint(0, experts, (tokens, k), generator=g, device="cuda")
    if kind == "drop":
        ids[torch.rand(tokens, k, generator=g, device="cuda") < 0.3] = -1
        ids[torch.rand(tokens, k, generator=g, device="cuda") < 0.05] = experts
    elif kind == "none":
        ids.fill_(-7)
    elif kind == "one":
        ids.fill_(experts - 1)
    elif kind == "far" and tokens:
        far = torch.iinfo(dtype)
        ids[0, 0], ids[-1, -1] = far.max, far.min
        if dtype == torch.int64:
            ids[tokens // 2, 0] = 1 << 32  # an expert's number in its low 32 bits
    return ids.to(dtype)


def check_plan(ids, experts, got):
    offsets, source, position = plan64(ids, experts)
    assert got[0].tolist() == offsets
    assert got[1].tolist() == source
    assert got[2].reshape(-1).tolist() == position
    assert got[2].shape == ids.shape


@pytest.mark.parametrize("tokens,k,experts", [
    (0, 2, 5), (1, 1, 1), (1, 8, 64), (31, 1, 3), (33, 3, 7), (1024, 2, 32), (4097, 3, 1024),
    (5000, 4, 257), (40001, 2, 64), (100003, 3, 1)])
@pytest.mark.parametrize("kind", ["all", "drop"])
def test_sort(tokens, k, experts, kind):
    for dtype in (torch.int32, torch.int64):
        ids = make_ids(tokens, k, experts, kind, dtype, seed=tokens + k)
        check_plan(ids, experts, tbe.tbe_expert_sort(ids, experts))


@pytest.mark.parametrize("kind", ["none", "one", "far"])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens", [3, 9000])
def test_sort_of_unusual_ids(kind, dtype, tokens):
    ids = make_ids(tokens, 2, 16, kind, dtype)
    check_plan(ids, 16, tbe.tbe_expert_sort(ids, 16))


def test_sort_of_more_assignments_than_any_split_holds():
    # against a stable sort: every expert's assignments in their order
    tokens, k, experts = 700_001, 5, 300
    ids = make_ids(tokens, k, experts, "drop", torch.int32, seed=3)
    offsets, source, position = tbe.tbe_expert_sort(ids, experts)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.sort(key, stable=True).indices
    kept = int((key < experts).sum())
    assert int(offsets[-1]) == kept and int(offsets[0]) == 0
    assert torch.equal(offsets.diff().long(), torch.bincount(key, minlength=experts + 1)[:experts])
    assert torch.equal(source[:kept].long(), order[:kept])
    assert bool((source[kept:] == -1).all())
    back = torch.full_like(flat, -1)
    back[order[:kept]] = torch.arange(kept, device="cuda")
    assert torch.equal(position.reshape(-1).long(), back)


def test_sort_of_many_assignments_in_a_graph():
    ids = make_ids(90_000, 3, 40, "drop", torch.int64, seed=1)
    o, s, p = tbe.tbe_expert_sort(ids, 40)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tbe.tbe_expert_sort(ids, 40, offsets=o, source=s, position=p)
    ids.copy_(make_ids(90_000, 3, 40, "drop", torch.int64, seed=2))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check_plan(ids, 40, (o, s, p))


def rows_of(tokens, width, dtype, seed, layout):
    """Rows in several layouts: dense, with a row stride, or off every 16-byte boundary."""
    g = gen(seed)
    data = torch.randn(tokens, width, generator=g, device="cuda").to(dtype)
    if layout == "dense":
        return data
    pad = {"strided": 24, "odd": 3}[layout]
    buf = torch.full((tokens * (width + pad) + 1,), float("nan"), dtype=dtype, device="cuda")
    at = 1 if layout == "odd" else 0
    view = buf[at:at + tokens * (width + pad)].view(tokens, width + pad)[:, :width]
    view.copy_(data)
    return view


def close(got, ref, terms, count, dtype):
    """count: roundings in fp32 on the way to each result."""
    bound = count * 2.0 ** -24 * terms + HALF_ULP[dtype] * (ref.abs() + terms * count * 2.0 ** -24) \
        + SMALLEST[dtype]
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), float((got.double() - ref).abs().max()))


def pool64(y, position, w):
    p = position.long()
    kept = p >= 0
    rows = y.double()[p.clamp_min(0)]
    rows = torch.where(kept[..., None], rows, 0.0)
    if w is not None:
        rows = rows * torch.where(kept, w.double(), 0.0)[..., None]
    return rows.sum(1), rows.abs().sum(1)


SHAPES = [(1, 1, 1, 1), (1, 2, 8, 1024), (5, 3, 4, 7), (64, 2, 16, 64), (257, 4, 5, 1001),
          (300, 8, 33, 264), (7, 32, 40, 48), (1000, 2, 8, 1030), (33, 1, 3, 4104),
          (3, 9, 12, 20001)]


@pytest.mark.parametrize("tokens,k,experts,width", SHAPES)
@pytest.mark.parametrize("layout", ["dense", "strided", "odd"])
def test_dispatch_and_combine(tokens, k, experts, width, layout):
    for dtype in DTYPES:
        ids = make_ids(tokens, k, experts, "drop" if tokens > 1 else "all", torch.int32, seed=width)
        offsets, source, position = tbe.tbe_expert_sort(ids, experts)
        kept = int(offsets[-1])
        x = rows_of(tokens, width, dtype, 1, layout)
        out = rows_of(tokens * k, width, dtype, 2, layout)
        rows = tbe.tbe_expert_dispatch(x, offsets, position, out=out)
        assert rows is out
        assert torch.equal(rows[:kept], x[(source[:kept] // k).long()])
        assert not rows[kept:].any()
        y = rows_of(tokens * k, width, dtype, 3, layout)
        w = torch.randn(tokens, k, generator=gen(4), device="cuda")
        for weights in (w, None):
            ref, terms = pool64(y, position, weights)
            got = tbe.tbe_expert_combine(y, position, weights,
                                         out=rows_of(tokens, width, dtype, 5, layout))
            close(got, ref, terms, 2 * k, dtype)
        ref, terms = pool64(y, position, None)
        close(tbe.tbe_expert_dispatch_backward(y, position), ref, terms, 2 * k, dtype)


@pytest.mark.parametrize("tokens,k,experts,width", SHAPES)
@pytest.mark.parametrize("layout", ["dense", "strided", "odd"])
def test_combine_backward(tokens, k, experts, width, layout):
    for dtype in DTYPES:
        ids = make_ids(tokens, k, experts, "drop" if tokens > 1 else "all", torch.int64, seed=k)
        offsets, source, position = tbe.tbe_expert_sort(ids, experts)
        kept = int(offsets[-1])
        g = rows_of(tokens, width, dtype, 1, layout)
        y = rows_of(tokens * k, width, dtype, 2, layout)
        w = torch.randn(tokens, k, generator=gen(4), device="cuda")
        src = source[:kept].long()
        for weights in (w, None):
            gy, gw = tbe.tbe_expert_combine_backward(
                g, y, offsets, position, weights, grad_y=rows_of(tokens * k, width, dtype, 3, layout))
            s = (torch.ones_like(w) if weights is None else w).reshape(-1)[src].double()
            ref = g.double()[src // k] * s[:, None]
            close(gy[:kept], ref, ref.abs(), 1, dtype)
            assert not gy[kept:].any()
            prods = g.double()[src // k] * y.double()[:kept]
            ref = torch.zeros(tokens * k, dtype=torch.float64, device="cuda")
            terms = torch.zeros_like(ref)
            ref[src], terms[src] = prods.sum(1), prods.abs().sum(1)
            close(gw.reshape(-1), ref, terms, width, torch.float32)


def test_one_gradient_without_the_other():
    tokens, k, width = 70, 2, 40
    ids = make_ids(tokens, k, 4, "drop", torch.int32, seed=3)
    offsets, _, position = tbe.tbe_expert_sort(ids, 4)
    g, y = (rows_of(n, width, torch.bfloat16, n, "dense") for n in (tokens, tokens * k))
    w = torch.randn(tokens, k, generator=gen(4), device="cuda")
    want_y, want_w = tbe.tbe_expert_combine_backward(g, y, offsets, position, w)
    got_y, got_w = torch.full_like(want_y, 9.0), torch.full_like(want_w, 9.0)
    stream = torch.cuda.current_stream().cuda_stream

    def call(y_, gy, gw):
        return tbe._load().tbe_expert_combine_backward(
            g.data_ptr(), y_, 4, tokens, k, width, width, width, offsets.data_ptr(), 4,
            position.data_ptr(), w.data_ptr(), gy, width, gw, stream)

    assert call(None, got_y.data_ptr(), None) == 0  # y is not read
    assert call(y.data_ptr(), None, got_w.data_ptr()) == 0
    assert call(None, None, None) == 0
    assert torch.equal(got_y, want_y) and torch.equal(got_w, want_w)


def test_gradients_against_differences():
    # combine is linear in y and in the weights, dispatch in x: central
    # differences of a scalar loss in fp64 give the gradients up to rounding
    tokens, k, experts, width = 6, 3, 4, 10
    ids = make_ids(tokens, k, experts, "drop", torch.int32, seed=8)
    offsets, source, position = tbe.tbe_expert_sort(ids, experts)
    y = rows_of(tokens * k, width, torch.float32, 1, "dense")
    w = torch.randn(tokens, k, generator=gen(2), device="cuda")
    g = rows_of(tokens, width, torch.float32, 3, "dense")

    def loss(y_, w_):
        return float((pool64(y_, position, w_)[0] * g.double()).sum())

    gy, gw = tbe.tbe_expert_combine_backward(g, y, offsets, position, w)
    h = 0.5
    for t, grad in ((y, gy), (w, gw)):
        for i in range(t.numel()):
            d = torch.zeros(t.numel(), device="cuda", dtype=torch.float64)
            d[i] = h
            up, down = t.double() + d.view(t.shape), t.double() - d.view(t.shape)
            f = (lambda v: loss(v, w)) if t is y else (lambda v: loss(y, v))
            assert abs((f(up) - f(down)) / (2 * h) - float(grad.reshape(-1)[i])) < 1e-5

    # dispatch: rows = P x, so its gradient is P^T
    x = rows_of(tokens, width, torch.float32, 5, "dense")
    gr = rows_of(tokens * k, width, torch.float32, 6, "dense")
    gx = tbe.tbe_expert_dispatch_backward(gr, position)
    one = torch.zeros_like(x)
    for n, c in [(0, 0), (3, 9), (5, 4)]:
        one.zero_()
        one[n, c] = 1.0
        diff = float((tbe.tbe_expert_dispatch(one, offsets, position).double() * gr.double()).sum())
        assert abs(diff - float(gx[n, c])) < 1e-5


def test_a_token_with_no_expert_and_values_behind_dropped_places():
    ids = torch.tensor([[-1, -1], [0, 9], [2, 0]], dtype=torch.int32, device="cuda")
    offsets, source, position = tbe.tbe_expert_sort(ids, 3)
    y = torch.ones(6, 40, device="cuda")
    y[3:] = float("nan")  # no kept place
    w = torch.full((3, 2), 2.0, device="cuda")
    w[0], w[1, 1] = float("nan"), float("inf")  # weights of dropped assignments
    out = tbe.tbe_expert_combine(y, position, w)
    assert out.tolist() == [[0.0] * 40, [2.0] * 40, [4.0] * 40]
    g = torch.ones(3, 40, device="cuda")
    g[0] = float("nan")  # its token has no expert
    gy, gw = tbe.tbe_expert_combine_backward(g, y, offsets, position, w)
    assert gy.tolist() == [[2.0] * 40] * 3 + [[0.0] * 40] * 3
    assert gw.tolist() == [[0.0, 0.0], [40.0, 0.0], [40.0, 40.0]]


@pytest.mark.parametrize("dtype", DTYPES)
def test_infinities_and_nan_stay_in_their_rows(dtype):
    ids = torch.tensor([[0, 1], [1, 0], [0, 1]], dtype=torch.int32, device="cuda")
    offsets, source, position = tbe.tbe_expert_sort(ids, 2)
    x = torch.randn(3, 24, device="cuda").to(dtype)
    x[1, 5], x[1, 6], x[2, 0] = float("inf"), float("nan"), -float("inf")
    rows = tbe.tbe_expert_dispatch(x, offsets, position)
    want = x[(source // 2).long()]
    assert torch.equal(torch.nan_to_num(rows), torch.nan_to_num(want))
    assert torch.equal(rows.isnan(), want.isnan())
    w = torch.tensor([[1.0, 0.5], [1.0, 1.0], [0.0, 1.0]], device="cuda")
    out = tbe.tbe_expert_combine(rows, position, w).float()
    assert out[1, 5] == float("inf") and out[1, 6].isnan()
    assert out[2, 0].isnan()  # 0 * -inf
    assert out[0].isfinite().all() and out[1, 7:].isfinite().all()


def test_positions_out_of_range_count_as_dropped():
    position = torch.tensor([[0, 99], [-5, 2]], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 1 << 30], dtype=torch.int32, device="cuda")
    y = torch.arange(1, 5, device="cuda").float()[:, None].repeat(1, 16)
    assert tbe.tbe_expert_combine(y, position)[:, 0].tolist() == [1.0, 3.0]
    out = torch.full((4, 16), 7.0, device="cuda")
    tbe.tbe_expert_dispatch(y[:2].contiguous(), offsets, position, out=out)
    assert out[:, 0].tolist() == [1.0, 7.0, 2.0, 7.0]


def test_rows_past_32_bit_element_offsets():
    tokens, width = 70_000, 32_776  # 2.3e9 elements
    ids = torch.randint(0, 4, (tokens, 1), device="cuda", dtype=torch.int32)
    offsets, source, position = tbe.tbe_expert_sort(ids, 4)
    x = torch.empty(tokens, width, dtype=torch.float16, device="cuda")
    x.copy_(torch.arange(tokens, device="cuda")[:, None] % 1024)
    rows = tbe.tbe_expert_dispatch(x, offsets, position)
    want = (source % 1024).half()
    for c in (0, width // 2, width - 1):
        assert torch.equal(rows[:, c], want)
    out = tbe.tbe_expert_combine(rows, position)
    assert torch.equal(out[:, ::4097], x[:, ::4097])
    gy, gw = tbe.tbe_expert_combine_backward(out, rows, offsets, position)
    assert torch.equal(gy[:, ::4097], rows[:, ::4097])


def test_another_stream_and_a_graph():
    tokens, k, experts, width = 512, 2, 8, 256
    ids = make_ids(tokens, k, experts, "drop", torch.int32)
    x = rows_of(tokens, width, torch.bfloat16, 1, "dense")
    w = torch.rand(tokens, k, device="cuda")

    def layer(stream=None):
        o, s, p = tbe.tbe_expert_sort(ids, experts, stream=stream)
        rows = tbe.tbe_expert_dispatch(x, o, p, stream=stream)
        return rows, tbe.tbe_expert_combine(rows, p, w, stream=stream)

    want = [t.clone() for t in layer()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    x2 = rows_of(tokens, width, torch.bfloat16, 9, "dense")
    ids.copy_(make_ids(tokens, k, experts, "drop", torch.int32, seed=5))
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    again = layer()
    assert all(torch.equal(a, b) for a, b in zip(held, again))
    assert not torch.equal(held[1], want[1])


def test_refusals_on_the_gpu():
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    o, s, p = tbe.tbe_expert_sort(ids, 2)
    x = torch.zeros(4, 16, device="cuda")
    for error, call in [
            (ValueError, lambda: tbe.tbe_expert_sort(ids, 0)),
            (ValueError, lambda: tbe.tbe_expert_sort(ids, 1025)),
            (ValueError, lambda: tbe.tbe_expert_sort(ids.t(), 2)),
            (ValueError, lambda: tbe.tbe_expert_sort(ids, 2, source=s[:-1])),
            (TypeError, lambda: tbe.tbe_expert_sort(ids, 2, offsets=o.long())),
            (ValueError, lambda: tbe.tbe_expert_dispatch(x[:3], o, p)),
            (ValueError, lambda: tbe.tbe_expert_dispatch(x.t().contiguous().t(), o, p)),
            (ValueError, lambda: tbe.tbe_expert_dispatch(x[:1].expand(4, 16), o, p)),
            (TypeError, lambda: tbe.tbe_expert_dispatch(x, o, p, out=x.half().repeat(2, 1))),
            (ValueError, lambda: tbe.tbe_expert_dispatch(x, o, p, out=x)),
            (TypeError, lambda: tbe.tbe_expert_dispatch(x, o, p.long())),
            (ValueError, lambda: tbe.tbe_expert_combine(x, p)),
            (TypeError, lambda: tbe.tbe_expert_combine(x.repeat(2, 1), p, torch.ones(4, 2).cuda().half())),
            (ValueError, lambda: tbe.tbe_expert_combine(x.repeat(2, 1), p, torch.ones(2, 4).cuda())),
            (TypeError, lambda: tbe.tbe_expert_combine_backward(x, x.repeat(2, 1).half(), o, p)),
            (ValueError, lambda: tbe.tbe_expert_combine_backward(x, x, o, p))]:
        with pytest.raises(error):
            call()
