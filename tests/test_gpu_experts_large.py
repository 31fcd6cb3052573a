"""Batches that fill the GPU take other launches than small ones: the gradients of combine a group
a token, four of its rows at a time, and groups of a quarter of the threads for rows, in dispatch
and combine.  Both with dropped assignments, weights, numbers of rows that are no multiple of four,
rows off 16-byte boundaries and tokens that end inside a warp, against 64-bit forms.

Tolerances: as a result summed in fp32 from t terms, 2 t roundings of 2^-24 of the sum of |terms|,
and half a unit in the last place of its type."""
import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]
HALF_ULP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}

# (tokens, k, experts, width): narrow rows of parts of a warp, a warp's, and wide ones
SHAPES = [(5003, 3, 16, 32), (5001, 5, 7, 264), (4099, 2, 9, 600), (2500, 5, 9, 2048),
          (3001, 1, 4, 1032), (1300, 9, 33, 4104), (65539, 4, 64, 8)]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def by_token(tokens, width, dtype):
    """Rows on 16-byte boundaries, enough tokens for 24 warps a multiprocessor."""
    size = torch.empty(0, dtype=dtype).element_size()
    return width * size % 16 == 0 and tokens * -(-width * size // 512) >= 152 * 24


def problem(tokens, k, experts, width, dtype, pad=0):
    g = gen(width + k)
    ids = torch.randint(0, experts, (tokens, k), generator=g, device="cuda")
    ids[torch.rand(tokens, k, generator=g, device="cuda") < 0.2] = -1
    ids[tokens // 3] = -1  # a token without an expert
    offsets, source, position = tbe.tbe_expert_sort(ids, experts)

    def rows(n):
        return torch.randn(n, width + pad, generator=g, device="cuda").to(dtype)[:, :width]

    weights = torch.randn(tokens, k, generator=g, device="cuda")
    weights[position < 0] = float("nan")  # not read
    return offsets, source, position, rows, weights


def close(got, ref, terms, count, dtype):
    fp32 = count * 2.0 ** -24 * terms
    bad = ~((got.double() - ref).abs() <= fp32 + HALF_ULP[dtype] * (ref.abs() + fp32) +
            SMALLEST[dtype])
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


def test_the_shapes_reach_the_launch_a_token():
    reached = {(s, d) for s in SHAPES for d in DTYPES if by_token(s[0], s[3], d)}
    assert len({s for s, _ in reached}) >= 6 and {d for _, d in reached} == set(DTYPES)


@pytest.mark.parametrize("tokens,k,experts,width", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_combine_backward(tokens, k, experts, width, dtype, pad):
    offsets, source, position, rows, w = problem(tokens, k, experts, width, dtype, pad)
    kept = int(offsets[-1])
    g, y = rows(tokens), rows(tokens * k)
    src = source[:kept].long()
    for weights in (w, None):
        gy = torch.full((tokens * k, width + pad), 3.0, dtype=dtype, device="cuda")
        gy, gw = tbe.tbe_expert_combine_backward(g, y, offsets, position, weights,
                                                 grad_y=gy[:, :width])
        s = (torch.ones_like(w) if weights is None else w).reshape(-1)[src].double()
        ref = g.double()[src // k] * s[:, None]
        close(gy[:kept], ref, ref.abs(), 1, dtype)
        assert not gy[kept:].any()
        products = g.double()[src // k] * y.double()[:kept]
        ref = torch.zeros(tokens * k, dtype=torch.float64, device="cuda")
        terms = torch.zeros_like(ref)
        ref[src], terms[src] = products.sum(1), products.abs().sum(1)
        close(gw.reshape(-1), ref, terms, 2 * width, torch.float32)
        # the same bits again, and one gradient without the other
        again = [torch.full_like(gy, 9.0), torch.full_like(gw, 9.0)]
        dt = {torch.float16: 1, torch.bfloat16: 4, torch.float32: 5}[dtype]

        def call(y_, gy_, gw_):
            return tbe._load().tbe_expert_combine_backward(
                g.data_ptr(), y_, dt, tokens, k, width, g.stride(0), y.stride(0),
                offsets.data_ptr(), experts, position.data_ptr(),
                None if weights is None else weights.data_ptr(), gy_, again[0].stride(0), gw_,
                torch.cuda.current_stream().cuda_stream)

        assert call(None, again[0].data_ptr(), None) == 0
        assert call(y.data_ptr(), None, again[1].data_ptr()) == 0
        assert torch.equal(again[0], gy)
        # (alone, its rows' vectors begin on y's boundaries: another order of the sum)
        if pad % 8 == 0 and width * g.element_size() % 16 == 0:
            assert torch.equal(again[1], gw)
        else:
            close(again[1].reshape(-1), ref, terms, 2 * width, torch.float32)


@pytest.mark.parametrize("tokens,k,experts,width", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_dispatch_and_combine(tokens, k, experts, width, dtype, pad):
    offsets, source, position, rows, w = problem(tokens, k, experts, width, dtype, pad)
    kept = int(offsets[-1])
    x, y = rows(tokens), rows(tokens * k)
    out = torch.full((tokens * k, width + pad), 3.0, dtype=dtype, device="cuda")
    tbe.tbe_expert_dispatch(x, offsets, position, out=out[:, :width])
    assert torch.equal(out[:kept, :width], x[(source[:kept] // k).long()])
    assert not out[kept:, :width].any() and bool((out[:, width:] == 3.0).all())
    p = position.long()
    for weights in (w, None):
        v = y.double()[p.clamp_min(0)]
        v = v if weights is None else v * w.double()[..., None]
        v = torch.where((p >= 0)[..., None], v, 0.0)
        got = tbe.tbe_expert_combine(y, position, weights)
        close(got, v.sum(1), v.abs().sum(1), 2 * k, dtype)
