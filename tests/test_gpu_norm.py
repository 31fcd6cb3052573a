"""Root-mean-square norm and its gradients on the GPU, against plain 64-bit forms
written here.

Tolerances, in units u = 2^-24: a row's squares are summed by at most 64 additions a
thread, 5 in a warp and 16 over the warps, 1 / sqrt halves that error and adds 4, the division, eps
and the two products add 4: below 64 u = 2^-18 relative to the result, plus half a unit in
the last place of its type.  The gradient's dot product has the same additions and two
products more a term, so each of its terms is off by less than 2^-17 of its magnitude.  A
column's sum over R rows has at most R additions of terms that are off by 2^-17."""
import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}
SHAPES = [(1, 1), (1, 1024), (3, 5), (4, 1024), (5, 127), (33, 128), (300, 129), (7, 1001),
          (65, 2048), (2, 16384), (3, 16383), (10, 8200), (700, 48), (1300, 264), (6, 4100)]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def make(rows, width, dtype, seed, weight="own"):
    g = gen(seed)
    x, res, gy, gh = (randn(g, rows, width).to(dtype) for _ in range(4))
    x *= torch.exp(randn(g, rows, 1)).to(dtype)
    w = None if weight is None else (1 + 0.3 * randn(g, width))
    return x, res, gy, gh, w if w is None or weight == "fp32" else w.to(dtype)


def norm64(h, w, eps):
    h = h.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    return y if w is None else y * w.double()


def near(got, ref, size=None, rel=2.0 ** -18):
    half = torch.finfo(got.dtype).eps / 2
    size = ref.abs() if size is None else size
    bound = rel * size + half * (ref.abs() + rel * size) + SMALLEST[got.dtype] / 2
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("rows,width", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weight", ["own", "fp32", None])
def test_norm(rows, width, dtype, weight):
    x, res, _, _, w = make(rows, width, dtype, rows + width, weight)
    near(tbe.tbe_rms_norm(x, w, eps=1e-5), norm64(x, w, 1e-5))
    y, h = tbe.tbe_rms_norm(x, w, residual=res, eps=1e-5)
    assert torch.equal(h, (x.float() + res.float()).to(dtype))
    near(y, norm64(h, w, 1e-5))


def check_8_bits(q, scale, h, w):
    rows, width = h.shape
    assert q.shape == (rows, width) and scale.shape == (rows, -(-width // 128))
    y = norm64(h, w, 1e-6)
    amax = torch.stack([b.abs().amax(1) for b in y.split(128, 1)], 1)
    want = (amax / 448).clamp_min(2.0 ** -126)
    assert bool(((scale.double() - want).abs() <= 2.0 ** -17 * want).all())
    s = scale.double().repeat_interleave(128, 1)[:, :width]
    off = (q.double() * s - y).abs()
    # e4m3: half a step is 2^-4 of the value, and 2^-10 below its normals
    assert bool((off <= (2.0 ** -4 + 2.0 ** -16) * y.abs() + 2.0 ** -10 * s).all())


@pytest.mark.parametrize("rows,width", SHAPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_in_8_bits(rows, width, dtype):
    x, res, _, _, w = make(rows, width, dtype, rows * 3 + width, "fp32")
    x[rows // 2] = 0
    if width > 300:
        x[0, 128:256] = 0  # a block of zeros
    res[rows // 2] = 0
    q, scale, h = tbe.tbe_rms_norm_fp8(x, w, residual=res)
    assert torch.equal(h, (x.float() + res.float()).to(dtype))
    check_8_bits(q, scale, h, w)
    if dtype == torch.float32:  # the quantising is that of tbe_quantize_rows
        q2, scale2 = tbe.tbe_quantize_rows(tbe.tbe_rms_norm(h, w))
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
        assert torch.equal(scale, scale2)
        q3, scale3 = tbe.tbe_rms_norm_fp8(h, w)
        assert torch.equal(q.view(torch.uint8), q3.view(torch.uint8))
        assert torch.equal(scale, scale3)


def gradient64(gy, h, w, gh, eps):
    """(grad_x, the magnitude of its terms, grad_weight, the sum of its |terms|)."""
    gy, h = gy.double(), h.double()
    u = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    d = gy if w is None else gy * w.double()
    unit = h * u
    dx = u * (d - unit * (d * unit).mean(1, keepdim=True))
    size = u * (d.abs() + unit.abs() * (d * unit).abs().mean(1, keepdim=True))
    if gh is not None:
        dx, size = dx + gh.double(), size + gh.double().abs()
    return dx, size, (gy * unit).sum(0), (gy * unit).abs().sum(0)


@pytest.mark.parametrize("rows,width", SHAPES + [(5000, 40), (2500, 1032)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weight", ["own", "fp32", None])
def test_gradients(rows, width, dtype, weight):
    h, _, gy, gh, w = make(rows, width, dtype, rows + 2 * width, weight)
    for given in (None, gh):
        dx, dw = tbe.tbe_rms_norm_backward(gy, h, w, grad_h=given, eps=1e-5)
        rx, size, rw, total = gradient64(gy, h, w, given, 1e-5)
        near(dx, rx, size, 2.0 ** -17)
        assert dw.dtype == torch.float32
        off = (dw.double() - rw).abs()
        assert bool((off <= (2.0 ** -17 + rows * 2.0 ** -24) * total + 2.0 ** -149).all())
        again, dw2 = tbe.tbe_rms_norm_backward(gy, h, w, grad_h=given, eps=1e-5)
        assert torch.equal(dx, again) and torch.equal(dw, dw2)
        alone, none = tbe.tbe_rms_norm_backward(gy, h, w, grad_h=given, eps=1e-5,
                                                need_weight=False)
        assert none is None and torch.equal(alone, dx)


def test_gradients_against_differences():
    # central differences of the 64-bit form: their own error is below 1e-7 here
    rows, width, eps, step = 3, 10, 1e-5, 1e-4
    h, _, gy, _, w = make(rows, width, torch.float32, 4, "fp32")
    dx, dw = tbe.tbe_rms_norm_backward(gy, h, w, eps=eps)
    loss = lambda a, b: float((norm64(a, b, eps) * gy.double()).sum())
    _, size, _, total = gradient64(gy, h, w, None, eps)
    for r in range(rows):
        for c in range(width):
            d = torch.zeros(rows, width, dtype=torch.float64, device="cuda")
            d[r, c] = step
            diff = (loss(h.double() + d, w) - loss(h.double() - d, w)) / (2 * step)
            assert abs(diff - float(dx[r, c])) <= 2.0 ** -16 * float(size[r, c]) + 1e-5
    for c in range(width):
        d = torch.zeros(width, dtype=torch.float64, device="cuda")
        d[c] = step
        diff = (loss(h, w.double() + d) - loss(h, w.double() - d)) / (2 * step)
        assert abs(diff - float(dw[c])) <= 2.0 ** -16 * float(total[c]) + 1e-7


def test_rows_that_are_zero_huge_tiny_or_not_finite():
    x = torch.ones(7, 300, device="cuda")
    x[0], x[1], x[2] = 0.0, 1e18, 1e-25
    x[3, 7], x[4, 9] = float("nan"), float("inf")
    x[5] = 2.0 ** 70  # its square overflows
    y = tbe.tbe_rms_norm(x, eps=1e-6)
    assert bool((y[0] == 0).all())
    near(y[1:3], norm64(x[1:3], None, 1e-6))
    assert bool(y[3].isnan().all())
    assert bool(y[4, 9].isnan()) and float(y[4, 0]) == 0
    assert bool((y[5] == 0).all())
    near(y[6:], norm64(x[6:], None, 1e-6))
    q, scale = tbe.tbe_rms_norm_fp8(x, eps=1e-6)
    assert bool((q[0].float() == 0).all()) and bool((scale[0] == 2.0 ** -126).all())
    assert bool(q[3].float().isnan().all()) and bool(q[4, 9].float().isnan())
    assert bool((tbe.tbe_rms_norm(x[:1], eps=0.0)).isnan().all())


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 3), (5, 1)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_rows(dtype, pad, shift):
    rows, width = 37, 136
    g = gen(pad)
    cut = lambda: randn(g, rows, width + pad).to(dtype)[:, shift:shift + width]
    x, res, gy, gh = cut(), cut(), cut(), cut()
    w = (1 + 0.1 * randn(g, width + 1)).to(dtype)[1:]  # off 16 bytes
    room = torch.full((rows, 4 * (width + pad)), 7.0, dtype=dtype, device="cuda")
    at = [room[:, i * (width + pad) + shift:][:, :width] for i in range(3)]
    y, h = tbe.tbe_rms_norm(x, w, residual=res, out=at[0], h=at[1])
    assert torch.equal(h, (x.float() + res.float()).to(dtype))
    near(y, norm64(h, w, 1e-6))
    dx, dw = tbe.tbe_rms_norm_backward(gy, h, w, grad_h=gh, grad_x=at[2])
    rx, size, rw, total = gradient64(gy, h, w, gh, 1e-6)
    near(dx, rx, size, 2.0 ** -17)
    assert bool(((dw.double() - rw).abs() <= (2.0 ** -17 + rows * 2.0 ** -24) * total).all())
    q8 = torch.zeros(rows, width + pad, dtype=torch.float8_e4m3fn, device="cuda")
    q, scale = tbe.tbe_rms_norm_fp8(x, w, out=q8[:, shift:shift + width])
    # rows off 16 bytes are summed in another order, so the norm may differ in its last bits:
    # held to the formula, as every other row is
    check_8_bits(q, scale, x, w)
    assert bool((q8[:, :shift].float() == 0).all())
    for a in at:
        a.fill_(7.0)
    assert bool((room == 7).all())


@pytest.mark.parametrize("rows,width,pad,shift", [
    (2437, 137, 0, 0), (2500, 1001, 0, 0), (2439, 1001, 6, 3), (20_001, 261, 3, 7),
    (2433, 4099, 5, 2), (41, 2051, 13, 5), (3, 1001, 0, 0), (2440, 136, 16, 1)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("weight", ["own", "fp32", None])
def test_rows_off_16_bytes_among_nan(rows, width, pad, shift, dtype, weight):
    # all matrices alike, what lies between the rows not a number
    _, _, _, _, w = make(1, width, dtype, width, weight)
    nan = lambda: torch.full((rows * (width + pad) + 64,), float("nan"), dtype=dtype, device="cuda")
    g = gen(rows)

    def cut(value=None):
        room = nan()
        rows_of = room[shift:shift + rows * (width + pad)].view(rows, width + pad)[:, :width]
        if value is not None:
            rows_of.copy_(value)
        return room, rows_of

    x, res, gy, gh = (cut(randn(g, rows, width).to(dtype))[1] for _ in range(4))
    rooms = [cut() for _ in range(3)]
    y, h = tbe.tbe_rms_norm(x, w, residual=res, out=rooms[0][1], h=rooms[1][1])
    assert torch.equal(h, (x.float() + res.float()).to(dtype))
    near(y, norm64(h, w, 1e-6))
    near(tbe.tbe_rms_norm(x, w, out=y), norm64(x, w, 1e-6))
    for given in (None, gh):
        dx, dw = tbe.tbe_rms_norm_backward(gy, h, w, grad_h=given, grad_x=rooms[2][1])
        rx, size, rw, total = gradient64(gy, h, w, given, 1e-6)
        near(dx, rx, size, 2.0 ** -17)
        assert bool(((dw.double() - rw).abs() <= (2.0 ** -17 + rows * 2.0 ** -24) * total).all())
        again, dw2 = tbe.tbe_rms_norm_backward(gy, h, w, grad_h=given)  # on other boundaries
        near(again, rx, size, 2.0 ** -17)
        assert bool(((dw2.double() - rw).abs() <= (2.0 ** -17 + rows * 2.0 ** -24) * total).all())
    for room, written in rooms:
        written.zero_()
        assert int(room.isnan().sum()) == room.numel() - rows * width


def test_without_rows():
    none = torch.zeros(0, 24, device="cuda")
    assert tbe.tbe_rms_norm(none).shape == (0, 24)
    q, scale = tbe.tbe_rms_norm_fp8(none)
    assert q.shape == (0, 24) and scale.shape == (0, 1)
    dx, dw = tbe.tbe_rms_norm_backward(none, none)
    assert dx.shape == (0, 24) and bool((dw == 0).all())


def test_many_rows():
    rows, width = 70_001, 72
    x, res, gy, gh, w = make(rows, width, torch.bfloat16, 2)
    y, h = tbe.tbe_rms_norm(x, w, residual=res)
    near(y, norm64(h, w, 1e-6))
    dx, dw = tbe.tbe_rms_norm_backward(gy, h, w, grad_h=gh)
    rx, size, rw, total = gradient64(gy, h, w, gh, 1e-6)
    near(dx, rx, size, 2.0 ** -17)
    assert bool(((dw.double() - rw).abs() <= (2.0 ** -17 + rows * 2.0 ** -24) * total).all())


def test_in_a_graph_on_a_stream_with_a_workspace():
    rows, width = 900, 520
    x, res, gy, gh, w = make(rows, width, torch.bfloat16, 6)
    ws = torch.empty(tbe.tbe_rms_norm_workspace_size(rows, width), dtype=torch.uint8,
                     device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dx, dw = tbe.tbe_rms_norm_backward(gy, x, w, grad_h=gh, ws=ws, stream=side)
    y, h = tbe.tbe_rms_norm(x, w, residual=res, stream=side)
    q, scale, h8 = tbe.tbe_rms_norm_fp8(x, w, residual=res, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = [t.clone() for t in (y, h, q.view(torch.uint8), scale, h8, dx, dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tbe.tbe_rms_norm(x, w, residual=res, out=y, h=h)
        tbe.tbe_rms_norm_fp8(x, w, residual=res, out=q, scale=scale, h=h8)
        tbe.tbe_rms_norm_backward(gy, x, w, grad_h=gh, grad_x=dx, grad_weight=dw, ws=ws)
    keep = x.clone()
    x.zero_()
    graph.replay()
    x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((y, h, q.view(torch.uint8), scale, h8, dx, dw), want):
        assert torch.equal(a, b)
