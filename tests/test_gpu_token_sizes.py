"""Token embedding, norm and routing at the largest sizes they take and past 32 bits of
elements, on the GPU.

Values are small integers, or random in a few rows at both ends with zeros between them, so
that results are exact or held to the tolerances of the small tests' plain forms."""
import pytest
import torch

import table_embedding_bag_gb300 as tbe
from .test_gpu_norm import check_8_bits, gradient64, near, norm64
from .test_gpu_route import gradient64 as route_gradient64
from .test_gpu_route import route64

pytestmark = pytest.mark.gpu

MOST = (1 << 31) - 1


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def at_the_ends(g, rows, width, dtype, n=3):
    """(zeros but for the first and the last n rows, the places of those)."""
    x = torch.zeros(rows, width, dtype=dtype, device="cuda")
    at = torch.cat([torch.arange(n), torch.arange(rows - n, rows)]).cuda()
    x[at] = torch.randn(2 * n, width, generator=g, device="cuda").to(dtype)
    return x, at


@pytest.mark.parametrize("width", [1 << 20, (1 << 20) - 1])
def test_the_widest_rows(width):
    g = gen(1)
    table = torch.randint(-8, 9, (5, width), generator=g, device="cuda").bfloat16()
    ids = torch.tensor([4, -1, 0, 4, 2], device="cuda")
    got = tbe.tbe_embed(table, ids)
    assert torch.equal(got[[0, 2, 3, 4]], table[[4, 0, 4, 2]]) and not bool(got[1].any())
    for n in (5, 1030):  # without a sort and with one
        ids = torch.randint(-1, 5, (n,), generator=g, device="cuda")
        ids[ids == 3] = 1
        grad = torch.randint(-1, 2, (n, width), generator=g, device="cuda",
                             dtype=torch.int8).bfloat16()
        for out in (torch.bfloat16, torch.float32):
            got = tbe.tbe_embed_backward(grad, ids, 5, out_dtype=out)
            for row in range(5):
                want = grad[ids == row].sum(0, dtype=torch.float32)  # whole numbers: exact
                assert torch.equal(got[row], want.to(out))


def test_lookup_and_gradient_past_32_bits_of_tokens_rows():
    n, rows, width = 540_001, 60_000, 4096  # 2.2 billion elements
    g = gen(2)
    table = torch.randint(-8, 9, (rows, width), generator=g, device="cuda",
                          dtype=torch.int8).half()
    ids = torch.randint(0, rows, (n,), generator=g, device="cuda")
    got = tbe.tbe_embed(table, ids)
    for i in range(0, n, 60_000):
        assert torch.equal(got[i:i + 60_000], table[ids[i:i + 60_000]])
    value = (torch.arange(n, device="cuda") % 7).half()
    got.copy_(value[:, None].expand(-1, width))
    grad = tbe.tbe_embed_backward(got, ids, rows)  # sums below 2048: exact
    want = torch.zeros(rows, device="cuda").index_add_(0, ids, value.float())
    assert float(want.max()) < 2048 and torch.equal(grad, want.half()[:, None].expand(-1, width))


@pytest.mark.parametrize("n", [900, 5000])
def test_the_most_rows(n):
    rows = MOST - 1025
    g = gen(3)
    ids = torch.randint(0, rows, (n,), generator=g, device="cuda")
    ids[:4] = torch.tensor([rows - 1, 0, rows - 1, rows - 2], device="cuda")
    ids[4:6] = torch.tensor([rows, MOST], device="cuda")
    grad = torch.ones(n, 1, dtype=torch.float16, device="cuda")
    grad[4:6] = 5
    got = tbe.tbe_embed_backward(grad, ids, rows)
    kept, count = ids[(ids < rows)].unique(return_counts=True)
    assert torch.equal(got[kept, 0].float(), count.float())
    assert int(torch.count_nonzero(got)) == kept.numel()
    out = tbe.tbe_embed(got, ids.int())
    assert torch.equal(out[ids < rows], got[ids[ids < rows]]) and not bool(out[4:6].any())


@pytest.mark.parametrize("width", [16384, 16383])
def test_norms_past_32_bits(width):
    rows = 131_085  # 2.15 billion elements
    g = gen(4)
    x, at = at_the_ends(g, rows, width, torch.bfloat16)
    res, _ = at_the_ends(g, rows, width, torch.bfloat16)
    y, h = tbe.tbe_rms_norm(x, residual=res)
    assert torch.equal(h[at], (x[at].float() + res[at].float()).bfloat16())
    near(y[at], norm64(h[at], None, 1e-6))
    assert not bool(y[3:-3].any())
    del y
    q, scale = tbe.tbe_rms_norm_fp8(h)
    check_8_bits(q.view(torch.uint8)[at].view(q.dtype), scale[at], h[at], torch.ones(width, device="cuda"))
    assert bool((scale[3:-3] == 2.0 ** -126).all())
    del q
    dx, dw = tbe.tbe_rms_norm_backward(res, h)
    rx, size, rw, total = gradient64(res[at], h[at], None, None, 1e-6)
    near(dx[at], rx, size, 2.0 ** -17)
    assert not bool(dx[3:-3].any())
    assert bool(((dw.double() - rw).abs() <= (2.0 ** -17 + 6 * 2.0 ** -24) * total).all())


def test_the_most_rows_of_a_norm():
    x, at = at_the_ends(gen(5), MOST, 1, torch.float16)
    y = tbe.tbe_rms_norm(x)
    near(y[at], norm64(x[at], None, 1e-6))
    assert int(torch.count_nonzero(y)) == int(torch.count_nonzero(y[at]))
    dx, dw = tbe.tbe_rms_norm_backward(y, x, grad_x=torch.empty_like(x))
    rx, size, rw, total = gradient64(y[at], x[at], None, None, 1e-6)
    near(dx[at], rx, size, 2.0 ** -17)
    assert bool(((dw.double() - rw).abs() <= (2.0 ** -17 + 6 * 2.0 ** -24) * total).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_routing_past_32_bits(score):
    tokens, experts, k = 2_100_003, 1024, 4  # 2.15 billion logits
    logits, at = at_the_ends(gen(6), tokens, experts, torch.bfloat16)
    ids, weights = tbe.tbe_expert_route(logits, k, score=score)
    want_ids, want = route64(logits[at], k, score=score)
    assert torch.equal(ids[at].long(), want_ids)
    assert bool(((weights[at].double() - want).abs() <= 2.0 ** -17 * want).all())
    assert bool((ids[3:-3] == torch.arange(k, device="cuda")).all())  # ties
    assert bool(((weights[3:-3] - 0.25).abs() <= 2.0 ** -19).all())
    gw = torch.zeros(tokens, k, device="cuda")
    gw[at] = torch.randn(6, k, generator=gen(7), device="cuda")
    got = tbe.tbe_expert_route_backward(gw, logits, ids, score=score)
    ref, size = route_gradient64(gw[at], logits[at], ids[at], score, True, 1.0)
    bound = 2.0 ** -16 * size + 2.0 ** -8 * (ref.abs() + 2.0 ** -16 * size) + 2.0 ** -133
    assert bool(((got[at].double() - ref).abs() <= bound).all())
    assert not bool(got[3:-3].any())


def test_routing_the_most_tokens():
    logits = torch.zeros(MOST, 1, dtype=torch.float16, device="cuda")
    ids, weights = tbe.tbe_expert_route(logits, 1, renormalize=False)
    assert not bool(ids.any()) and bool(((weights - 1).abs() <= 2.0 ** -17).all())
    del ids, weights
    logits[MOST - 1] = -float("inf")
    ids, weights = tbe.tbe_expert_route(logits, 1)
    assert ids[-2:, 0].tolist() == [0, -1] and float(weights[-1]) == 0
    assert abs(float(weights[-2]) - 1) <= 2.0 ** -17
    assert int(torch.count_nonzero(ids)) == 1
