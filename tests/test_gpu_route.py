"""Routing to experts and its gradient on the GPU, against plain 64-bit forms written
here.

Tolerances, in units u = 2^-24: an exponential of a difference x is off by 2 |x| + 4,
a row's sum by ten additions and the terms' own errors, a quotient by 1: with |x| below
30 a weight is off by less than 2^-17 of itself, and a gradient by less than 2^-16 of
the magnitude of its terms, plus half a unit in the last place of its type."""
import math

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


def scores64(logits, score):
    l = logits.double()
    if score == "sigmoid":
        return torch.sigmoid(l)
    return torch.softmax(l, 1).nan_to_num(0.0)  # rows that are closed throughout


def route64(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_best=1,
            renormalize=True, scale=1.0):
    """The best expert that is left, k times; ties go to the first (as max does)."""
    n, experts = logits.shape
    s = scores64(logits, score)
    c = s.clone() if bias is None else s + bias.double()
    if bias is None and (groups == 1 or group_best == 1):
        c = logits.double().clone()
    c[logits == -math.inf] = -math.inf
    at_row = torch.arange(n, device="cuda")
    if groups > 1:
        best = c.view(n, groups, -1).topk(min(group_best, experts // groups), 2).values
        worth = best[:, :, 0].clone()
        if best.shape[2] > 1:
            worth += torch.where(best[:, :, 1] == -math.inf, 0.0, best[:, :, 1])
        taken = torch.zeros(n, groups, dtype=torch.bool, device="cuda")
        for _ in range(top_groups):
            v, g = worth.max(1)
            taken[at_row, g] |= v > -math.inf
            worth[at_row, g] = -math.inf
        c[~taken.repeat_interleave(experts // groups, 1)] = -math.inf
    ids, w = [], []
    for _ in range(k):
        v, e = c.max(1)
        on = v > -math.inf
        ids.append(torch.where(on, e, -1))
        w.append(torch.where(on, s[at_row, e], 0.0))
        c[at_row, e] = -math.inf
    ids, w = torch.stack(ids, 1), torch.stack(w, 1)
    if renormalize:
        # through logarithms: 64 bits too lose scores below 2^-1074, whose ratios are still defined
        l = logits.double().gather(1, ids.clamp_min(0))
        logs = torch.nn.functional.logsigmoid(l) if score == "sigmoid" else l
        logs = torch.where(ids >= 0, logs, -math.inf)
        w = torch.softmax(logs, 1)
        w = torch.where((ids >= 0).any(1, keepdim=True), w, 0.0)
    return ids, w * scale


def check(logits, k, **how):
    ids, weights = tbe.tbe_expert_route(logits, k, **how)
    want_ids, want = route64(logits, k, **how)
    assert ids.dtype == torch.int32 and torch.equal(ids.long(), want_ids)
    off = (weights.double() - want).abs()
    assert bool((off <= 2.0 ** -17 * want.abs() + 2.0 ** -126).all()), float(off.max())
    return ids, weights


HOW = [
    dict(),
    dict(renormalize=False),
    dict(score="sigmoid"),
    dict(score="sigmoid", renormalize=False, scale=2.5),
    dict(bias=True),
    dict(bias=True, renormalize=False),
    dict(bias=True, score="sigmoid", scale=0.5),
]


def with_bias(how, experts, g):
    return dict(how, bias=0.1 * randn(g, experts)) if how.get("bias") else how


@pytest.mark.parametrize("tokens,experts,k", [
    (1, 1, 1), (3, 2, 2), (4, 16, 2), (33, 17, 5), (100, 32, 31), (257, 64, 4), (65, 100, 6),
    (500, 128, 8), (77, 256, 8), (40, 511, 3), (20, 1000, 31), (9, 1024, 8), (5000, 60, 1)])
@pytest.mark.parametrize("how", HOW)
def test_choice_and_weights(tokens, experts, k, how):
    for dtype in DTYPES:
        g = gen(tokens + experts)
        logits = (1.5 * randn(g, tokens, experts)).to(dtype)
        check(logits, k, **with_bias(how, experts, g))


@pytest.mark.parametrize("experts,groups,top_groups,k", [
    (8, 4, 2, 3), (64, 8, 4, 8), (256, 8, 4, 8), (96, 32, 3, 9), (60, 5, 2, 24), (1024, 16, 1, 7),
    (30, 30, 4, 4), (64, 2, 2, 6)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("how", HOW)
def test_groups(experts, groups, top_groups, k, best, how):
    for dtype in DTYPES:
        g = gen(experts + k)
        logits = (1.5 * randn(g, 300, experts)).to(dtype)
        logits[randn(g, 300, experts) > 1.2] = -math.inf
        check(logits, k, groups=groups, top_groups=top_groups, group_best=best,
              **with_bias(how, experts, g))


@pytest.mark.parametrize("how", HOW)
def test_closed_experts(how):
    g = gen(1)
    logits = randn(g, 200, 24)
    logits[randn(g, 200, 24) > 0] = -math.inf
    logits[7] = -math.inf                 # nothing is left
    logits[8] = -math.inf
    logits[8, 20] = -3.0                  # one is
    logits[9] = torch.finfo(torch.float32).min
    logits[10, 5] = torch.finfo(torch.float32).min
    how = with_bias(how, 24, g)
    ids, weights = check(logits, 6, **how)
    assert ids[7].tolist() == [-1] * 6 and bool((weights[7] == 0).all())
    assert ids[8].tolist() == [20] + [-1] * 5
    if how.get("bias") is not None:
        how["bias"][3] = -math.inf        # closed to all
        ids, _ = check(logits, 6, **how)
        assert not bool((ids == 3).any())


def test_ties_go_to_the_lower_expert_and_group():
    logits = torch.zeros(5, 48, device="cuda")
    logits[1, 30] = 1.0
    logits[2] = -0.0
    logits[2, 40:] = 0.0
    logits[3, :10] = -1.0
    for how in (dict(), dict(bias=torch.zeros(48, device="cuda")),
                dict(score="sigmoid", bias=torch.full((48,), 0.25, device="cuda")),
                dict(groups=6, top_groups=2, group_best=2),
                dict(groups=6, top_groups=2, bias=torch.zeros(48, device="cuda"))):
        ids, _ = check(logits, 4, **how)
        assert ids[0].tolist() == [0, 1, 2, 3] and ids[2].tolist() == [0, 1, 2, 3]
        assert ids[1, 0] == 30


def test_choices_that_fp32_does_not_tell_apart():
    # score + bias agree to a few units of fp32 and differ in 64 bits
    g = gen(2)
    logits = randn(g, 2000, 40)
    s = torch.sigmoid(logits.double())
    bias = (0.9 - torch.sigmoid(torch.zeros(40, dtype=torch.float64, device="cuda"))).float()
    logits = (1e-6 * logits).float()      # scores within 1e-6 of a half
    check(logits, 8, score="sigmoid", bias=bias)
    check(logits, 8, bias=bias)
    check(logits, 8, score="sigmoid", bias=bias, groups=8, top_groups=3, group_best=2)
    big = torch.full((40,), 4096.0, device="cuda")  # swallows the score's last bits in fp32
    check(randn(g, 500, 40), 8, score="sigmoid", bias=big)
    # choices of both signs, large beside the groups' worth
    mixed = torch.where(torch.arange(40, device="cuda") % 2 == 0, 300.0, -299.5)
    check(randn(g, 2000, 40), 6, score="sigmoid", bias=mixed + 1e-5 * randn(g, 40), groups=10,
          top_groups=3, group_best=2)
    assert s.shape == (2000, 40)


@pytest.mark.parametrize("experts,k", [(16, 3), (24, 7), (100, 8), (256, 8), (600, 15), (1000, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_rows_that_need_exact_arithmetic(experts, k, score):
    # logits that differ in their last bits, so that most rows' choices do
    g = gen(experts)
    logits = 1.0 + 2.0 ** -22 * torch.randint(0, 400, (300, experts), generator=g,
                                              device="cuda").float()
    bias = torch.full((experts,), 0.125, device="cuda")
    bias[::3] += 2.0 ** -27
    for how in (dict(), dict(renormalize=False)):
        check(logits, k, score=score, bias=bias, **how)
    groups = 4
    check(logits, min(k, experts // 2), score=score, bias=bias, groups=groups, top_groups=2,
          group_best=2)
    check(logits, min(k, experts // 2), score=score, groups=groups, top_groups=2, group_best=2)


@pytest.mark.parametrize("experts,k", [
    (32, 4), (40, 3), (64, 4), (64, 8), (96, 9), (128, 8), (128, 9), (100, 12), (128, 16), (256, 8)])
@pytest.mark.parametrize("how", [HOW[0], HOW[5], HOW[6]])
def test_rows_with_many_and_few_candidates_side_by_side(experts, k, how):
    # few values, so that many choices are alike; the largest side by side; most or all closed
    g = gen(experts * k)
    logits = torch.randint(-2, 3, (400, experts), generator=g, device="cuda") / 2
    logits[1::7] += randn(g, experts) * 0.01
    logits[2::7] = randn(g, logits[2::7].shape[0], experts)
    logits[3::7, 5:5 + k + 2] += 4.0
    closed = torch.rand(logits[4::7].shape, generator=g, device="cuda") < 0.97
    logits[4::7] = torch.where(closed, -math.inf, logits[4::7])
    logits[5::14] = -math.inf
    logits[6::7] = 0.25
    check(logits, k, **with_bias(how, experts, g))
    if how.get("bias"):
        check(logits, k, **dict(how, bias=torch.zeros(experts, device="cuda")))


def test_extreme_logits():
    logits = torch.full((6, 20), -100.0, device="cuda")
    logits[0, 3] = 100.0
    logits[1] = -300.0 - torch.arange(20, device="cuda")
    logits[2] = torch.arange(20, device="cuda") * 3000.0
    for renorm in (True, False):
        for score in ("softmax", "sigmoid"):
            ids, w = tbe.tbe_expert_route(logits, 3, score=score, renormalize=renorm)
            want_ids, want = route64(logits, 3, score=score, renormalize=renorm)
            assert torch.equal(ids.long(), want_ids)
            # fp32 loses what is below 2^-126
            assert bool(((w.double() - want).abs() <= 2.0 ** -16 * want + 2.0 ** -126).all())


@pytest.mark.parametrize("how", HOW)
def test_nan_and_infinity_show(how):
    g = gen(3)
    logits = randn(g, 8, 40)
    logits[1, 30] = float("nan")
    logits[2, 30] = float("inf")
    logits[3, 4], logits[3, 39] = float("inf"), float("inf")
    how = with_bias(how, 40, g)
    ids, w = tbe.tbe_expert_route(logits, 5, **how)
    for row in ids.tolist():
        assert len(set(row)) == 5 and all(0 <= e < 40 for e in row)
    assert bool(w[1].isnan().any())
    if how.get("score") != "sigmoid":
        assert bool(w[2].isnan().any()) and bool(w[3].isnan().any())
    else:
        assert 30 in ids[2].tolist() or how.get("bias") is not None
    keep = torch.tensor([0, 4, 5, 6, 7], device="cuda")
    want_ids, want = route64(logits[keep], 5, **how)
    assert torch.equal(ids[keep].long(), want_ids)
    if how.get("bias") is not None:
        how["bias"][7] = float("nan")
        ids, _ = tbe.tbe_expert_route(logits[4:], 5, **how)
        assert bool((ids[:, 0] == 7).all())


def test_int64_ids_strides_and_a_given_stream():
    g = gen(4)
    wide = randn(g, 100, 73)
    logits = wide[:, 5:69]
    ids = torch.empty(100, 6, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tbe.tbe_expert_route(logits, 6, ids=ids, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(ids, route64(logits, 6)[0])
    assert tbe.tbe_expert_route(logits[:0], 3)[0].shape == (0, 3)


def gradient64(grad_weights, logits, ids, score, renormalize, scale):
    """The gradient by automatic differentiation, and a bound on its terms' magnitude."""
    l = logits.double().clone().requires_grad_()
    experts = l.shape[1]
    on = (ids >= 0) & (ids < experts)
    at = ids.clamp(0, experts - 1).long()
    chosen = torch.where(on, l.gather(1, at), 0.0)
    if score == "sigmoid":
        s = torch.sigmoid(chosen)
    elif renormalize:
        top = torch.where(on, chosen, -1e30).max(1, keepdim=True).values.detach()
        s = torch.exp(torch.where(on, chosen - top, 0.0))
    else:
        s = torch.softmax(l, 1).gather(1, at)
    s = torch.where(on, s, 0.0)
    w = s / s.sum(1, keepdim=True).clamp_min(1e-300) if renormalize else s
    g = torch.where(on, grad_weights.double() * scale, 0.0)
    grad = torch.autograd.grad((w * g).sum(), l)[0].nan_to_num(0.0)
    w, total = w.detach(), (w.detach() * g.abs()).sum(1, keepdim=True)
    size = torch.zeros_like(grad).scatter_add_(1, at, torch.where(on, w * (g.abs() + total), 0.0))
    if score == "softmax" and not renormalize:
        size += torch.softmax(logits.double(), 1).nan_to_num(0.0) * total
    return grad, size


def check_gradient(gw, logits, ids, how):
    got = tbe.tbe_expert_route_backward(gw, logits, ids, **how)
    assert got.dtype == logits.dtype and got.shape == logits.shape
    ref, size = gradient64(gw, logits, ids, how.get("score", "softmax"),
                           how.get("renormalize", True), how.get("scale", 1.0))
    half = torch.finfo(got.dtype).eps / 2
    bound = 2.0 ** -16 * size + half * (ref.abs() + 2.0 ** -16 * size) + SMALLEST[got.dtype]
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    assert torch.equal(got, tbe.tbe_expert_route_backward(gw, logits, ids, **how))
    return got


GRAD_HOW = [dict(h) for h in HOW[:4]]


@pytest.mark.parametrize("tokens,experts,k", [
    (1, 1, 1), (3, 2, 2), (4, 16, 2), (33, 17, 5), (100, 32, 31), (257, 64, 4), (65, 100, 6),
    (77, 256, 8), (40, 511, 3), (20, 1000, 31), (9, 1024, 8)])
@pytest.mark.parametrize("how", GRAD_HOW)
def test_gradient(tokens, experts, k, how):
    for dtype in DTYPES:
        g = gen(tokens + experts)
        logits = (1.5 * randn(g, tokens, experts)).to(dtype)
        ids, _ = tbe.tbe_expert_route(logits, k, **how)
        check_gradient(randn(g, tokens, k), logits, ids, how)


@pytest.mark.parametrize("how", GRAD_HOW)
def test_gradient_of_closed_dropped_and_repeated_experts(how):
    g = gen(5)
    logits = randn(g, 300, 24)
    logits[randn(g, 300, 24) > 0.3] = -math.inf
    logits[7] = -math.inf
    ids, _ = tbe.tbe_expert_route(logits, 9, **how)
    gw = randn(g, 300, 9)
    gw[ids < 0] = float("nan")           # not used
    got = check_gradient(gw, logits, ids, how)
    assert bool((got[7] == 0).all()) and bool((got[logits == -math.inf] == 0).all())
    logits = randn(g, 300, 24)
    ids = torch.randint(-2, 27, (300, 9), generator=g, device="cuda")  # twice, and out of range
    gw = randn(g, 300, 9)
    gw[(ids < 0) | (ids >= 24)] = float("inf")
    check_gradient(gw, logits, ids, how)
    far = ids.clone()
    far[:, 0] = (1 << 32) + 3             # an expert in its low 32 bits only
    check_gradient(gw.nan_to_num(0.0, 0.0), logits, far, how)


@pytest.mark.parametrize("how", GRAD_HOW)
def test_gradient_against_differences(how):
    # central differences of the 64-bit weights at a fixed choice: their own error is below 1e-8
    g = gen(6)
    logits, step = randn(g, 4, 7), 1e-5
    ids, _ = tbe.tbe_expert_route(logits, 3, **how)
    gw = randn(g, 4, 3)
    got = tbe.tbe_expert_route_backward(gw, logits, ids, **how)

    def loss(l):
        s = scores64(l, how.get("score", "softmax")).gather(1, ids.long())
        if how.get("renormalize", True):
            s = s / s.sum(1, keepdim=True)
        return float((s * gw.double()).sum()) * how.get("scale", 1.0)

    _, size = gradient64(gw, logits, ids, how.get("score", "softmax"),
                         how.get("renormalize", True), how.get("scale", 1.0))
    for r in range(4):
        for c in range(7):
            d = torch.zeros(4, 7, dtype=torch.float64, device="cuda")
            d[r, c] = step
            diff = (loss(logits.double() + d) - loss(logits.double() - d)) / (2 * step)
            assert abs(diff - float(got[r, c])) <= 2.0 ** -16 * float(size[r, c]) + 1e-7


def test_gradient_into_strided_rows_and_in_a_graph():
    g = gen(7)
    logits = randn(g, 500, 64).bfloat16()
    bias = 0.1 * randn(g, 64)
    how = dict(score="sigmoid", scale=2.5)
    more = dict(groups=8, top_groups=3, group_best=2)
    room = torch.full((500, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    ids, weights = tbe.tbe_expert_route(logits, 6, bias=bias, **how, **more)
    gw = randn(g, 500, 6)
    tbe.tbe_expert_route_backward(gw, logits, ids, out=room[:, 3:67], **how)
    assert torch.equal(room[:, 3:67], tbe.tbe_expert_route_backward(gw, logits, ids, **how))
    assert bool((room[:, :3] == 7).all()) and bool((room[:, 67:] == 7).all())
    grad = torch.empty_like(logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tbe.tbe_expert_route(logits, 6, bias=bias, ids=ids, weights=weights, **how, **more)
        tbe.tbe_expert_route_backward(gw, logits, ids, out=grad, **how)
    for seed in (8, 9):
        logits.copy_(randn(gen(seed), 500, 64))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids.long(), route64(logits, 6, bias=bias, **how, **more)[0])
        ref, size = gradient64(gw, logits, ids, "sigmoid", True, 2.5)
        assert bool(((grad.double() - ref).abs() <= 2.0 ** -7 * size + 1e-30).all())
