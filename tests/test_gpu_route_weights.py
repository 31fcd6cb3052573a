"""Routing weights to fp32's last bits, on the GPU, against 64 bits.

In units u = 2^-24.  The logits are whole numbers, so their differences are exact.  expf is off by
two units in the last place at most, 4 u; a sum of E positive terms, added along a tree of
log2 E levels, by a unit a level and its terms' 4 u; 1 + e by one unit and e's 4 u; a division
and the scale by a unit each."""
import math

import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SMALLEST = 2.0 ** -149
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def whole(tokens, experts, low, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return -torch.randint(0, -low, (tokens, experts), generator=g, device="cuda").float()


@pytest.mark.parametrize("experts,k", [(2, 2), (16, 8), (64, 4), (128, 8), (256, 31), (1000, 5)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("biased", [False, True])
def test_softmax_weights(experts, k, dtype, biased):
    logits = whole(300, experts, -85, experts + k)
    logits[:, 0] = 0.0
    logits = logits.to(dtype)  # whole numbers up to 85: exact in every type
    bias = None
    if biased:  # the unlikely are chosen
        bias = torch.arange(experts, device="cuda").float()
    levels = math.ceil(math.log2(experts))
    for renormalize, off in ((True, 4 + 4 + 5 + 1), (False, 4 + 4 + levels + 1)):
        ids, w = tbe.tbe_expert_route(logits, k, bias=bias, renormalize=renormalize, scale=1.0)
        l = logits.double()
        chosen = l.gather(1, ids.long())
        ref = torch.softmax(chosen if renormalize else l, 1)
        if not renormalize:
            ref = ref.gather(1, ids.long())
        assert float(ref[:, -1].min()) < 2.0 ** -60 or not biased or experts < 16
        assert bool(((w.double() - ref).abs() <= off * U * ref + 2 * SMALLEST).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_sigmoid_weights(dtype):
    values = torch.arange(-104, 105, device="cuda").to(dtype)
    ids, w = tbe.tbe_expert_route(values[:, None], 1, score="sigmoid", renormalize=False)
    assert not bool(ids.any())
    l = values.double()
    ref = torch.where(l < 0, torch.exp(l) / (1 + torch.exp(l)), 1 / (1 + torch.exp(-l)))
    assert float(ref[1]) > SMALLEST  # e^-103; the first, e^-104, is less than half of it
    # the exponential twice, the sum, the quotient; two steps at fp32's end
    assert bool(((w[:, 0].double() - ref).abs() <= (4 + 4 + 1 + 1) * U * ref + 2 * SMALLEST).all())
    logits = whole(300, 24, -58, 3).to(dtype)
    ids, w = tbe.tbe_expert_route(logits, 6, score="sigmoid", scale=1.0)
    s = torch.sigmoid(logits.double().gather(1, ids.long()))
    ref = s / s.sum(1, keepdim=True)
    assert bool(((w.double() - ref).abs() <= (2 * 10 + 5 + 1) * U * ref).all())
    far = -60.0 - whole(300, 24, -40, 4).abs()
    far = far.to(dtype)
    ids, w = tbe.tbe_expert_route(far, 6, score="sigmoid", scale=1.0)
    s = torch.softmax(torch.nn.functional.logsigmoid(far.double().gather(1, ids.long())), 1)
    assert bool(((w.double() - s).abs() <= (2 * 10 + 5 + 1) * U * s).all())


@pytest.mark.parametrize("top", [-18, -19, -30, -59, -60, -61, -90])
def test_sigmoid_weights_whose_scores_underflow(top):
    # the ratio of two scores of which fp32 holds the smaller one badly or not at all
    logits = torch.full((90, 8), float(top), device="cuda")
    logits[:, 3] = top - torch.arange(90, device="cuda").float()
    if top == -18:  # the scores themselves are taken: to e^-87
        logits = logits[:60]
    how = dict(score="sigmoid", scale=1.0)
    ids, w = tbe.tbe_expert_route(logits, 8, **how)
    l = logits.double().gather(1, ids.long())
    s = torch.softmax(torch.nn.functional.logsigmoid(l), 1)
    # the scores' own off by a quarter of a unit more than exponentials, a normal result
    bound = (2 * 10 + 5 + 1) * U * s + 2.0 ** -126
    assert bool(((w.double() - s).abs() <= bound).all())
    # its gradient by differences of logarithms: d w_j / d l_i = w_j (1 - s_i) (i == j) - w_j w_i (1 - s_i)
    gw = torch.ones_like(w)
    gw[:, -1] = 3.0
    got = tbe.tbe_expert_route_backward(gw, logits, ids, **how).gather(1, ids.long())
    one = 1 / (1 + torch.exp(l))
    ref = s * one * (gw.double() - (gw.double() * s).sum(1, keepdim=True))
    size = s * (gw.double() + (gw.double() * s).sum(1, keepdim=True))
    assert bool(((got.double() - ref).abs() <= 2.0 ** -18 * size + 2.0 ** -126).all())
