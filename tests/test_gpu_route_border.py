"""Routing where fp32 does not tell the last expert that is chosen from one behind it, on the
GPU, against the plain 64-bit form of test_gpu_route.py.

Rows have one close pair, at the border, so that nothing else in them asks for exact
arithmetic."""
import math

import pytest
import torch

from .test_gpu_route import check, gen, route64

pytestmark = pytest.mark.gpu

# experts and chosen ones of rows of 8, 16 and 32 lanes, in rounds and by candidates
SIZES = [(16, 1), (16, 5), (24, 3), (33, 2), (64, 3), (64, 7), (100, 1), (128, 6), (128, 8), (96, 12),
         (256, 1), (256, 2), (256, 8), (600, 4), (1000, 8)]


@pytest.mark.parametrize("experts,k", SIZES)
@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_a_likely_expert_of_low_bias_behind_unlikely_ones(experts, k, place):
    # Softmax.  One expert has much of the score, with the error of the row's sum, and with its bias
    # it comes to what the k-th choice and the next one come to, whose scores, and so whose
    # errors, are next to nothing.
    rows, g = 4000, gen(experts + k)
    likely = {"first": 0, "middle": experts // 2, "last": experts - 1}[place]
    others = [e for e in range(experts) if e != likely]
    chosen, close = others[:k - 1], others[k - 1:k + 1]
    rest = torch.tensor(others[k + 1:], device="cuda")
    # The rest have 0.8 of the likely one's score, shared at random, so that each row's sum is
    # rounded in its own way; and a little more or less, which moves the likely one's by a few of
    # its errors.
    l = 3 * torch.rand(rows, experts, generator=g, device="cuda", dtype=torch.float64)
    l[:, rest] += math.log(0.8) - torch.logsumexp(l[:, rest], 1, keepdim=True)
    l[:, rest] += 2e-6 * torch.rand(rows, 1, generator=g, device="cuda", dtype=torch.float64) - 1e-6
    l[:, chosen], l[:, close], l[:, likely] = -20.0, -25.0, 0.0
    logits = l.float()
    bias = torch.full((experts,), -2.0, dtype=torch.float64, device="cuda")
    bias[chosen] = 2.0 - 0.1 * torch.arange(k - 1, dtype=torch.float64, device="cuda")
    bias[close] = torch.tensor([2.0 ** -6, 2.0 ** -6 - 3 * 2.0 ** -30], dtype=torch.float64, device="cuda")
    bias[likely] = 2.0 ** -6 - 1 / 1.8
    bias = bias.float()
    want, _ = route64(logits, k, bias=bias)
    assert bool((want[:, -1] == likely).any()) and bool((want[:, -1] == close[0]).any())
    assert bias[close[0]] > bias[close[1]]
    check(logits, k, bias=bias)
    check(logits, k, bias=bias, renormalize=False)


@pytest.mark.parametrize("experts,k", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kinds", [1, 2, 3])
def test_experts_alike_at_the_border(experts, k, score, kinds):
    # The k-th choice and the next one have the same logit and bias, and behind them stand
    # choices that fp32 holds to be the same, or next to it, and that are larger.  Biases below a
    # half whose sums with the score are above it, where fp32's steps are twice as wide.
    rows, g = 3000, gen(experts * k + kinds)
    low = 0.5 - 2.0 ** -23
    kind = torch.randint(0, kinds, (experts,), generator=g, device="cuda")
    bias = torch.tensor([low, low + 2.0 ** -25, low - 2.0 ** -24], device="cuda")[kind]
    alike = torch.tensor([0.0, 0.0, 1.25 * 2.0 ** -22], device="cuda")[kind]
    assert kinds == 1 or bias.unique().numel() > 1
    # by chance some are chosen for certain, some are alike and the others far behind
    chance = torch.rand(rows, experts, generator=g, device="cuda")
    sure = max(k - 2, 0) / experts
    logits = torch.where(chance < sure + 4 / experts, alike, -4.0)
    certain = 4 + 0.125 * torch.arange(experts, device="cuda") % 8
    logits = torch.where(chance < sure, certain, logits)
    check(logits, k, score=score, bias=bias)
    if kinds < 3:
        check(logits.bfloat16(), k, score=score, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [3, 64, 128, 256])
def test_an_expert_behind_two_alike(score, experts):
    # the smallest case: of the first three the last is ahead, by less than fp32 holds
    logits = torch.full((5, experts), -30.0, device="cuda")
    logits[:, :3] = 0.0
    bias = torch.zeros(experts, device="cuda")
    bias[:3] = 0.5 - 2.0 ** -23
    bias[2] += 2.0 ** -25
    assert check(logits, 1, score=score, bias=bias)[0].tolist() == [[2]] * 5
    assert check(logits, 2, score=score, bias=bias)[0].tolist() == [[2, 0]] * 5


@pytest.mark.parametrize("experts,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_coarse_logits_with_stepped_biases(experts, k, dtype):
    # as a rule of balance leaves them: biases that rose and fell by one step a time
    g = gen(experts - k)
    logits = (0.5 * torch.randn(2000, experts, generator=g, device="cuda")).to(dtype)
    steps = torch.randint(-3, 4, (experts,), generator=g, device="cuda")
    for score in ("softmax", "sigmoid"):
        check(logits, k, score=score, bias=1e-3 * steps.float())
        check(logits, k, score=score, bias=2.0 ** -24 * steps.float())


@pytest.mark.parametrize("experts", [12, 64, 128, 256])
def test_scores_at_the_end_of_fp32(experts):
    # softmax scores around 2^-126, one of which an approximate exponential may hold to be zero,
    # with biases that are as small
    end = 126 * math.log(2.0)
    for places in (1, 2, 3):
        logits = torch.full((15, experts), -math.inf, device="cuda")
        logits[:, 0] = 0.0
        first = -end + 2.0 ** -17 * (torch.arange(15, device="cuda") - 7).double()
        logits[:, 5] = first.float()
        logits[:, 7] = logits[:, 5] - places * 2.0 ** -17
        bias = torch.zeros(experts, dtype=torch.float64, device="cuda")
        bias[7] = (places + 0.5) * 2.0 ** -143  # a half more than what the score is less
        for k in (1, 2, 3):
            check(logits, k, bias=bias.float())
