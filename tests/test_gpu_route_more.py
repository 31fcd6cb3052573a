"""More of routing on the GPU: groups that take 33 to 64 experts a lane, and biases that differ by
less than the choice's last bit in fp32, among choices most of which need exact arithmetic."""
import math

import pytest
import torch

from .test_gpu_route import HOW, check, gen, randn, with_bias

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts,groups,top_groups,k", [(1020, 17, 3, 8), (1020, 20, 4, 20),
                                                         (1024, 32, 5, 9), (660, 20, 20, 31)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("how", HOW)
def test_groups_of_many_experts(experts, groups, top_groups, k, best, how):
    for dtype in (torch.float16, torch.bfloat16, torch.float32):
        g = gen(experts + k)
        logits = (1.5 * randn(g, 200, experts)).to(dtype)
        logits[randn(g, 200, experts) > 1.2] = -math.inf
        check(logits, k, groups=groups, top_groups=top_groups, group_best=best,
              **with_bias(how, experts, g))


@pytest.mark.parametrize("experts,k", [(16, 3), (24, 7), (100, 8), (256, 8), (600, 15), (1000, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_that_differ_by_their_last_bits(experts, k, score):
    g = gen(experts)
    logits = 1.0 + 2.0 ** -22 * torch.randint(0, 400, (300, experts), generator=g,
                                              device="cuda").float()
    bias = torch.full((experts,), 0.125, device="cuda")
    bias[::3] += 2.0 ** -26  # fp32's step there
    assert bias.unique().numel() == 2
    for how in (dict(), dict(renormalize=False)):
        check(logits, k, score=score, bias=bias, **how)
    for groups, top_groups in ((4, 2), (2, 1)):
        check(logits, min(k, experts // 2), score=score, bias=bias, groups=groups,
              top_groups=top_groups, group_best=2)
