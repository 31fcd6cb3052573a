"""Token embedding, norm, routing and the expert layer as one run, forward and
backward, against the same run written in 64 bits.

Tolerance: the 8-bit rows are off by 2^-4 of a value, the weights likewise; each sum
over a row's columns averages those errors, so results are compared by their 2-norm: within
2^-3 of it (both errors at once, four times over).  What does not go through 8 bits is held to
its own type."""
import importlib.util
import math
import os

import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu


def test_embed_norm_route_experts_and_back():
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    tokens, rows, width, experts, k = 600, 1000, 256, 8, 2
    ids = torch.randint(-1, rows, (tokens,), generator=g, device="cuda")
    table, weight = rand(rows, width).bfloat16(), (1 + 0.1 * rand(width)).bfloat16()
    router, w = rand(experts, width) / 16, rand(experts, width, width) / 16
    res, bias = rand(tokens, width).bfloat16(), 0.05 * rand(experts)
    w8, w8_t = tbe.tbe_quantize_weights(w), tbe.tbe_quantize_weights(w.mT.contiguous())

    x = tbe.tbe_embed(table, ids, 1.5)
    y, h = tbe.tbe_rms_norm(x, weight, residual=res)
    q, scale, h8 = tbe.tbe_rms_norm_fp8(x, weight, residual=res)
    assert torch.equal(h, h8)
    logits = y.float() @ router.T
    chosen, cw = tbe.tbe_expert_route(logits, k, bias=bias, score="sigmoid")
    offsets, source, position = tbe.tbe_expert_sort(chosen, experts)
    dispatched = tbe.tbe_expert_dispatch_fp8(y, offsets, position)
    out_rows = tbe.tbe_expert_product(*dispatched, *w8, offsets, out_dtype=torch.float32)
    out = tbe.tbe_expert_combine(out_rows, position, cw)
    # one expert for everybody takes the norm's 8-bit rows as they are
    dense = tbe.tbe_expert_product(q, scale, w8[0][:1], w8[1][:1], out_dtype=torch.float32)

    grad_out = rand(tokens, width)
    g_rows, g_w = tbe.tbe_expert_combine_backward(grad_out, out_rows, offsets, position, cw)
    g_in = tbe.tbe_expert_product(*tbe.tbe_quantize_rows(g_rows), *w8_t, offsets,
                                  out_dtype=torch.float32)
    g_y = tbe.tbe_expert_dispatch_backward(g_in, position)
    g_logits = tbe.tbe_expert_route_backward(g_w, logits, chosen, score="sigmoid")
    g_y = (g_y + g_logits @ router).bfloat16()
    g_x, g_weight = tbe.tbe_rms_norm_backward(g_y, h, weight)
    g_table = tbe.tbe_embed_backward(g_x, ids, rows, 1.5, out_dtype=torch.float32)

    # the same in 64 bits, with the choice that was made
    t64, w64 = table.double().requires_grad_(), weight.double().requires_grad_()
    on = ids >= 0
    x64 = torch.where(on[:, None], t64[ids.clamp_min(0)] * 1.5, 0.0)
    h64 = x64 + res.double()
    y64 = h64 / torch.sqrt(h64.square().mean(1, keepdim=True) + 1e-6) * w64
    l64 = y64 @ router.double().T
    s64 = torch.sigmoid(l64)
    c64 = (s64 + bias.double()).detach()
    want = c64.sort(1, descending=True).indices[:, :k]
    # the logits come from bf16 rows: choices may differ where c agree to 2^-6
    assert float((want == chosen).double().mean()) > 0.9
    s64 = s64.gather(1, chosen.long())
    cw64 = s64 / s64.sum(1, keepdim=True)
    o64 = torch.einsum("nkij,nj->nki", w.double()[chosen.long()], y64)
    out64 = (o64 * cw64[..., None]).sum(1)
    near = lambda a, b: float((a.double() - b).norm()) <= 2.0 ** -3 * float(b.norm())
    assert near(out, out64.detach())
    assert near(dense, (y64 @ w.double()[0].T).detach())
    (out64 * grad_out.double()).sum().backward()
    assert near(g_table, t64.grad) and near(g_weight, w64.grad)


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "token_layer.py")
    spec = importlib.util.spec_from_file_location("token_layer_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_example_runs(example):
    losses, norms = example.train(steps=3, tokens=700, rows=300, width=256)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses + norms)
    assert all(v > 0 for v in losses + norms)


def test_the_examples_gradients(example):
    # against automatic differentiation in 64 bits with the choice that was made
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    layer = example.TokenLayer(200, 256, 8, 2, g)
    ids = torch.randint(-1, 200, (500,), generator=g, device="cuda")
    position = torch.randn(500, 256, generator=g, device="cuda").bfloat16()
    grad_out = torch.randn(500, 256, generator=g, device="cuda")
    out = layer.forward(ids, position)
    grads = layer.backward(grad_out)
    w8, scale = layer.experts
    blocks = scale.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    w = w8.double() * blocks[:, :256, :256]
    table, weight, router = (p.double().requires_grad_() for p in
                             (layer.table, layer.weight, layer.router))
    x = torch.where((ids >= 0)[:, None], table[ids.clamp_min(0)] * layer.scale, 0.0)
    h = x + position.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * weight
    s = torch.sigmoid(y @ router.T).gather(1, layer.chosen.long())
    cw = s / s.sum(1, keepdim=True)
    answers = torch.einsum("nkij,nj->nki", w[layer.chosen.long()], y)
    want = h + (answers * cw[..., None]).sum(1)
    near = lambda a, b: float((a.double() - b).norm()) <= 2.0 ** -3 * float(b.norm())
    assert near(out, want.detach())
    (want * grad_out.double()).sum().backward()
    for got, p in zip(grads, (table, weight, router)):
        assert near(got, p.grad)
