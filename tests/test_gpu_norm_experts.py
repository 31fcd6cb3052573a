"""The norm in 8 bits on its way into products, on the GPU: by one expert for all rows, and by
routed experts, whose rows are gathered by an index here; with fp32 rows both are bit for bit what
tbe_rms_norm and tbe_expert_dispatch_fp8 give."""
import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


@pytest.mark.parametrize("tokens,width,experts,k", [(1, 128, 4, 2), (300, 256, 8, 2), (77, 640, 5, 3)])
def test_the_same_rows_either_way(tokens, width, experts, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, res, weight = rand(tokens, width), rand(tokens, width), 1 + 0.1 * rand(width)
    y, h = tbe.tbe_rms_norm(x, weight, residual=res)
    q, scale, h8 = tbe.tbe_rms_norm_fp8(x, weight, residual=res)
    assert torch.equal(h, h8)
    ids, weights = tbe.tbe_expert_route(rand(tokens, experts), k)
    ids[::3, 0] = -1  # dropped
    offsets, source, position = tbe.tbe_expert_sort(ids, experts)
    rows, scales = tbe.tbe_expert_dispatch_fp8(y, offsets, position)
    kept = int(offsets[-1])
    token = source[:kept].long() // k
    assert torch.equal(bits(q)[token], bits(rows)[:kept])
    assert torch.equal(scale[token], scales[:kept])
    w8, w_scale = tbe.tbe_quantize_weights(rand(experts, width, width) / 16)
    gathered, gathered_scale = torch.zeros_like(bits(rows)), torch.zeros_like(scales)
    gathered[:kept], gathered_scale[:kept] = bits(q)[token], scale[token]
    want = tbe.tbe_expert_product(rows, scales, w8, w_scale, offsets, out_dtype=torch.float32)
    got = tbe.tbe_expert_product(gathered.view(rows.dtype), gathered_scale, w8, w_scale, offsets,
                                 out_dtype=torch.float32)
    assert torch.equal(got, want)
    # one expert for all rows takes them as they are
    one = tbe.tbe_expert_product(q, scale, w8[:1], w_scale[:1], out_dtype=torch.float32)
    same = tbe.tbe_expert_product(*tbe.tbe_quantize_rows(y), w8[:1], w_scale[:1],
                                  out_dtype=torch.float32)
    assert torch.equal(one, same)
