"""Every element of a product's output is defined: rows that belong to no expert are
zeros, before the first expert's as after the last one's."""
import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu


def operands(rows, n, k, experts, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    a, sa = tbe.tbe_quantize_rows(torch.randn(rows, k, generator=g, device="cuda"))
    w, sw = tbe.tbe_quantize_weights(torch.randn(experts, n, k, generator=g, device="cuda"))
    return a, sa, w, sw


@pytest.mark.parametrize("rows,n,k", [
    (400, 256, 1024), (3001, 500, 256), (20000, 1024, 512)])  # split, alone, pairs
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_a_part_of_the_experts_leaves_the_other_rows_zero(rows, n, k, dtype):
    a, sa, w, sw = operands(rows, n, k, 6)
    cuts = [0, rows // 5, rows // 5, rows // 3, rows // 2 + 1, rows - 40, rows - 7]
    offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    whole = tbe.tbe_expert_product(a, sa, w, sw, offsets, out_dtype=dtype)
    for first, last in [(2, 4), (1, 6), (5, 6), (0, 1)]:
        out = torch.full((rows, n), float("nan"), dtype=dtype, device="cuda")
        got = tbe.tbe_expert_product(a, sa, w[first:last], sw[first:last],
                                     offsets[first:last + 1], out=out)
        lo, hi = cuts[first], cuts[last]
        assert not got[:lo].any() and not got[hi:].any()
        assert torch.allclose(got[lo:hi].float(), whole[lo:hi].float(), rtol=2 ** -7, atol=2 ** -7)


@pytest.mark.parametrize("cuts", [[5, 5, 5], [20, 20, 20], [30, 40, 50], [12, 12, 3]])
def test_no_expert_has_a_row(cuts):
    a, sa, w, sw = operands(20, 24, 32, 2)
    out = torch.full((20, 24), float("nan"), device="cuda")
    tbe.tbe_expert_product(a, sa, w, sw, torch.tensor(cuts, dtype=torch.int32).cuda(), out=out)
    assert not out.any()
