"""A product whose device wait gave up does not pass for a whole one: the rows it may have lost
are NaN, with a status word or without.  The wait is made to run out by a test-only build
(-DTBE_TEST_STUCK_WAIT): no fault, no hang."""
import ctypes

import pytest
import torch

import table_embedding_bag_gb300 as tbe
from table_embedding_bag_gb300 import _build, experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def stuck_lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("stuck_lost")
    path = _build.build(extra_flags=["-DTBE_TEST_STUCK_WAIT=4096"], lib=str(d / "libtbe_lost.so"),
                        objdir=str(d / "obj"))
    return tbe.configure(ctypes.CDLL(path))


@pytest.mark.parametrize("rows,n,k,groups", [
    (20000, 1024, 512, 4), (3000, 520, 256, 8), (3, 256, 1024, 2)])  # pairs, alone, split
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_lost_rows_are_nan(stuck_lib, monkeypatch, rows, n, k, groups, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    a, sa = tbe.tbe_quantize_rows(torch.randn(rows, k, generator=g, device="cuda"))
    w, sw = tbe.tbe_quantize_weights(torch.randn(groups, n, k, generator=g, device="cuda"))
    used = rows - 1
    offsets = torch.linspace(0, used, groups + 1).int().cuda()
    monkeypatch.setattr(experts, "_lib_", stuck_lib)
    for pad in (0, 3):  # rows on 16-byte boundaries and off them
        out = torch.full((rows, n + pad), 7.0, dtype=dtype, device="cuda")
        tbe.tbe_expert_product(a, sa, w, sw, offsets, out=out[:, :n])
        torch.cuda.synchronize()
        assert bool(out[:used, :n].isnan().all())
        assert not out[used:, :n].any()  # a row of no expert is still zero
        assert bool((out[:, n:] == 7.0).all())
