"""The bounded-wait way out of the experts' product, without any fault or hang: a
test-only build (-DTBE_TEST_STUCK_WAIT) makes the epilogue's first wait one on an
mbarrier that nothing arrives on, bounded by a few thousand polls.  Every CTA
then gives up, lets its copies and MMAs end, frees its tensor memory and sets
TBE_ERR_TIMEOUT in the caller's status word; the context stays usable."""
import ctypes

import pytest
import torch

import table_embedding_bag_gb300 as tbe
from table_embedding_bag_gb300 import _build, experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def stuck_lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("stuck_product")
    path = _build.build(extra_flags=["-DTBE_TEST_STUCK_WAIT=4096"], lib=str(d / "libtbe_stuck.so"),
                        objdir=str(d / "obj"))
    return tbe.configure(ctypes.CDLL(path))


@pytest.mark.parametrize("rows,n,k,groups", [
    (20000, 1024, 512, 4), (3000, 512, 256, 8), (3, 256, 1024, 2)])  # CTAs in pairs, alone, split
def test_product_wait_runs_out_and_reports(stuck_lib, monkeypatch, rows, n, k, groups):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    a, sa = tbe.tbe_quantize_rows(torch.randn(rows, k, generator=g, device="cuda"))
    w, sw = tbe.tbe_quantize_weights(torch.randn(groups, n, k, generator=g, device="cuda"))
    offsets = torch.linspace(0, rows, groups + 1).int().cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = tbe.tbe_expert_product(a, sa, w, sw, offsets, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    monkeypatch.setattr(experts, "_lib_", stuck_lib)
    for _ in range(2):  # the second call finds tensor memory free again
        status.zero_()
        tbe.tbe_expert_product(a, sa, w, sw, offsets, status=status)
        torch.cuda.synchronize()
        assert int(status) & 4  # TBE_ERR_TIMEOUT
    monkeypatch.undo()
    status.zero_()
    got = tbe.tbe_expert_product(a, sa, w, sw, offsets, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and torch.equal(got, want)
