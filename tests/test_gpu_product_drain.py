"""The end of the experts' product: what is still in flight when its CTAs end.

The last MMAs of a pair of CTAs are issued by the first and arrive at barriers
of both, so both wait for that arrival, and a wait for it that runs out is
reported like any other.  A test-only build (-DTBE_TEST_STUCK_DRAIN) makes such
a wait run out after the MMAs are done; another (-DTBE_TEST_STUCK_COPY) makes the
second CTA of every pair give up while the first goes on.  No fault, no hang."""
import ctypes
import time

import pytest
import torch

import table_embedding_bag_gb300 as tbe
from table_embedding_bag_gb300 import _build, experts

pytestmark = pytest.mark.gpu

FORMS = [(20000, 1024, 512, 4), (3000, 512, 256, 8), (3, 256, 1024, 2)]  # pairs, alone, split


def operands(rows, n, k, groups, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    a, sa = tbe.tbe_quantize_rows(torch.randn(rows, k, generator=g, device="cuda"))
    w, sw = tbe.tbe_quantize_weights(torch.randn(groups, n, k, generator=g, device="cuda"))
    return a, sa, w, sw, torch.linspace(0, rows, groups + 1).int().cuda()


def stuck_build(d, flag):
    path = _build.build(extra_flags=[f"-D{flag}=4096"], lib=str(d / "libtbe_stuck.so"),
                        objdir=str(d / "obj"))
    return tbe.configure(ctypes.CDLL(path))


@pytest.fixture(scope="module")
def stuck_lib(tmp_path_factory):
    return stuck_build(tmp_path_factory.mktemp("stuck_drain"), "TBE_TEST_STUCK_DRAIN")


@pytest.fixture(scope="module")
def stuck_copy_lib(tmp_path_factory):
    return stuck_build(tmp_path_factory.mktemp("stuck_copy"), "TBE_TEST_STUCK_COPY")


@pytest.mark.parametrize("rows,n,k,groups", FORMS)
def test_a_drain_that_runs_out_is_reported(stuck_lib, monkeypatch, rows, n, k, groups):
    args = operands(rows, n, k, groups)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setattr(experts, "_lib_", stuck_lib)
    tbe.tbe_expert_product(*args, status=status)
    torch.cuda.synchronize()
    assert int(status) & 4  # TBE_ERR_TIMEOUT


@pytest.mark.parametrize("rows,n,k,groups", [
    (20000, 1024, 512, 4), (40000, 4096, 1152, 3), (20000, 2000, 256, 1)])
def test_one_cta_of_a_pair_gives_up(stuck_copy_lib, monkeypatch, rows, n, k, groups):
    # the copies that it leaves out are issued after all, so that every copy can be waited for
    args = operands(rows, n, k, groups)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = tbe.tbe_expert_product(*args, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    monkeypatch.setattr(experts, "_lib_", stuck_copy_lib)
    for _ in range(2):
        status.zero_()
        torch.cuda.synchronize()
        start = time.monotonic()
        tbe.tbe_expert_product(*args, status=status)
        torch.cuda.synchronize()
        # 4096 polls and the ways out, not the 4.7 s of a wait for copies that never come
        assert time.monotonic() - start < 3.0
        assert int(status) & 4  # TBE_ERR_TIMEOUT
    monkeypatch.undo()
    status.zero_()
    got = tbe.tbe_expert_product(*args, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and torch.equal(got, want)


def test_products_of_every_form_one_after_another():
    # each call's CTAs take over the shared memory of the ones before while those end
    cases = [operands(*f, seed=i) for i, f in enumerate(FORMS * 2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = [tbe.tbe_expert_product(*c, status=status).clone() for c in cases]
    torch.cuda.synchronize()
    for _ in range(50):
        got = [tbe.tbe_expert_product(*c, status=status) for c in cases]
    torch.cuda.synchronize()
    assert int(status) == 0
    assert all(torch.equal(g, w) for g, w in zip(got, want))
