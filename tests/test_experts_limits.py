"""Sizes near the ends of 32 bits are refused where a tile that begins inside a matrix would
end past what the kernels count, without a GPU."""
import ctypes

import pytest

import table_embedding_bag_gb300 as tbe

FAKE = 0x1000  # never dereferenced by the host-side checks
MOST = (1 << 31) - 1 - 512


@pytest.fixture(scope="module")
def lib():
    tbe.build()
    return tbe.configure(ctypes.CDLL(tbe.lib_path))


@pytest.mark.parametrize("rows,n,k,experts", [
    (MOST + 1, 16, 16, 1), (MOST + 385, 16, 16, 1), (MOST + 512, 16, 16, 1),
    (8, MOST + 1, 16, 1), (8, MOST + 512, 16, 1), (8, (MOST + 512) // 7, 16, 7),
    (8, 16, (1 << 31) - 16, 1)])
def test_products_that_end_past_32_bits(lib, rows, n, k, experts):
    before = lib.tbe_kernel_launches()
    assert lib.tbe_expert_product(FAKE, k, FAKE, FAKE, FAKE, FAKE, rows, n, k, experts, FAKE, 4, n,
                                  None, None) == tbe.TBE_EUNSUPPORTED
    assert lib.tbe_kernel_launches() == before


@pytest.mark.parametrize("n,k", [(1, MOST + 1), (1, MOST + 512), (MOST + 1, 1)])
def test_weights_that_end_past_32_bits(lib, n, k):
    before = lib.tbe_kernel_launches()
    assert lib.tbe_quantize_weights(FAKE, 4, 1, n, k, FAKE, FAKE, None) == tbe.TBE_EUNSUPPORTED
    assert lib.tbe_kernel_launches() == before
