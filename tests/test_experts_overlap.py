"""An output that shares memory with an input of its call is refused, without a GPU: which ranges
share memory is compared with the sets of their bytes, and the calls refuse before any launch."""
import ctypes
import random
import subprocess

import pytest

import table_embedding_bag_gb300 as tbe
from table_embedding_bag_gb300 import _build

BASE = 1 << 20  # never dereferenced by the host-side checks
F16, I32, BF16, F32 = 1, 2, 4, 5

SOURCE = r"""
#include <cstdio>
#include "rows.cuh"
int main() {
  long long a[4], b[4];
  while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld", a, a + 1, a + 2, a + 3, b, b + 1,
                    b + 2, b + 3) == 8)
    std::printf("%d\n", tbe::overlap({reinterpret_cast<void*>(a[0]), a[1], a[2], a[3]},
                                     {reinterpret_cast<void*>(b[0]), b[1], b[2], b[3]}));
}
"""


def held(p, rows, width, stride):
    return {p + r * stride + c for r in range(rows) for c in range(width)}


def test_overlap_is_that_of_the_bytes(tmp_path):
    (tmp_path / "t.cu").write_text(SOURCE)
    exe = str(tmp_path / "t")
    subprocess.run([_build._nvcc(), *_build.NVCC_FLAGS, str(tmp_path / "t.cu"), "-o", exe],
                   check=True)
    rng = random.Random(3)
    cases = []
    for i in range(6000):
        a, b = ([100 + rng.randint(0, 80), rng.randint(1, 6), w, w + rng.choice([0, 0, 1, 5, 20])]
                for w in (rng.randint(1, 12), rng.randint(1, 12)))
        if i % 2:
            b[3] = a[3] = max(a[3], b[3])  # columns of one buffer
        cases.append((a, b))
    lines = "".join(" ".join(map(str, a + b)) + "\n" for a, b in cases)
    out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout
    got = [line == "1" for line in out.split()]
    assert len(got) == len(cases)
    shared = beside = 0
    for (a, b), refused in zip(cases, got):
        meet = bool(held(*a) & held(*b))
        assert refused or not meet, (a, b)
        if a[3] == b[3] or 1 in (a[1], b[1]):
            assert refused == meet, (a, b)
            beside += not meet and a[0] < b[0] < a[0] + (a[1] - 1) * a[3]
        shared += meet
    assert shared > 500 and beside > 100  # both kinds were there


@pytest.fixture(scope="module")
def lib():
    tbe.build()
    return tbe.configure(ctypes.CDLL(tbe.lib_path))


def at(nbytes):
    return BASE + nbytes


X, OFF, POS, W, OUT = (at(i << 24) for i in range(5))  # 8 tokens, k = 2, width 32, 4 experts


@pytest.mark.parametrize("call,args", [
    # the sort, into its ids, and source and position in one buffer
    ("tbe_expert_sort", (X, I32, 8, 2, 4, OFF, W, X, None)),
    ("tbe_expert_sort", (X, I32, 8, 2, 4, X + 60, W, POS, None)),
    ("tbe_expert_sort", (X, I32, 8, 2, 4, OFF, POS, POS + 4, None)),
    # one expert each, in place; rows that begin in x's last row; columns that meet
    ("tbe_expert_dispatch", (X, F16, 8, 1, 32, 32, OFF, 4, POS, X, 32, None)),
    ("tbe_expert_dispatch", (X, F16, 8, 2, 32, 32, OFF, 4, POS, X + 510, 32, None)),
    ("tbe_expert_dispatch", (X, F16, 8, 1, 32, 64, OFF, 4, POS, X + 62, 64, None)),
    ("tbe_expert_dispatch_fp8", (X, F16, 8, 2, 32, 32, OFF, 4, POS, X + 256, 32, W, None)),
    ("tbe_expert_dispatch_fp8", (X, BF16, 8, 1, 32, 32, None, 0, None, X, 64, W, None)),
    ("tbe_quantize_weights", (X, F32, 2, 8, 16, X + 1008, W, None)),
    ("tbe_expert_combine", (X, F32, 8, 1, 32, 32, POS, None, X, 32, None)),
    ("tbe_expert_combine", (X, F32, 8, 2, 32, 32, POS, W, X + 2044, 32, None)),
    ("tbe_expert_combine_backward",
     (X, OUT, BF16, 8, 1, 32, 32, 32, OFF, 4, POS, None, X, 32, W, None)),
    ("tbe_expert_combine_backward",
     (X, OUT, BF16, 8, 2, 32, 32, 32, OFF, 4, POS, None, OUT + 2, 32, W, None)),
    ("tbe_expert_product", (X, 32, W, POS, W, OFF, 8, 16, 32, 2, X + 16, BF16, 16, None, None)),
    ("tbe_expert_product", (X, 32, W, POS, W, OFF, 8, 16, 32, 2, POS, BF16, 16, None, None)),
])
def test_outputs_over_inputs_are_refused(lib, call, args):
    before = lib.tbe_kernel_launches()
    assert getattr(lib, call)(*args) == tbe.TBE_EINVAL
    assert lib.tbe_kernel_launches() == before
