"""The rule that chooses how the CTAs of an experts' product share a tile, without a GPU: the row
tiles it counts with are those that experts can have."""
import random
import subprocess

import pytest

from table_embedding_bag_gb300 import _build

SMS = 152
ALONE, PAIR, SPLIT = range(3)

SOURCE = r"""
#include <cstdio>
#include "product_form.h"
int main() {
  long long rows, n, kb, experts, tile;
  int sms;
  while (std::scanf("%lld %lld %lld %lld %lld %d", &rows, &n, &kb, &experts, &tile, &sms) == 6) {
    const tbe::ProductForm f = tbe::product_form(rows, n, kb, experts, sms);
    std::printf("%lld %lld %d %d\n", (long long)tbe::most_row_tiles(rows, experts, tile),
                (long long)tbe::likely_row_tiles(rows, experts, tile), int(f.share), f.cluster);
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("form")
    (d / "t.cpp").write_text(SOURCE)
    exe = str(d / "t")
    subprocess.run(["g++", "-std=c++17", "-I", _build.CSRC, str(d / "t.cpp"), "-o", exe],
                   check=True)

    def run(cases):
        lines = "".join(" ".join(map(str, c)) + "\n" for c in cases)
        out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def test_row_tiles(ask):
    rng = random.Random(1)
    cases, most_seen, mean = [], [], []
    for _ in range(400):
        rows, experts = rng.randint(1, 40), rng.randint(1, 12)
        tile = rng.randint(1, 9)
        seen = []
        for _ in range(30):
            of = [rng.randrange(experts) for _ in range(rows)]
            seen.append(sum(-(-of.count(e) // tile) for e in range(experts)))
        one_row_each = min(rows, experts)  # the partition with the most tiles
        rest = rows - one_row_each
        seen.append(one_row_each - 1 + -(-(rest + 1) // tile))
        cases.append((rows, 64, 4, experts, tile, SMS))
        most_seen.append(max(seen))
        mean.append(sum(seen[:-1]) / 30)
    for c, (most, likely, _, _), at_most, expected in zip(cases, ask(cases), most_seen, mean):
        assert most >= at_most, c
        assert most == at_most or c[3] > 1, c
        assert 1 <= likely <= most, c
        if c[3] == 1:
            assert likely == -(-c[0] // c[4]), c
        if c[0] >= 4 * c[3] and c[4] > 2:  # experts with several rows: a tile for two experts
            assert abs(likely - expected) <= 1 + c[3] / 2, c


@pytest.mark.parametrize("rows,n,k", [
    (1, 1024, 128), (16, 128000, 4096), (100, 16384, 4096), (128, 32000, 4096), (64, 20000, 128)])
def test_one_expert_with_a_tile_of_rows_gets_no_pairs(ask, rows, n, k):
    # a pair's second CTA would hold no row
    (_, _, share, _), = ask([(rows, n, -(-k // 128), 1, 128, SMS)])
    assert share == ALONE


def test_many_rows_go_to_pairs_and_few_are_split(ask):
    assert ask([(65536, 4096, 16, 16, 128, SMS)])[0][2:] == (PAIR, 2)
    assert ask([(2048, 4096, 32, 1, 128, SMS)])[0][2:] == (PAIR, 2)
    assert ask([(1, 4096, 32, 1, 128, SMS)])[0][2:] == (SPLIT, 4)
    assert ask([(5000, 1000, 8, 8, 128, SMS)])[0][2:] == (ALONE, 1)


def test_every_form_can_be_launched(ask):
    rng = random.Random(2)
    cases = [(rng.choice([1, 127, 128, 129, 5000, 1 << 20]), rng.choice([1, 128, 4096, 128000]),
              rng.randint(1, 80), rng.choice([1, 2, 64, 1024]), 128, rng.choice([1, 2, 80, 152]))
             for _ in range(500)]
    for c, (most, _, share, cluster) in zip(cases, ask(cases)):
        if share == SPLIT:  # every part has blocks, and all parts are resident
            assert cluster in (2, 4, 8) and c[2] >= 2 * cluster
            assert most * -(-c[1] // 128) * cluster <= c[5]
        else:
            assert cluster == 1 + (share == PAIR)
