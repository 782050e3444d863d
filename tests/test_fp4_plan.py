"""The tiles that 4-bit products take, computed by the library's own host code."""
import os
import subprocess

import pytest

from tests.fp4_shapes import PLANS

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "maxsim_scoring_gb300", "csrc")
MAIN = """
#include <cstdio>
#include "linear_fp4_plan.h"
int main() {
    long long m, n, k;
    while (std::scanf("%lld %lld %lld", &m, &n, &k) == 3) {
        const maxsim::LinearFp4Plan p = maxsim::plan_linear_fp4(m, n, k);
        std::printf("%d %d %d %lld %lld %d %d\\n", p.tn, int(p.swap), p.splits, (long long)p.tiles, (long long)p.tiles_b, p.kb, p.kb_split);
    }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    where = tmp_path_factory.mktemp("plan")
    (where / "plan.cpp").write_text(MAIN)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, "-o", str(where / "plan"), str(where / "plan.cpp")])

    def of(sizes):
        out = subprocess.run([str(where / "plan")], input="\n".join(" ".join(map(str, s)) for s in sizes), text=True, capture_output=True, check=True)
        return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
    return of


def test_tested_products_reach_every_tile_kernel(plans):
    """Each size has the plan it is there for, so that a change of the plan cannot leave a kernel without its tests."""
    for size, got in zip(PLANS, plans(PLANS)):
        tn, swap, splits, tiles, _, _, _ = got
        want = PLANS[size]
        assert (tn, bool(swap), splits) == want[:3], size
        assert -(-tiles // 76) >= want[3] and (splits == 1 or tiles <= 36), size
    reached = {p[:2] for p in PLANS.values()}
    assert reached == {(tn, swap) for tn in (64, 128, 256) for swap in (False, True)}
    for tn in (64, 128, 256):  # 16-bit rows on their 16-byte boundaries, and off them
        assert {size[1] % 8 == 0 for size, p in PLANS.items() if p[:2] == (tn, False)} == {True, False}
    assert {p[2] for p in PLANS.values()} == {1, 2, 4}


def test_plans_cover_the_product(plans):
    """Tiles and stages of any sizes cover the operands, and a cluster's pairs share out all of K."""
    sizes = [(m, n, k) for m in (1, 63, 64, 65, 128, 255, 257, 5000, 1 << 20, (1 << 31) - 1024) for n in (1, 64, 129, 4096, 100000)
             for k in (32, 256, 288, 4096, 16384, 1 << 28)]
    for (m, n, k), (tn, swap, splits, tiles, tiles_b, kb, kb_split) in zip(sizes, plans(sizes)):
        a, b = (n, m) if swap else (m, n)
        assert bool(swap) == (n > m) and tiles_b == -(-b // tn) and tiles == -(-a // 256) * tiles_b and kb == -(-k // 256)
        assert splits in (1, 2, 4) and kb_split * splits >= kb > kb_split * (splits - 1)
        assert splits == 1 or (tn == 64 and tiles <= (36 if splits == 2 else 15))
