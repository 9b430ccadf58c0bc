"""The rule for the tiles of the cross entropy's fp32 products, asked through a host build of its own header."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_variable_size_amd", "csrc")
ASK = r"""
#include <stdio.h>
#include "linear_plan.hpp"
int main() {
  long m, n, k;
  while (scanf("%ld %ld %ld", &m, &n, &k) == 3) {
    const moe::Plan a = moe::fine_plan(m, n, k, false), b = moe::fine_plan(m, n, k, true);
    printf("%d %d %d %d %d\n", a.shape, a.splits, b.shape, b.splits, (int)moe::fine_whole(m, n, k));
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "ask.cpp").write_text(ASK)
    exe = str(d / "ask")
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, "-o", exe, str(d / "ask.cpp")], check=True)

    def run(sizes):
        text = "\n".join(" ".join(map(str, s)) for s in sizes)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(map(int, l.split())) for l in out.splitlines()]
    return run


def test_ranges_stay_within_their_limits(ask):
    sizes = [(m, n, k) for m in (1, 17, 129, 1000, 70001, 1 << 24) for n in (4, 65, 5003, 131072, 1 << 22) for k in (4, 63, 1001, 50257, 1 << 22)]
    for (m, n, k), (shape, splits, shape2, splits2, _) in zip(sizes, ask(sizes)):
        assert shape in (1, 2) and splits == 1 and shape2 in (1, 2) and 1 <= splits2 <= 16
        steps, tiles = -(-k // 16), -(-m // (64 * shape2)) * -(-n // (64 * shape2))
        assert splits2 == 1 or (steps >= 4 * splits2 and tiles * splits2 <= 1280 // shape2)


def test_sizes_that_the_gpu_tests_run_take_both_tiles_and_ranges(ask):
    whole = ask([(70, 300, 5), (777, 5003, 101), (1027, 8191, 35)])
    assert all(w[4] for w in whole)
    assert {w[0] for w in ask([(777, 5003, 1001), (65, 130, 67)])} == {1, 2}
    ranged = ask([(33, 700, 4100), (200, 900, 2633)])
    assert all(r[3] > 1 and not r[4] for r in ranged)
    assert {r[2] for r in ask([(33, 700, 4100), (777, 1001, 5003)])} == {1, 2}
