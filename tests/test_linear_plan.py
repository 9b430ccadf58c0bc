"""The linear layer's rule for its tiles, asked through a host build of its own header: the sizes that
the GPU tests of each tile run at do take that tile."""
import os
import shutil
import subprocess

import pytest

from tests.linear_tiles import PIPELINED, STAGED, outputs_and_reduction

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_variable_size_amd", "csrc")
ASK = r"""
#include <stdio.h>
#include "linear_plan.hpp"
int main() {
  long m, n, k;
  while (scanf("%ld %ld %ld", &m, &n, &k) == 3) {
    const moe::Plan p = moe::plan_of(m, n, k), s = moe::staged_plan(m, n, k, true);
    const long bm = moe::kShapeM[p.shape], bn = moe::kShapeN[p.shape];
    const long wgs = ((m + bm - 1) / bm) * ((n + bn - 1) / bn) * p.splits;
    printf("%ld %ld %d %d %d %d %ld\n", bm, bn, p.splits, moe::ring_stages(wgs, 256), s.shape, s.splits,
           (long)moe::launch_rows(m, n));
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


def test_pipelined_sizes_take_their_tiles(ask):
    got = ask([outputs_and_reduction(*c[:4]) for c in PIPELINED])
    assert len(got) == len(PIPELINED)
    for (product, M, K, N, tile, ranges), (bm, bn, splits, ring, _, _, _) in zip(PIPELINED, got):
        name = f"ring{ring}" if (bm, bn) == (128, 128) else f"{bm}x{bn}"
        assert (name, splits) == (tile, ranges), (product, M, K, N)
        # whole 16-byte chunks of every row, operands below 2 GiB
        rows = {"fwd": (K,), "dX": (N, K), "dW": (N, K)}[product]
        assert all(r % 8 == 0 for r in rows) and 2 * max(M * K, N * K, M * N) < 1 << 31


def test_every_tile_has_an_odd_and_an_even_number_of_stages():
    seen = {}
    for product, M, K, N, tile, ranges in PIPELINED:
        if ranges == 1:
            n = (outputs_and_reduction(product, M, K, N)[2] + 63) // 64
            assert n > 4
            seen.setdefault((product, tile), set()).add(n % 2)
    assert len(seen) == 12 and all(v == {0, 1} for v in seen.values())


def test_staged_sizes_take_wide_tiles(ask):
    got = ask([outputs_and_reduction(*c[:4]) for c in STAGED])
    for (product, M, K, N, run), g in zip(STAGED, got):
        assert g[4:6] == (2, 1), (product, M, K, N)
        rows = (K,) if product == "fwd" else (N, K)
        assert any(r % 8 for r in rows) and all(r % 4 == 0 for r in rows) == (run == 4)


def test_no_launch_holds_too_many_work_items(ask):
    """Every run of rows stays below 2^32 work-items in the kernel that takes most of them, keeps 16-byte
    lines, and splits no reduction (the workspace is sized for the whole product, which splits none)."""
    sizes = [(M, N, K) for M in (1, 300, (1 << 22) + 1, 1 << 25, (1 << 25) + 1, (1 << 26) + 77, 1 << 30,
                                 (1 << 31) - 513) for N in (1, 16, 17, 64, 500, 4096, 16384, 65536, 1 << 22)
             for K in (1, 8, 1 << 22) if M * N <= 1 << 37]
    runs = []
    for (M, N, K), g in zip(sizes, ask(sizes)):
        run = g[6]
        tiles = -(-N // 64)
        for rows in {min(run, M), M % run or run}:
            assert -(-rows // 64) * tiles * 256 < 1 << 32
            assert N > 16 or -(-rows // 16) * 1024 < 1 << 32
            if run < M:
                assert run % 64 == 0
                runs.append((rows, N, K))
        assert run == M or M > 1 << 25 or M * N > 1 << 35
    assert runs
    for size, (_, _, splits, _, _, staged_splits, _) in zip(runs, ask(runs)):
        assert splits == 1 and staged_splits == 1, size
