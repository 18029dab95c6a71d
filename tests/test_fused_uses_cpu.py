"""What a product is for decides, too, which kernel it takes (csrc/fused_choice.h,
compiled for the host)."""

from __future__ import annotations

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_fp32_gemm_row_amd", "csrc")
SOURCE = r"""
#include "fused_choice.h"
#include <cstdio>
using namespace gemm_f32_impl::fused;
int main() {
    int use, tb, space;
    long long b, M, N, K;
    while (std::scanf("%d %d %d %lld %lld %lld %lld", &use, &tb, &space, &b, &M, &N, &K) == 7) {
        const Choice c = choose(tb != 0, b, M, N, K, space != 0, static_cast<Use>(use));
        std::printf("%d %d %d %d\n", c.tile, c.splits, c.half ? 1 : 0, c.shape);
    }
    return 0;
}
"""
PLAIN, STATISTICS, PROBABILITIES = range(3)
ROWS = 3  # kRows


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    """choose([(use, tb, space, batch, M, N, K)]) -> [(tile, splits, half, shape)]"""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    tmp = tmp_path_factory.mktemp("uses")
    (tmp / "uses.cpp").write_text(SOURCE)
    exe = tmp / "uses"
    res = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(tmp / "uses.cpp"),
                          "-o", str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stderr

    def ask(wanted):
        text = "".join(" ".join(str(int(v)) for v in w) + "\n" for w in wanted)
        run = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60)
        assert run.returncode == 0
        lines = [tuple(map(int, ln.split())) for ln in run.stdout.splitlines()]
        assert len(lines) == len(wanted)
        return lines

    return ask


def sizes(n, most=(14, 17, 14)):
    rng = random.Random(2)
    return [tuple(int(round(2 ** rng.uniform(0, m))) for m in most) for _ in range(n)]


def test_probabilities_take_no_fp16_parts(choose):
    """Their range is not known: P W (rows as stored) and P^T X (rows transposed)."""
    drawn = sizes(5000)
    plain = choose([(PLAIN, 0, 1, 1, *s) for s in drawn])
    got = choose([(PROBABILITIES, 0, 1, 1, *s) for s in drawn])
    assert any(half for _, _, half, _ in plain) and not any(half for _, _, half, _ in got)
    # in all else as any product: what did not take them stays as it was, and slices stay allowed
    assert all(p == q for p, q in zip(plain, got) if not p[2])
    assert any(splits > 1 for _, splits, _, _ in got)


def test_few_columns_take_a_kernel_that_serves_them(choose):
    """The tiles load 4 neighbouring columns of a B stored K x N at once, and 4
    neighbouring rows of an A stored K x M: no choice may count on them where there are fewer."""
    wanted = [(use, 0, space, batch, M, N, K) for use in (PLAIN, PROBABILITIES) for space in (0, 1) for batch in (1, 50)
              for N in (1, 2, 3) for M in (1, 2, 3, 5, 16, 31, 32, 33, 64, 1000, 8192, 131072) for K in (1, 40, 4096, 1 << 20)]
    for want, (tile, splits, half, shape) in zip(wanted, choose(wanted)):
        _, _, space, _, M, N, K = want
        assert tile == ROWS and not half, (want, tile)
        assert 1 <= (shape & 15) <= N and shape >> 4 <= max(1, (M + 15) // 16), (want, shape)
        assert splits == 1 or (space and K >= 64 * splits), (want, splits)
    # few rows of either form
    wanted = [(use, tb, 1, 1, M, N, K) for use in range(3) for tb in (0, 1) for M in range(1, 33) for N in (1, 2, 3, 4, 100)
              for K in (1, 5000) if tb or use != STATISTICS]
    assert all(tile == ROWS for tile, _, _, _ in choose(wanted))
