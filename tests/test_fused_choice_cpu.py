"""Which kernel a fused product takes: csrc/fused_choice.h, the code that the
launches ask, compiled for the host."""

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
    int tb, space, statistics;
    long long b, M, N, K;
    while (std::scanf("%d %d %d %lld %lld %lld %lld", &tb, &space, &statistics, &b, &M, &N, &K) == 7) {
        const Choice c = choose(tb != 0, b, M, N, K, space != 0, statistics ? kStatistics : kPlain);
        std::printf("%d %d %d %d\n", c.tile, c.splits, c.half ? 1 : 0, c.shape);
    }
    return 0;
}
"""
ROWS = 3  # kRows


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    """choose([(tb, space, statistics, batch, M, N, K)]) -> [(tile, splits, half, shape)]"""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    tmp = tmp_path_factory.mktemp("choice")
    (tmp / "choice.cpp").write_text(SOURCE)
    exe = tmp / "choice"
    res = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                          str(tmp / "choice.cpp"), "-o", str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stderr

    def ask(wanted):
        text = "".join(" ".join(str(int(v)) for v in w) + "\n" for w in wanted)
        run = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60)
        assert run.returncode == 0
        lines = [tuple(map(int, ln.split())) for ln in run.stdout.splitlines()]
        assert len(lines) == len(wanted)
        return lines

    return ask


def drawn(n):
    rng = random.Random(1)
    size = lambda most: int(round(2 ** rng.uniform(0, most)))
    return [(rng.random() < 0.5, rng.random() < 0.7, rng.random() < 0.3, rng.choice([1, 1, 1, 2, 40]),
             size(14), size(17), size(14)) for _ in range(n)]


def test_choices_are_ones_that_the_kernels_take(choose):
    wanted = drawn(20000) + [(tb, 1, 0, 1, M, N, K) for tb in (0, 1) for M in range(1, 40) for N in range(1, 40)
                             for K in (0, 1, 64)]
    for (tb, space, statistics, batch, M, N, K), (tile, splits, half, shape) in zip(wanted, choose(wanted)):
        what = (tb, space, statistics, batch, M, N, K, tile, splits, half, shape)
        assert tile in (0, 1, 2, ROWS) and 1 <= splits <= 32, what
        if statistics or not space:
            assert splits == 1, what
        if splits > 1:
            assert K >= 64 * splits, what  # every slice has work
        if half:
            assert space and tile in (0, 1) and 64 <= K <= 1 << 22, what
        if tile == ROWS:
            assert shape in (0, 17, 18, 20, 33, 34, 36, 66), what
            if shape == 0:
                assert tb and M <= 4, what
            else:
                r, c = shape >> 4, shape & 15
                # neighbours that a lane loads at once exist
                assert (tb or c <= N) and r <= M + 15 and (r <= 2 or M >= r), what
            assert not statistics or M <= 512, what  # whose pieces are of 16 columns
        else:
            assert M > 32 or N < 4, what


def test_every_kernel_is_taken(choose):
    seen = {(tile, half, shape if tile == ROWS else 0, min(splits, 2))
            for tile, splits, half, shape in choose(drawn(20000))}
    for tile in (0, 1, 2):
        assert (tile, 0, 0, 1) in seen
    for tile in (0, 1):
        assert (tile, 1, 0, 1) in seen and (tile, 1, 0, 2) in seen
    for tile in (1, 2):
        assert (tile, 0, 0, 2) in seen
    for shape in (0, 17, 18, 20, 33, 34, 36, 66):
        assert (ROWS, 0, shape, 1) in seen, shape


# Microseconds of each kernel's best number of slices, measured: {(rows of a B
# stored N x K?, M, N, K): {(tile or shape, half): time}}
MEASURED = {
    (1, 400, 9504, 999): {(0, 0): 98.2, (0, 1): 81.2, (1, 0): 83.9, (1, 1): 75.2, (2, 0): 79.8, (36, 0): 120.7},
    (1, 54, 2720, 13019): {(1, 0): 70.7, (1, 1): 79.7, (2, 0): 52.3, (34, 0): 81.8, (66, 0): 68.3},
    (1, 96, 12249, 332): {(1, 0): 23.3, (1, 1): 28.3, (2, 0): 17.5, (17, 0): 25.9, (36, 0): 30.6},
    (1, 1215, 128, 1088): {(1, 0): 16.4, (2, 0): 14.6, (17, 0): 18.6, (18, 0): 17.2, (34, 0): 13.8, (66, 0): 15.6},
    (1, 160, 4032, 6240): {(0, 0): 90.8, (0, 1): 95.5, (1, 0): 72.9, (1, 1): 72.1, (2, 0): 71.6},
    (1, 721, 1760, 9152): {(0, 0): 160.4, (0, 1): 119.4, (1, 0): 152.3, (1, 1): 124.3, (2, 0): 168.1},
    (1, 192, 96, 3454): {(1, 0): 18.5, (2, 0): 16.0, (17, 0): 10.6, (18, 0): 10.6, (34, 0): 11.0, (66, 0): 12.7},
    (1, 1666, 256, 704): {(1, 0): 19.0, (2, 0): 16.3, (17, 0): 25.1, (34, 0): 17.6, (36, 0): 15.6, (66, 0): 15.3},
    (0, 1922, 4683, 430): {(0, 0): 87.2, (0, 1): 66.7, (1, 0): 72.8, (1, 1): 69.4, (2, 0): 67.8, (36, 0): 117.3},
    (0, 53, 11803, 96): {(1, 0): 15.0, (2, 0): 10.8, (17, 0): 15.6, (34, 0): 11.0, (36, 0): 8.2, (66, 0): 10.1},
    (0, 8087, 6038, 352): {(0, 0): 241.2, (0, 1): 179.6, (1, 0): 213.3, (1, 1): 181.4, (2, 0): 265.2},
    (0, 59, 1267, 1376): {(1, 0): 20.5, (2, 0): 16.7, (17, 0): 12.3, (18, 0): 10.2, (34, 0): 12.8, (66, 0): 13.0},
    (0, 94, 130, 96): {(1, 0): 14.7, (2, 0): 10.5, (17, 0): 4.1, (18, 0): 4.3, (34, 0): 5.5, (66, 0): 5.8},
    (0, 54, 2720, 13019): {(1, 0): 72.1, (2, 0): 52.2, (17, 0): 98.3, (34, 0): 75.8, (36, 0): 63.9},
}


def test_products_take_a_quick_kernel(choose):
    """Within a tenth of the best of the kernels that were timed."""
    got = choose([(tb, 1, 0, 1, M, N, K) for tb, M, N, K in MEASURED])
    for (size, times), (tile, splits, half, shape) in zip(MEASURED.items(), got):
        key = (shape if tile == ROWS else tile, half)
        assert times[key] <= 1.1 * min(times.values()), f"{size} takes {key}"
