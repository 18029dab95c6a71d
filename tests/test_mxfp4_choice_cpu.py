"""Which kernel the MXFP4 products of the tile tests take: csrc/mxfp4_choice.h,
the code that the launches ask, compiled for the host."""

from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from tests import mxfp4_tile_cases as cases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_fp32_gemm_row_amd", "csrc")

SOURCE = r"""
#include "mxfp4_choice.h"
#include <cstdio>
using namespace gemm_f32_impl::mx;
int main() {
    char kind;
    long long b, M, N, K;
    while (std::scanf(" %c %lld %lld %lld %lld", &kind, &b, &M, &N, &K) == 5) {
        if (kind == 'P') {
            static const char *const names[] = {"256x256", "128x128", "rows"};
            const auto c = product_choice::choose(b, M, N, K, kMostSplits);
            const bool fit = product_choice::reaches(K / 2 + 64, N + 64);
            std::printf("%s %d\n", fit ? names[c.kernel] : "rows", c.splits);
        } else {
            static const char *const names[] = {"128x256", "64x256", "64x128"};
            const bool t = kind == 'T';
            const auto c = weight_choice::choose(t, b, M, N, K, kMostSplits);
            const bool fit = weight_choice::tiles_fit(t, b, M, N, K, K + 64, (t ? K : N) / 2 + 64, N + 64);
            std::printf("%s %d\n", fit && c.tile != weight_choice::kDirect ? names[c.tile] : "direct", c.splits);
        }
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    """choose([(kind, (batch, M, N, K))]) -> [(kernel, slices of K)]"""
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
        text = "".join(f"{kind} {' '.join(map(str, size))}\n" for kind, size in wanted)
        run = subprocess.run([str(exe)], input=text, capture_output=True, text=True, timeout=60)
        assert run.returncode == 0
        lines = [ln.split() for ln in run.stdout.splitlines()]
        assert len(lines) == len(wanted)
        return [(name, int(n)) for name, n in lines]

    return ask


def test_product_tile_cases_take_their_tiles(choose):
    want = cases.products()
    got = choose([("P", size) for _, size, _ in want])
    assert got == [(tile, n) for tile, _, n in want]


def test_weight_tile_cases_take_their_tiles(choose):
    want = cases.weights()
    got = choose([(op, size) for op, _, size, _ in want])
    assert got == [(tile, n) for _, tile, _, n in want]


def test_direct_cases_take_no_tile(choose):
    got = choose(cases.DIRECT)
    assert [name for name, _ in got] == ["rows" if kind == "P" else "direct" for kind, _ in cases.DIRECT]


# microseconds measured in a graph (so that no call waits for its host): tiles of
# 128 x 128, of 32 x 32
MEASURED = {(1000, 1023, 777): (7.8, 6.0), (1024, 1024, 777): (7.5, 5.5), (108, 4379, 1761): (9.5, 7.5),
            (2109, 522, 693): (8.0, 6.5), (1024, 512, 4096): (12.8, 11.4), (128, 4096, 4096): (12.8, 11.4),
            (221, 3869, 1061): (8.7, 7.9), (511, 1023, 2077): (10.7, 7.7), (256, 256, 256): (5.9, 2.9),
            (2048, 2048, 512): (8.2, 13.7), (1000, 1000, 4000): (16.1, 24.8), (100, 8193, 1500): (8.7, 10.4),
            (640, 10496, 128): (10.1, 16.6), (1888, 1760, 128): (7.8, 10.1), (193, 5046, 512): (6.5, 6.2),
            (1300, 1300, 1000): (8.4, 11.9), (2000, 2000, 500): (8.6, 14.2), (1024, 1024, 1024): (7.4, 7.4)}


def test_small_products_take_the_quicker_kernel(choose):
    """Within 5% of the better of two kernels that were timed."""
    got = choose([("P", (1, *size)) for size in MEASURED])
    for (size, (medium, rows)), (name, _) in zip(MEASURED.items(), got):
        assert {"128x128": medium, "rows": rows}[name] <= 1.05 * min(medium, rows), f"{size} takes {name}"


def test_tile_cases_cover_every_compiled_form():
    """Each tile with and without slices and a batch, edges inside a tile, and
    both of its compiled forms (K a multiple of 512, or of 4, and not)."""
    for tile, sizes in cases.PRODUCTS.items():
        m, n = map(int, tile.split("x"))
        for whole in (True, False):
            mine = {s: k for s, k in sizes.items() if (s[3] % 512 == 0) == whole}
            assert any(k > 1 for k in mine.values()) and any(k == 1 for k in mine.values()), (tile, whole)
            assert any(s[0] > 1 for s in mine) and any(s[0] == 1 for s in mine), (tile, whole)
            assert any(s[1] % m and s[2] % n for s in mine), (tile, whole)
        held = 256 if m == 256 else 512  # workgroups of the persistent launch
        assert any(s[0] * -(-s[1] // m) * -(-s[2] // n) > held for s, k in sizes.items() if k == 1), tile
    for key, sizes in cases.WEIGHTS.items():
        for quads in (True, False):
            mine = {s: k for s, k in sizes.items() if (s[3] % 4 == 0) == quads}
            assert any(k > 1 for k in mine.values()) and any(k == 1 for k in mine.values()), (key, quads)
            assert any(s[0] == 1 for s in mine), (key, quads)
        assert any(s[0] > 1 for s in sizes), key


def test_far_strides_leave_the_tiles(choose):
    """(the GPU tests run such strides on the kernels of 64-bit offsets)"""
    src = (r'#include "mxfp4_choice.h"' "\nusing namespace gemm_f32_impl::mx;\n"
           "static_assert(kBlock == 32 && kBlockBytes == 16, \"\");\n"
           "int main() { constexpr int64_t far = int64_t{1} << 57;\n"
           "  if (product_choice::reaches(1 << 22, 64) || product_choice::reaches(64, 1 << 20)) return 1;\n"
           "  if (!product_choice::reaches((1 << 22) - 1, (1 << 20) - 1)) return 2;\n"
           "  if (product_choice::reaches(far, 64) || product_choice::reaches(64, far)) return 3;\n"
           "  for (bool t : {true, false}) {\n"
           "    if (!weight_choice::tiles_fit(t, 1, 4096, 4096, 4096, 4096, 2048, 4096)) return 4;\n"
           "    if (weight_choice::tiles_fit(t, 1, 4096, 4096, 4096, far, 2048, 4096)) return 5;\n"
           "    if (weight_choice::tiles_fit(t, 1, 4096, 4096, 4096, 4096, far, 4096)) return 6;\n"
           "    if (weight_choice::tiles_fit(t, 1, 4096, 4096, 4096, 4096, 2048, far)) return 7;\n"
           "    if (weight_choice::tiles_fit(t, 1 << 30, 4096, 4096, 4096, 4096, 2048, 4096)) return 8;\n"
           "  }\n  return 0; }\n")
    import tempfile

    with tempfile.TemporaryDirectory() as tmp:
        path = os.path.join(tmp, "far.cpp")
        with open(path, "w") as f:
            f.write(src)
        exe = os.path.join(tmp, "far")
        res = subprocess.run([shutil.which("g++"), "-std=c++17", "-I", CSRC, path, "-o", exe],
                             capture_output=True, text=True, timeout=120)
        assert res.returncode == 0, res.stderr
        assert subprocess.run([exe], timeout=60).returncode == 0
