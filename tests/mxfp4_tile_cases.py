"""Sizes that the tile kernels of the MXFP4 products are tested at, with the
tile and the slices of K that each is meant to take: a CPU test compares both
with the library's choice, so that a change of its predictions cannot leave a
tile without tests."""

from __future__ import annotations

# (batch, M, N, K): ragged edges on every side, more tiles than the chip holds
# (a workgroup then walks on to another tile), K a multiple of 512 and not
PRODUCTS = {
    "256x256": {
        (1, 4278, 2263, 1536): 1,
        (20, 385, 1479, 1024): 1,
        (5, 970, 671, 38912): 4,
        (1, 2815, 3525, 1292): 1,
        (1, 5000, 5003, 4100): 1,
        (20, 148, 2699, 580): 1,
        (20, 500, 3000, 640): 1,
        (3, 646, 1678, 28794): 4,
    },
    "128x128": {
        (1, 300, 5046, 512): 1,
        (20, 500, 97, 512): 1,
        (2, 32, 45, 36352): 15,
        (1, 700, 2252, 500): 1,
        (1, 4133, 4161, 1000): 1,
        (9, 97, 944, 1000): 1,
        (1, 37, 33, 29556): 8,
    },
}

# K a multiple of 4 and not; a few blocks of K and many
WEIGHTS = {
    ("T", "128x256"): {
        (1, 4133, 2100, 516): 1,
        (20, 520, 530, 600): 1,
        (1, 5915, 1333, 36): 1,
        (1, 4215, 137, 3684): 8,
        (20, 82, 135, 5640): 15,
        (1, 4133, 2100, 515): 1,
        (20, 520, 530, 601): 1,
        (1, 1858, 4627, 34): 1,
        (1, 5527, 154, 2135): 6,
        (9, 75, 223, 15041): 30,
    },
    ("T", "64x256"): {
        (1, 2500, 2024, 700): 1,
        (9, 2289, 131, 100): 1,
        (1, 2088, 2472, 40): 1,
        (1, 346, 129, 22528): 59,
        (3, 67, 146, 19968): 52,
        (1, 700, 9000, 1569): 1,
        (1, 924, 5785, 39): 1,
        (20, 93, 1968, 38): 1,
        (1, 766, 135, 10941): 29,
        (3, 65, 193, 21846): 57,
    },
    ("T", "64x128"): {
        (1, 2127, 2024, 512): 1,
        (20, 148, 2699, 580): 1,
        (1, 970, 1414, 100): 1,
        (1, 784, 68, 9944): 26,
        (3, 114, 73, 9728): 26,
        (1, 2127, 2024, 515): 1,
        (9, 1446, 130, 69): 1,
        (1, 4181, 263, 35): 1,
        (1, 36, 2234, 11491): 30,
    },
    ("N", "128x256"): {
        (1, 4133, 2100, 516): 1,
        (20, 520, 530, 600): 1,
        (1, 5915, 1333, 36): 1,
        (1, 2088, 134, 4004): 16,
        (5, 72, 413, 8192): 32,
        (1, 4133, 2100, 515): 1,
        (20, 1954, 163, 33): 1,
        (1, 5527, 154, 2135): 6,
        (20, 78, 142, 6467): 13,
    },
    ("N", "64x256"): {
        (1, 2500, 2024, 700): 1,
        (1, 2127, 2024, 512): 1,
        (9, 2289, 131, 100): 1,
        (1, 346, 129, 22528): 59,
        (1, 2127, 2024, 515): 1,
        (1, 700, 9000, 1569): 1,
        (5, 3714, 133, 135): 1,
        (1, 766, 135, 10941): 29,
    },
    ("N", "64x128"): {
        (1, 970, 1414, 100): 1,
        (9, 1446, 130, 68): 1,
        (1, 5912, 231, 40): 1,
        (1, 784, 68, 9944): 26,
        (1, 970, 1414, 101): 1,
        (9, 1446, 130, 69): 1,
        (1, 4181, 263, 35): 1,
        (1, 296, 36, 23574): 62,
    },
}

# The kernels that read their operands straight from memory, at the sizes of
# the tests that tiles and they share: rows of A that share an instruction, and
# the one or two that take a kernel of multiply-adds.
DIRECT = [("P", (1, 40, 300, 1000)), ("T", (1, 1, 300, 1000)), ("T", (1, 2, 301, 2081)), ("T", (1, 7, 300, 1000)),
          ("T", (1, 16, 2001, 515)), ("T", (1, 33, 500, 777)), ("N", (1, 1, 300, 1000)), ("N", (1, 16, 2001, 515)),
          ("N", (1, 33, 500, 777))]


def products():
    """[(tile, (batch, M, N, K), slices)]"""
    return [(tile, size, n) for tile, sizes in PRODUCTS.items() for size, n in sizes.items()]


def weights():
    """[(op, tile, (batch, M, N, K), slices)]"""
    return [(op, tile, size, n) for (op, tile), sizes in WEIGHTS.items() for size, n in sizes.items()]


def ident(case):
    return "-".join("x".join(map(str, c)) if isinstance(c, tuple) else str(c) for c in case)
