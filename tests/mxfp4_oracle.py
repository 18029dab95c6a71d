"""Plain implementations of the MXFP4 operators in 64 bits (numpy), written
from the format's definition: the reference of the tests."""

from __future__ import annotations

import numpy as np

ELEMENTS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def blocks(n: int) -> int:
    return -(-n // 32)


def quantize(X: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """(codes, scales) of float32 X (..., rows, cols), blocks along the last axis."""
    cols = X.shape[-1]
    nb = blocks(cols)
    x = np.zeros((*X.shape[:-1], nb * 32))
    x[..., :cols] = X.astype(np.float64)
    x = x.reshape(*X.shape[:-1], nb, 32)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    amax = np.abs(x).max(-1)
    # frexp: amax = m 2^q with 0.5 <= m < 1, so floor(log2 amax) = q - 1
    q = np.frexp(np.where(amax > 0, amax, 1.0))[1].astype(np.int64)
    e = np.where(amax > 0, np.clip(q - 1 - 2, -127, 127), -127)
    v = np.ldexp(x, -e[..., None])
    m = np.abs(v)
    code = np.zeros(m.shape, np.int64)
    for i in range(7):  # past the middle of elements i and i + 1, or on it with i + 1 even
        mid = (ELEMENTS[i] + ELEMENTS[i + 1]) / 2
        code += (m > mid) | ((m == mid) & ((i + 1) % 2 == 0))
    code |= np.where(np.signbit(v), 8, 0)
    code = np.where(bad[..., None], 0, code).reshape(*X.shape[:-1], nb * 16, 2)
    codes = (code[..., 0] | code[..., 1] << 4).astype(np.uint8)
    scales = np.zeros((*X.shape[:-1], blocks(nb * 8) * 4), np.uint8)
    scales[..., :nb] = np.where(bad, 255, e + 127)
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray, cols: int) -> np.ndarray:
    """The float64 values (..., rows, cols) that codes and scales stand for."""
    nb = blocks(cols)
    c = codes[..., : nb * 16]
    nibble = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], nb, 32)
    v = np.where(nibble & 8, -1.0, 1.0) * ELEMENTS[nibble & 7]
    e = scales[..., :nb].astype(np.int64)
    with np.errstate(invalid="ignore"):
        v = np.ldexp(v, (e - 127)[..., None]) * np.where(e == 255, np.nan, 1.0)[..., None]
    return v.reshape(*c.shape[:-1], nb * 32)[..., :cols]


def random_matrix(rng, shape, cols, spread=4) -> tuple[np.ndarray, np.ndarray]:
    """Random codes and scales of a (*shape, cols) matrix, scales within
    2^+-spread, the columns past `cols` zero."""
    nb = blocks(cols)
    nibble = rng.integers(0, 16, (*shape, nb * 32))
    nibble[..., cols:] = 0
    pair = nibble.reshape(*shape, nb * 16, 2)
    codes = (pair[..., 0] | pair[..., 1] << 4).astype(np.uint8)
    scales = rng.integers(0, 256, (*shape, blocks(nb * 8) * 4)).astype(np.uint8)
    scales[..., :nb] = rng.integers(127 - spread, 128 + spread, (*shape, nb))
    return codes, scales
