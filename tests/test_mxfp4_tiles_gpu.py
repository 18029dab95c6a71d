"""The tile kernels of the MXFP4 products, at sizes that take them (see
tests/mxfp4_tile_cases.py), against float64 products on the GPU.

Every comparison is of equal values: operands are chosen so that each a * b,
and with that every partial sum in any order, is a multiple of some unit u and
the sum S of the magnitudes is below 2^24 u, so that no addition of at least 24
bits rounds.  Elements are multiples of 1/2; scales within 2^+-s make them
multiples of 2^-(1 + s).  S < 2^24 u is checked for every product.
"""

from __future__ import annotations

import numpy as np
import pytest

from dense_fp32_gemm_row_amd import binding as b
from tests import mxfp4_oracle as ref
from tests import mxfp4_tile_cases as cases
from tests.gpu_util import log, to_host

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
OPS = {"T": b.OP_T, "N": b.OP_N}
MEAN = {0: 2.25, 2: 3.49}  # of an element's magnitude times a scale within 2^+-s


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch

    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    b.load()
    yield
    torch.cuda.synchronize()


def power_of_two(n):
    """2^n in float64 for integers -127 <= n <= 127, exactly."""
    import torch

    return torch.tensor(2.0 ** np.arange(-127.0, 128.0), device=DEV)[(n + 127).long()]


def generator(seed):
    import torch

    return torch.Generator(device=DEV).manual_seed(seed)


class Matrix:
    """`batch` random matrices of the format on the GPU, the codes and scales
    inside wider rows whose other bytes are 0xff, scale bytes past the last
    block anything.  `exponents` (along the rows' axis, or None) are added to
    the scales' bytes of a row, `block_exponents` to those of a block."""

    def __init__(self, seed, batch, rows, cols, spread, exponents=None, block_exponents=None):
        import torch

        g = generator(seed)
        nb, words = ref.blocks(cols), ref.blocks(ref.blocks(cols) * 8) * 4
        codes = torch.randint(0, 256, (batch, rows, nb * 16), generator=g, device=DEV, dtype=torch.uint8)
        keep = (torch.arange(nb * 32, device=DEV) < cols).to(torch.uint8) * 15
        codes &= keep[0::2] | (keep[1::2] << 4)
        power = torch.randint(-spread, spread + 1, (batch, rows, nb), generator=g, device=DEV)
        scales = torch.randint(0, 256, (batch, rows, words), generator=g, device=DEV).to(torch.uint8)
        byte = power + 127
        if exponents is not None:
            byte = byte + exponents.view(1, -1, 1)
        if block_exponents is not None:
            byte = byte + block_exponents.view(1, 1, -1)
        assert int(byte.min()) >= 0 and int(byte.max()) <= 254
        scales[..., :nb] = byte.to(torch.uint8)
        self.cols, self.batch, self.rows = cols, batch, rows
        self._power, self._seed = power, seed
        self.codes, self.scales = self._wide(codes, 48), self._wide(scales, 12)

    @staticmethod
    def _wide(x, pad):
        import torch

        wide = torch.full((*x.shape[:-1], x.shape[-1] + pad), 255, dtype=torch.uint8, device=DEV)
        wide[..., : x.shape[-1]] = x
        return wide[..., : x.shape[-1]]

    def values(self, i):
        """Matrix i in float64, without the exponents that were added."""
        import torch

        c = self.codes[i]
        nib = torch.stack((c & 15, c >> 4), -1).view(self.rows, -1)[:, : self.cols].long()
        table = torch.tensor(np.concatenate([ref.ELEMENTS, -ref.ELEMENTS]), device=DEV)
        return table[nib] * power_of_two(self._power[i]).repeat_interleave(32, 1)[:, : self.cols]

    def held(self, batched):
        if batched:
            return b.Mxfp4(self.codes, self.scales, self.cols)
        return b.Mxfp4(self.codes[0], self.scales[0], self.cols)


class Guarded:
    """An output (batch, M, N) of rows `ldc` floats apart inside a buffer whose
    other cells have to stay as they are.  `lines`: rows are whole cache lines."""

    def __init__(self, batch, M, N, lines):
        import torch

        ldc = (N + 63) // 32 * 32 if lines else (N + 3) | 1
        self.buffer = torch.full((batch, M + 2, ldc), 77.0, device=DEV)
        at = (0, 0) if lines else (1, 1)
        self.where = (slice(None), slice(at[0], at[0] + M), slice(at[1], at[1] + N))
        self.out = self.buffer[self.where]

    def tensor(self, batched):
        return self.out if batched else self.out[0]

    def result(self):
        """What was written; the rest is checked."""
        import torch

        got = self.out.clone()
        self.out.fill_(77.0)
        torch.cuda.synchronize()
        assert bool((self.buffer == 77.0).all()), "write outside C"
        return got


class Workspace:
    """`need` bytes inside a buffer whose end has to stay as it is (None: no bytes needed)."""

    def __init__(self, need):
        import torch

        self.words = need // 4
        self.buffer = torch.full((self.words + 64,), 77.0, device=DEV)
        self.tensor = self.buffer[: self.words] if need else None

    def check(self):
        assert bool((self.buffer[self.words:] == 77.0).all()), "write outside the workspace"


def exact(got, pairs, limit, what):
    """got (batch, M, N) equals the products of `pairs` (a (M x K), w (K x N), float64)."""
    for i, (a, w) in enumerate(pairs):
        S = float((a.abs() @ w.abs()).max())
        assert S < limit, f"{what}: sums of {S} are not exact"
        bad = (got[i].double() != a @ w).nonzero()
        assert len(bad) == 0, f"{what}: product {i}, {len(bad)} cells differ, first at {bad[0].tolist()}"


def spread_for(K):
    """s of the scales of two operands in the format: their products are
    multiples of 2^-(2 + 2 s), the mean magnitude 6.9 (s = 1) or 12.1 (s = 2)."""
    return 2 if K <= 10000 else 1


# ---- both operands in the format -------------------------------------------------

def run_product(A, B, size, lines, what, batched):
    batch, M, N, K = size
    out = Guarded(batch, M, N, lines)
    work = Workspace(b.gemm_mxfp4_workspace_size(batch, M, N, K))
    b.gemm_mxfp4(A, B, out.tensor(batched), work.tensor)
    got = out.result()
    work.check()
    return got


@pytest.mark.parametrize("case", cases.products(), ids=cases.ident)
def test_product_tile(case):
    """Rows of C that are whole lines (streamed stores) and that are not, each
    written at their cells alone; the same without a workspace."""
    tile, size, slices = case
    batch, M, N, K = size
    log(f"product tile {case}")
    s = spread_for(K)
    A, B = Matrix(1, batch, M, K, s), Matrix(2, batch, N, K, s)
    many = batch > 1
    pairs = [(A.values(i), B.values(i).t().contiguous()) for i in range(batch)]
    for lines in (False, True):
        got = run_product(A.held(many), B.held(many), size, lines, f"lines={lines}", many)
        exact(got, pairs, 2.0 ** (22 - 2 * s), f"{case} lines={lines}")
    need = b.gemm_mxfp4_workspace_size(*size)
    assert need == (0 if slices == 1 else 4 * slices * batch * M * N)


@pytest.mark.parametrize("tile", sorted(cases.PRODUCTS))
def test_product_tile_of_one_matrix_in_a_batch(tile):
    """Batch stride 0 of either operand."""
    size = next(s for s in cases.PRODUCTS[tile] if s[0] >= 9)
    batch, M, N, K = size
    log(f"one matrix {size}")
    A, B = Matrix(3, batch, M, K, 2), Matrix(4, batch, N, K, 2)
    one_a = b.Mxfp4(A.codes[:1].expand(batch, -1, -1), A.scales[:1].expand(batch, -1, -1), K)
    one_b = b.Mxfp4(B.codes[:1].expand(batch, -1, -1), B.scales[:1].expand(batch, -1, -1), K)
    a, w = [A.values(i) for i in range(batch)], [B.values(i).t().contiguous() for i in range(batch)]
    got = run_product(one_a, B.held(True), size, False, "one A", True)
    exact(got, [(a[0], w[i]) for i in range(batch)], 2.0 ** 18, "one A")
    got = run_product(A.held(True), one_b, size, False, "one B", True)
    exact(got, [(a[i], w[0]) for i in range(batch)], 2.0 ** 18, "one B")


def few(table, n_blocks):
    """Of each form of a tile the first unsliced, unbatched size of some blocks."""
    seen = {}
    for size, slices in table.items():
        if slices == 1 and size[0] == 1 and size[3] >= 32 * n_blocks:
            seen.setdefault((size[3] % 4 == 0, size[3] % 512 == 0), size)
    return list(seen.values())


PRODUCT_FEW = [(tile, size) for tile, sizes in cases.PRODUCTS.items() for size in few(sizes, 8)]
WEIGHT_FEW = [(op, tile, size) for (op, tile), sizes in cases.WEIGHTS.items() for size in few(sizes, 3)]


@pytest.mark.parametrize("case", PRODUCT_FEW, ids=cases.ident)
def test_product_tile_nan_blocks(case):
    """A block of scale 255 makes its row (column) of C NaN, nothing else: in
    the first, a middle and the last block, in first and last rows."""
    import torch

    tile, size = case
    _, M, N, K = size
    log(f"NaN blocks {case}")
    A, B = Matrix(5, 1, M, K, 2), Matrix(6, 1, N, K, 2)
    last = ref.blocks(K) - 1
    rows, cols = {0: 0, M // 2: last // 2, M - 1: last}, {1: 0, N // 2 + 1: 3, N - 2: last}
    for m, j in rows.items():
        A.scales[0, m, j] = 255
    for n, j in cols.items():
        B.scales[0, n, j] = 255
    want = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    want[list(rows)] = True
    want[:, list(cols)] = True
    got = run_product(A.held(False), B.held(False), size, False, "", False)[0]
    assert torch.equal(got.isnan(), want)
    assert torch.equal(got[~want].double(), (A.values(0) @ B.values(0).t().contiguous())[~want])


@pytest.mark.parametrize("case", PRODUCT_FEW + [("rows", s) for k, s in cases.DIRECT if k == "P"], ids=cases.ident)
def test_product_far_exponents(case):
    """Scale bytes from 0 to 254, one operand's against the other's: values that
    FP32 does not hold, with products that it does."""
    tile, size = case
    _, M, N, K = size
    log(f"far exponents {case}")
    nb = ref.blocks(K)
    t = far_exponents(nb, 125)  # the random part of the scales moves a byte by 2 more
    A, B = Matrix(7, 1, M, K, 2, block_exponents=t), Matrix(8, 1, N, K, 2, block_exponents=-t)
    got = run_product(A.held(False), B.held(False), size, True, "", False)
    exact(got, [(A.values(0), B.values(0).t().contiguous())], 2.0 ** 18, str(case))


def far_exponents(n, most):
    import torch

    t = torch.randint(-most, most + 1, (n,), generator=generator(9), device=DEV)
    t[0], t[-1] = most, -most
    return t


# ---- A in FP32 ----------------------------------------------------------------------

def weight_matrix(op, seed, batch, N, K, spread, exponents=None):
    """W (N x K for op T, K x N for op N); `exponents` along k, of whole blocks for T."""
    if op == "T":
        return Matrix(seed, batch, N, K, spread, block_exponents=None if exponents is None else exponents[::32])
    return Matrix(seed, batch, K, N, spread, exponents=exponents)


def weight_values(op, W, i):
    """K x N, float64"""
    v = W.values(i)
    return v.t().contiguous() if op == "T" else v


def rows_of(x):
    """x (batch, M, K) inside wider rows of NaN, so that lda > K."""
    import torch

    wide = torch.full((*x.shape[:-1], x.shape[-1] + 3), float("nan"), device=DEV)
    wide[..., : x.shape[-1]] = x
    return wide[..., : x.shape[-1]]


def integers(seed, batch, M, K, spread):
    """Integers small enough for exact sums: products with W are multiples of
    2^-(1 + s), and S is about K times the means of both, here a quarter of 2^(23 - s)."""
    import torch

    most = max(1, min(4095, int(2.0 ** (22 - spread) / (K * MEAN[spread]))))
    return torch.randint(-most, most + 1, (batch, M, K), generator=generator(seed), device=DEV).float()


def run_weight(op, x, W, size, lines, batched):
    batch, M, N, K = size
    out = Guarded(batch, M, N, lines)
    work = Workspace(b.gemm_mxfp4_weight_workspace_size(OPS[op], *size))
    b.gemm_mxfp4_weight(x if batched else x[0], W, out.tensor(batched), work.tensor, op=OPS[op])
    got = out.result()
    work.check()
    return got


@pytest.mark.parametrize("case", cases.weights(), ids=cases.ident)
def test_weight_tile(case):
    op, tile, size, slices = case
    batch, M, N, K = size
    log(f"weight tile {case}")
    s = 2 if K <= 2200 else 0
    W, x = weight_matrix(op, 11, batch, N, K, s), integers(12, batch, M, K, s)
    X, many = rows_of(x), batch > 1
    pairs = [(x[i].double(), weight_values(op, W, i)) for i in range(batch)]
    for lines in (False, True):
        got = run_weight(op, X, W.held(many), size, lines, many)
        exact(got, pairs, 2.0 ** (23 - s), f"{case} lines={lines}")
    need = b.gemm_mxfp4_weight_workspace_size(OPS[op], *size)
    assert need == (0 if slices == 1 else 4 * slices * batch * M * N)


@pytest.mark.parametrize("case", cases.weights(), ids=cases.ident)
def test_weight_tile_keeps_every_bit_of_a(case):
    """One non-zero element of W, +-1, a column of C: the product picks values
    of A, which come back bit for bit (24-bit significands, tiny and huge
    ones), whatever the scales of the other blocks."""
    import torch

    op, tile, size, slices = case
    batch, M, N, K = size
    log(f"every bit {case}")
    g = generator(13)
    x = torch.randn(batch, M, K, generator=g, device=DEV) * torch.exp2(
        torch.randint(-80, 120, (batch, M, K), generator=g, device=DEV).float())
    W = weight_matrix(op, 14, batch, N, K, 2)
    W.codes.zero_()
    W.scales.copy_(torch.randint(0, 253, W.scales.shape, generator=g, device=DEV).to(torch.uint8))
    many = batch > 1
    k = torch.randint(0, K, (batch, N), generator=g, device=DEV)
    k[:, 0], k[:, -1] = K - 1, 0
    negative = torch.randint(0, 2, (batch, N), generator=g, device=DEV)
    n = torch.arange(N, device=DEV).expand(batch, N)
    i = torch.arange(batch, device=DEV)[:, None].expand(batch, N)
    row, col = (n, k) if op == "T" else (k, n)
    W.scales[i, row, col // 32] = 127
    element = (2 + 8 * negative).to(torch.uint8) << (4 * (col % 2)).to(torch.uint8)
    # (two columns of op N may share a byte: they are added, in different halves)
    flat = torch.zeros(W.codes.shape, dtype=torch.int32, device=DEV)
    flat.index_put_((i, row, col // 2), element.to(torch.int32), accumulate=True)
    W.codes.copy_(flat.to(torch.uint8))
    got = run_weight(op, rows_of(x), W.held(many), size, False, many)
    want = torch.gather(x, 2, k[:, None, :].expand(batch, M, N)) * (1.0 - 2.0 * negative)[:, None, :]
    bad = (got != want).nonzero()
    assert len(bad) == 0, f"{len(bad)} cells differ, first at {bad[0].tolist()}"


@pytest.mark.parametrize("case", WEIGHT_FEW, ids=cases.ident)
def test_weight_tile_infinities_and_nan(case):
    """Infinities and NaN of A reach their own rows of C alone, as in FP32."""
    import torch

    op, tile, size = case
    _, M, N, K = size
    log(f"infinities {case}")
    W, x = weight_matrix(op, 15, 1, N, K, 2), integers(16, 1, M, K, 2)
    x[0, 0, 3], x[0, 1, K // 2], x[0, 2, K - 1] = float("inf"), -float("inf"), float("nan")
    x[0, M - 1, 0], x[0, M - 1, 1] = float("inf"), -float("inf")
    x.view(torch.int32)[0, 5, 5] = 0x7F800001  # a NaN whose payload is its lowest bit
    rows = [0, 1, 2, 5, M - 1]
    got = run_weight(op, rows_of(x), W.held(False), size, False, False)[0]
    w64 = weight_values(op, W, 0)
    with np.errstate(invalid="ignore"):
        want = np.stack([(to_host(x[0, r]).astype(np.float64)[:, None] * to_host(w64)).sum(0) for r in rows])
    mine = to_host(got[rows]).astype(np.float64)
    assert np.array_equal(np.isnan(mine), np.isnan(want))
    odd = np.isinf(want)
    assert odd.any() and np.array_equal(mine[odd], want[odd])
    rest = torch.ones(M, dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert torch.equal(got[rest].double(), x[0, rest].double() @ w64)


@pytest.mark.parametrize("case", WEIGHT_FEW, ids=cases.ident)
def test_weight_tile_nan_blocks(case):
    """A block of scale 255 makes the columns of C that it reaches NaN, nothing else."""
    import torch

    op, tile, size = case
    _, M, N, K = size
    log(f"NaN blocks {case}")
    W, x = weight_matrix(op, 17, 1, N, K, 2), integers(18, 1, M, K, 2)
    want = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    if op == "T":
        for n, j in {0: 0, N // 2: 1, N - 1: ref.blocks(K) - 1}.items():
            W.scales[0, n, j] = 255
            want[:, n] = True
    else:
        for k, j in {0: 0, K // 2: 2, K - 1: ref.blocks(N) - 1}.items():
            W.scales[0, k, j] = 255
            want[:, 32 * j : 32 * j + 32] = True
    got = run_weight(op, rows_of(x), W.held(False), size, False, False)[0]
    assert torch.equal(got.isnan(), want)
    assert torch.equal(got[~want].double(), (x[0].double() @ weight_values(op, W, 0))[~want])


@pytest.mark.parametrize("case", WEIGHT_FEW + [(k, "direct", s) for k, s in cases.DIRECT if k != "P"],
                         ids=cases.ident)
def test_weight_far_exponents(case):
    """Scale bytes of W from 0 to 252 against A's exponents: an integer of A
    and an element of W times 2^-t and 2^t.  At the ends of the exponents the
    integers are +-1, so that A stays a finite FP32 value."""
    import torch

    op, tile, size = case
    _, M, N, K = size
    log(f"far exponents {case}")
    x = integers(19, 1, M, K, 0)
    if op == "T":
        t = far_exponents(ref.blocks(K), 125).repeat_interleave(32)[:K]
    else:
        t = far_exponents(K, 125)
    t = torch.where(t == -125, torch.full_like(t, -127), t)
    small = t < -110
    x = torch.where(small, torch.sign(x), x)
    W = weight_matrix(op, 20, 1, N, K, 0, exponents=t)
    X = (x.double() * power_of_two(-t)).float()  # exact: at most 12 bits, |t| <= 127
    assert bool((X.double() == x.double() * power_of_two(-t)).all()) and bool(X.isfinite().all())
    got = run_weight(op, rows_of(X), W.held(False), size, False, False)
    exact(got, [(x[0].double(), weight_values(op, W, 0))], 2.0 ** 23, str(case))


@pytest.mark.parametrize("op,tile", sorted(cases.WEIGHTS))
def test_weight_tile_of_one_matrix_in_a_batch(op, tile):
    """Batch stride 0 of either operand."""
    size = next(s for s, n in cases.WEIGHTS[op, tile].items() if s[0] > 1 and n == 1)
    batch, M, N, K = size
    log(f"one matrix {op} {tile} {size}")
    W, x = weight_matrix(op, 21, batch, N, K, 0), integers(22, batch, M, K, 0)
    one = b.Mxfp4(W.codes[:1].expand(batch, -1, -1), W.scales[:1].expand(batch, -1, -1), W.cols)
    w = [weight_values(op, W, i) for i in range(batch)]
    got = run_weight(op, rows_of(x), one, size, False, True)
    exact(got, [(x[i].double(), w[0]) for i in range(batch)], 2.0 ** 23, "one W")
    got = run_weight(op, x[:1].expand(batch, M, K), W.held(True), size, False, True)
    exact(got, [(x[0].double(), w[i]) for i in range(batch)], 2.0 ** 23, "one A")


# ---- the same call again, and from a graph ------------------------------------------

def test_tiles_in_a_graph():
    """A captured run of tile products (walking tiles, slices, both forms of
    W), replayed between eager runs, repeats them bit for bit."""
    import torch

    sizes = [(1, 4133, 4161, 1000), (1, 2815, 3525, 1292), (3, 646, 1678, 28794)]
    mats = [(Matrix(31, *(s[0], s[1], s[3]), 2).held(s[0] > 1), Matrix(32, *(s[0], s[2], s[3]), 2).held(s[0] > 1))
            for s in sizes]
    batch, M, N, K = 1, 2127, 2024, 512
    x = torch.randn(M, K, generator=generator(33), device=DEV)
    wt, wn = (weight_matrix(op, 34, 1, N, K, 4).held(False) for op in ("T", "N"))
    deep = weight_matrix("N", 35, 1, 129, 22528, 4).held(False)
    xd = torch.randn(346, 22528, generator=generator(36), device=DEV)

    def step():
        return [b.gemm_mxfp4(p, q) for p, q in mats] + [
            b.gemm_mxfp4_weight(x, wt), b.gemm_mxfp4_weight(x, wn, op=b.OP_N), b.gemm_mxfp4_weight(xd, deep, op=b.OP_N)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        x.copy_(torch.randn(M, K, generator=generator(40 + i), device=DEV))
        xd.copy_(torch.randn(346, 22528, generator=generator(50 + i), device=DEV))
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip([o.clone() for o in outs], step()):
            assert torch.equal(got, want), f"replay {i}"
