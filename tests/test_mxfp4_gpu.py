"""The MXFP4 operators on the GPU against plain implementations in 64 bits.

Conversions are compared byte for byte.  Products: every a * b is exact in
FP32 (for an FP32 operand, each of its three parts times an element is); the
matrix cores add at most 16 of them, and the running sum, per rounding, and
a rounding loses less than a unit in the last place, 2^-23, of a value that
is at most S = sum |a b|.  With P products (K, or 3 K) an error is below
(P / 16 + 8) 2^-23 S, the 8 for adding slices of K.  Sums of elements under
equal scales are multiples of 1/4 below 2^22 and have to be exact.
"""

from __future__ import annotations

import threading

import numpy as np
import pytest

from dense_fp32_gemm_row_amd import binding as b
from tests import mxfp4_oracle as ref
from tests.gpu_util import log, to_dev, to_host

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def gpu():
    import torch

    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    b.load()
    yield
    torch.cuda.synchronize()


def held(codes, scales, cols, pad_q=0, pad_s=0):
    """An Mxfp4 on the GPU; with padding, inside rows whose other bytes are 0xff."""
    import torch

    def put(x, pad):
        if not pad:
            return to_dev(x)
        wide = torch.full((*x.shape[:-1], x.shape[-1] + pad), 255, dtype=torch.uint8, device="cuda:0")
        wide[..., : x.shape[-1]] = to_dev(x)
        return wide[..., : x.shape[-1]]

    return b.Mxfp4(put(codes, pad_q), put(scales, pad_s), cols)


def check_product(got, a64, w64, K, parts=1, what=""):
    """got (M x N) against a64 (M x K) @ w64 (N x K)^T within the derived bound."""
    want = a64 @ np.swapaxes(w64, -1, -2)
    S = np.abs(a64) @ np.swapaxes(np.abs(w64), -1, -2)
    bound = (parts * K / 16 + 8) * ULP * S
    err = np.abs(got.astype(np.float64) - want)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    worst = np.unravel_index(np.argmax(err - bound), err.shape) if err.size else None
    assert (err <= bound).all(), f"{what}: at {worst} {got[worst]} vs {want[worst]}, bound {bound[worst]:.3g}"


def inputs(rng, rows, cols, kind):
    if kind == "normal":
        x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal(cols))
    elif kind == "wide":  # every exponent, subnormals and zeros among them
        x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-150, 126, (rows, cols))
        x[rng.random((rows, cols)) < 0.1] = 0.0
    elif kind == "ties":  # multiples of 1/8: ties at every border
        x = rng.integers(-64, 65, (rows, cols)) / 8.0
    elif kind == "tiny":  # blocks of subnormals alone
        x = rng.integers(-40, 41, (rows, cols)) * 2.0 ** -149
    else:
        x = np.zeros((rows, cols))
        x[rng.random((rows, cols)) < 0.5] = -0.0
    return x.astype(np.float32)


# ---- conversions ---------------------------------------------------------------

SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (3, 64), (5, 127), (2, 128), (7, 129), (33, 777),
          (40, 1024), (31, 1100), (32, 4), (65, 300), (257, 2049), (1000, 1)]


def quantize_guarded(X, both):
    """Quantises X into matrices with guard bytes around every row; returns
    [(codes, scales)] and checks the guards."""
    import torch

    rows, cols = X.shape
    out, guards = [], []
    for r, c in ((rows, cols), (cols, rows)):
        nb, w = ref.blocks(c), ref.blocks(ref.blocks(c) * 8) * 4
        q = torch.full((r + 2, nb * 16 + 32), 0xAB, dtype=torch.uint8, device="cuda:0")
        s = torch.full((r + 2, w + 8), 0xCD, dtype=torch.uint8, device="cuda:0")
        out.append(b.Mxfp4(q[1:-1, 16:-16], s[1:-1, 4:-4], c))
        guards.append((q, s))
    if both == "both":
        b.mxfp4_quantize_both(X, out[0], out[1])
    elif both == "rows":
        b.mxfp4_quantize(X, out[0])
    else:
        b.mxfp4_quantize(X.T, out[1])
    res = []
    for i, ((q, s), o) in enumerate(zip(guards, out)):
        if (both, i) in (("rows", 1), ("cols", 0)):
            assert (to_host(q) == 0xAB).all() and (to_host(s) == 0xCD).all()
            res.append(None)
            continue
        res.append((to_host(o.codes).copy(), to_host(o.scales).copy()))
        o.codes[...] = 0xAB
        o.scales[...] = 0xCD
        assert (to_host(q) == 0xAB).all(), "write outside the codes"
        assert (to_host(s) == 0xCD).all(), "write outside the scales"
    return res


@pytest.mark.parametrize("kind", ["normal", "wide", "ties", "tiny", "zeros"])
@pytest.mark.parametrize("form", ["rows", "cols", "both"])
def test_quantize(form, kind):
    rng = np.random.default_rng(len(form) * 7 + len(kind))
    for rows, cols in SHAPES:
        log(f"quantize {form} {kind} {rows}x{cols}")
        x = inputs(rng, rows, cols, kind)
        # rows of X at an odd stride and offset
        buf = to_dev(np.full((rows, cols + 3), np.nan, np.float32))
        X = buf[:, 1 : 1 + cols]
        X.copy_(to_dev(x))
        got = quantize_guarded(X, form)
        for g, want in zip(got, (ref.quantize(x), ref.quantize(np.ascontiguousarray(x.T)))):
            if g is not None:
                assert np.array_equal(g[1], want[1]), "scales"
                assert np.array_equal(g[0], want[0]), "codes"


@pytest.mark.parametrize("form", ["rows", "cols", "both"])
def test_quantize_not_finite(form):
    rng = np.random.default_rng(8)
    x = rng.standard_normal((70, 100)).astype(np.float32)
    x[3, 40] = np.inf
    x[5, 99] = -np.inf
    x[40, 0] = np.nan
    x[69, 31:33] = np.nan
    x.view(np.uint32)[50, 50] = 0x7F800001  # a NaN whose payload is its lowest bit
    got = quantize_guarded(to_dev(x), form)
    for g, want in zip(got, (ref.quantize(x), ref.quantize(np.ascontiguousarray(x.T)))):
        if g is not None:
            assert np.array_equal(g[1], want[1]) and np.array_equal(g[0], want[0])
            assert (g[1] == 255).sum() >= 5


def test_quantize_batched_and_views():
    import torch

    rng = np.random.default_rng(9)
    x = rng.standard_normal((3, 50, 71)).astype(np.float32)
    X = to_dev(np.pad(x, ((0, 0), (0, 2), (0, 1))))[:, :50, :71]
    q, qt = b.mxfp4_quantize_both(X)
    for got, want in ((q, ref.quantize(x)), (qt, ref.quantize(np.ascontiguousarray(x.swapaxes(1, 2)))),
                      (b.mxfp4_quantize(X.transpose(1, 2)), ref.quantize(np.ascontiguousarray(x.swapaxes(1, 2)))),
                      (b.mxfp4_quantize_both(X.transpose(1, 2))[1], ref.quantize(x)),
                      (b.mxfp4_quantize(X[1:2].expand(3, 50, 71)), ref.quantize(np.repeat(x[1:2], 3, 0)))):
        assert np.array_equal(to_host(got.codes), want[0])
        assert np.array_equal(to_host(got.scales), want[1])
    assert q.shape == (3, 50, 71) and qt.shape == (3, 71, 50)
    for shape in ((0, 40), (40, 0), (2, 0, 40), (0, 4, 40)):
        q, qt = b.mxfp4_quantize_both(torch.empty(shape, device="cuda:0"))
        assert q.shape == shape and b.mxfp4_dequantize(q).shape == shape


def test_dequantize_every_code_and_scale():
    nib = np.tile(np.arange(16), 2)
    codes = np.tile((nib[0::2] | nib[1::2] << 4).astype(np.uint8), (256, 1))
    scales = np.zeros((256, 4), np.uint8)
    scales[:, 0] = np.arange(256)
    got = to_host(b.mxfp4_dequantize(held(codes, scales, 32, 16, 4)))
    with np.errstate(over="ignore"):
        want = ref.values(codes, scales, 32).astype(np.float32)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(np.signbit(got[:255]), np.signbit(want[:255]))


@pytest.mark.parametrize("shape", SHAPES)
def test_dequantize(shape):
    import torch

    rng = np.random.default_rng(sum(shape))
    rows, cols = shape
    log(f"dequantize {shape}")
    c, s = ref.random_matrix(rng, (rows,), cols, 60)
    buf = torch.full((rows + 2, cols + 2), 7.0, device="cuda:0")
    b.mxfp4_dequantize(held(c, s, cols, 32, 4), buf[1:-1, 1:-1])
    got = to_host(buf)
    assert np.array_equal(got[1:-1, 1:-1], ref.values(c, s, cols).astype(np.float32))
    got[1:-1, 1:-1] = 7.0
    assert (got == 7.0).all(), "write outside Y"
    c3, s3 = np.stack([c, c]), np.stack([s, s])
    assert np.array_equal(to_host(b.mxfp4_dequantize(held(c3, s3, cols))),
                          ref.values(c3, s3, cols).astype(np.float32))


# ---- products --------------------------------------------------------------------

PRODUCTS = [(1, 1, 1), (1, 1, 33), (1, 32, 64), (2, 5, 31), (16, 16, 128), (17, 33, 160), (1, 300, 777),
            (3, 1000, 2080), (31, 64, 100), (33, 31, 95), (37, 130, 515), (64, 70, 1056), (100, 129, 300),
            (129, 255, 257), (256, 256, 256), (300, 277, 1029), (511, 40, 700), (260, 520, 2048),
            (64, 96, 8192), (1, 64, 16400)]


def product_out(M, N, call):
    """Runs call(out) on an `out` inside guard cells at an odd stride."""
    import torch

    buf = torch.full((M + 2, N + 3), float("nan"), device="cuda:0")
    call(buf[1:-1, 1:-2])
    got = to_host(buf)
    inner = got[1:-1, 1:-2].copy()
    got[1:-1, 1:-2] = np.nan
    assert np.isnan(got).all(), "write outside C"
    return inner


@pytest.mark.parametrize("shape", PRODUCTS)
def test_product(shape):
    M, N, K = shape
    log(f"product {shape}")
    rng = np.random.default_rng(M + N + K)
    a, w = ref.random_matrix(rng, (M,), K), ref.random_matrix(rng, (N,), K)
    A, W = held(*a, K, 48, 8), held(*w, K, 16, 4)
    got = product_out(M, N, lambda out: b.gemm_mxfp4(A, W, out))
    check_product(got, ref.values(*a, K), ref.values(*w, K), K, 1, str(shape))
    for s in (a[1], w[1]):
        s[...] = 125
    got = to_host(b.gemm_mxfp4(held(*a, K), held(*w, K)))
    assert np.array_equal(got, ref.values(*a, K) @ ref.values(*w, K).T), "equal scales: exact"


def wide_floats(rng, rows, cols):
    """24 significant bits, magnitudes over 2^+-12."""
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-12, 13, (rows, cols))
    return x.astype(np.float32)


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("shape", PRODUCTS)
def test_weight_product(shape, op):
    M, N, K = shape
    log(f"weight product {op} {shape}")
    rng = np.random.default_rng(M + N + K + 1)
    x = wide_floats(rng, M, K)
    buf = to_dev(np.full((M, K + 1), np.nan, np.float32))
    buf[:, :K] = to_dev(x)
    w = ref.random_matrix(rng, (N,), K) if op == "T" else ref.random_matrix(rng, (K,), N)
    w64 = ref.values(*w, K) if op == "T" else ref.values(*w, N).T
    W = held(*w, K if op == "T" else N, 16, 4)
    code = b.OP_T if op == "T" else b.OP_N
    got = product_out(M, N, lambda out: b.gemm_mxfp4_weight(buf[:, :K], W, out, op=code))
    check_product(got, x.astype(np.float64), w64, K, 3, f"{op} {shape}")
    x = rng.integers(-64, 65, (M, K)).astype(np.float32)
    w[1][...] = 127
    w64 = ref.values(*w, K) if op == "T" else ref.values(*w, N).T
    got = to_host(b.gemm_mxfp4_weight(to_dev(x), held(*w, K if op == "T" else N), op=code))
    assert np.array_equal(got, x.astype(np.float64) @ w64.T), "integers: exact"


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_weight_product_keeps_every_bit_of_a(op, M):
    """One non-zero element of W, 1, per output column: the product picks
    values of A, which come back bit for bit (24-bit significands, tiny and
    huge ones)."""
    rng = np.random.default_rng(M)
    K = N = 96
    x = (rng.standard_normal((M, K)) * 2.0 ** rng.integers(-100, 120, (M, K))).astype(np.float32)
    perm = rng.permutation(K)
    eye = np.zeros((N, K), np.float32)
    eye[np.arange(N), perm] = 1.0
    q = ref.quantize(eye if op == "T" else np.ascontiguousarray(eye.T))
    got = to_host(b.gemm_mxfp4_weight(to_dev(x), held(*q, 96), op=b.OP_T if op == "T" else b.OP_N))
    assert np.array_equal(got, x[:, perm])


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("M", [3, 70, 200])
def test_weight_product_infinities_and_nan(op, M):
    """Infinities and NaN of A reach their own rows of C alone, as in FP32."""
    rng = np.random.default_rng(M)
    K, N = 160, 64
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[0, 3], x[1, 100], x[2, 159] = np.inf, -np.inf, np.nan
    if M > 3:
        x[M - 1, 0], x[M - 1, 1] = np.inf, -np.inf
        x.view(np.uint32)[5, 5] = 0x7F800001
    w = ref.quantize(rng.standard_normal((N, K) if op == "T" else (K, N)).astype(np.float32))
    w64 = ref.values(*w, K) if op == "T" else ref.values(*w, N).T
    with np.errstate(invalid="ignore"):
        want = (x[:, None, :].astype(np.float64) * w64[None]).sum(-1)
    got = to_host(b.gemm_mxfp4_weight(to_dev(x), held(*w, K if op == "T" else N),
                                      op=b.OP_T if op == "T" else b.OP_N))
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isinf(got), np.isinf(want))
    m = ~np.isfinite(want) & ~np.isnan(want)
    assert np.array_equal(np.sign(got[m]), np.sign(want[m]))


@pytest.mark.parametrize("shape", [(3, 40, 200), (80, 300, 1000), (300, 280, 500)])
def test_nan_blocks(shape):
    """A block of scale 255 makes its row (column) of C NaN, nothing else."""
    M, N, K = shape
    rng = np.random.default_rng(11)
    a, w = ref.random_matrix(rng, (M,), K), ref.random_matrix(rng, (N,), K)
    a[1][M - 1, ref.blocks(K) - 1] = 255
    w[1][7, 2] = 255
    want = np.zeros((M, N), bool)
    want[M - 1] = want[:, 7] = True
    assert np.array_equal(np.isnan(to_host(b.gemm_mxfp4(held(*a, K), held(*w, K)))), want)
    want[M - 1] = False
    want[:, 7] = True
    x = to_dev(wide_floats(rng, M, K))
    assert np.array_equal(np.isnan(to_host(b.gemm_mxfp4_weight(x, held(*w, K)))), want)
    wn = ref.random_matrix(rng, (K,), N)
    wn[1][5, 1] = 255
    want[...] = False
    want[:, 32:64] = True
    assert np.array_equal(np.isnan(to_host(b.gemm_mxfp4_weight(x, held(*wn, N), op=b.OP_N))), want[:, :N])


def test_empty_sum_and_empty_products():
    import torch

    a = b.mxfp4_empty((5, 0), "cuda:0")
    w = b.mxfp4_empty((7, 0), "cuda:0")
    out = torch.full((5, 7), 3.0, device="cuda:0")
    assert (to_host(b.gemm_mxfp4(a, w, out)) == 0).all()
    out.fill_(3.0)
    assert (to_host(b.gemm_mxfp4_weight(torch.empty(5, 0, device="cuda:0"), w, out)) == 0).all()
    wn = b.mxfp4_empty((0, 7), "cuda:0")
    out.fill_(3.0)
    assert (to_host(b.gemm_mxfp4_weight(torch.empty(5, 0, device="cuda:0"), wn, out, op=b.OP_N)) == 0).all()
    assert b.gemm_mxfp4(b.mxfp4_empty((0, 64), "cuda:0"), b.mxfp4_empty((7, 64), "cuda:0")).shape == (0, 7)


@pytest.mark.parametrize("shape", [(4, 1, 100, 96), (3, 40, 70, 161), (5, 256, 300, 512), (2, 300, 130, 640)])
def test_batches(shape):
    nb, M, N, K = shape
    log(f"batch {shape}")
    rng = np.random.default_rng(nb)
    a, w = ref.random_matrix(rng, (nb, M), K), ref.random_matrix(rng, (nb, N), K)
    A, W = held(*a, K, 16, 4), held(*w, K)
    a64, w64 = ref.values(*a, K), ref.values(*w, K)
    check_product(to_host(b.gemm_mxfp4(A, W)), a64, w64, K, 1, "batch")
    one = b.Mxfp4(W.codes[1:2].expand(nb, -1, -1), W.scales[1:2].expand(nb, -1, -1), K)
    check_product(to_host(b.gemm_mxfp4(A, one)), a64, np.repeat(w64[1:2], nb, 0), K, 1, "one W")
    x = wide_floats(rng, nb * M, K).reshape(nb, M, K)
    X = to_dev(x)
    check_product(to_host(b.gemm_mxfp4_weight(X, W)), x.astype(np.float64), w64, K, 3, "weight")
    check_product(to_host(b.gemm_mxfp4_weight(X[:1].expand(nb, M, K), W)),
                  np.repeat(x[:1], nb, 0).astype(np.float64), w64, K, 3, "one X")
    wn = ref.random_matrix(rng, (nb, K), N)
    check_product(to_host(b.gemm_mxfp4_weight(X, held(*wn, N), op=b.OP_N)), x.astype(np.float64),
                  ref.values(*wn, N).swapaxes(1, 2), K, 3, "weight N")


DEEP = [(40, 50, 20000), (128, 256, 33000), (300, 200, 65536)]


@pytest.mark.parametrize("shape", DEEP)
def test_long_sums_with_and_without_workspace(shape):
    import torch

    M, N, K = shape
    log(f"long sums {shape}")
    rng = np.random.default_rng(K)
    a, w = ref.random_matrix(rng, (M,), K), ref.random_matrix(rng, (N,), K)
    A, W = held(*a, K), held(*w, K)
    a64, w64 = ref.values(*a, K), ref.values(*w, K)
    x = wide_floats(rng, M, K)
    X = to_dev(x)
    wn = ref.random_matrix(rng, (K,), N)
    Wn, wn64 = held(*wn, N), ref.values(*wn, N).T
    for none in (False, True):
        def run(call, size, *args):
            if not none:
                return call(None)
            out = torch.empty(M, N, device="cuda:0")
            assert args[0](out.data_ptr()) == 0
            return out
        sp = torch.cuda.current_stream().cuda_stream
        got = run(lambda _: b.gemm_mxfp4(A, W), 0, lambda o: b.gemm_mxfp4_product(
            1, M, N, K, A._c, W._c, o, N, 0, stream=sp))
        check_product(to_host(got), a64, w64, K, 1, f"none={none}")
        got = run(lambda _: b.gemm_mxfp4_weight(X, W), 0, lambda o: b.gemm_mxfp4_weight_product(
            b.OP_T, 1, M, N, K, X.data_ptr(), K, 0, W._c, o, N, 0, stream=sp))
        check_product(to_host(got), x.astype(np.float64), w64, K, 3, f"T none={none}")
        got = run(lambda _: b.gemm_mxfp4_weight(X, Wn, op=b.OP_N), 0, lambda o: b.gemm_mxfp4_weight_product(
            b.OP_N, 1, M, N, K, X.data_ptr(), K, 0, Wn._c, o, N, 0, stream=sp))
        check_product(to_host(got), x.astype(np.float64), wn64, K, 3, f"N none={none}")
    need = b.gemm_mxfp4_workspace_size(1, M, N, K)
    if need:
        with pytest.raises(b.GemmError):
            b.gemm_mxfp4(A, W, workspace=torch.empty(need - 4, dtype=torch.uint8, device="cuda:0"))
        out = torch.empty(need // 4 + M * N, device="cuda:0")
        with pytest.raises(b.GemmError):
            b.gemm_mxfp4(A, W, out[:M * N].view(M, N), workspace=out)


FEW = [(1, 3, 300, 8250), (1, 16, 40, 20001), (1, 5, 1000, 8200), (1, 13, 3500, 8192), (2, 9, 130, 12000),
       (1, 2, 77, 9000), (1, 16, 2000, 4096)]


@pytest.mark.parametrize("op", ["T", "N"])
@pytest.mark.parametrize("shape", FEW)
def test_few_rows_with_and_without_workspace(shape, op):
    import torch

    batch, M, N, K = shape
    rng = np.random.default_rng(K + N)
    rows, cols = (N, K) if op == "T" else (K, N)
    w = ref.random_matrix(rng, (batch, rows), cols)
    w64 = ref.values(*w, cols)
    w64 = w64 if op == "T" else np.swapaxes(w64, -1, -2)
    x = np.stack([wide_floats(rng, M, K) for _ in range(batch)])
    X, W, code = to_dev(x), held(*w, cols), b.OP_T if op == "T" else b.OP_N
    need = b.gemm_mxfp4_weight_workspace_size(code, batch, M, N, K)
    for work in {0, need}:
        out = torch.full((batch, M + 1, N + 3), 7.0, device="cuda:0")
        ws = torch.full((work // 4 + 8,), 7.0, device="cuda:0")
        assert b.gemm_mxfp4_weight_product(code, batch, M, N, K, X.data_ptr(), K, M * K, W._c, out.data_ptr(), N + 3,
                                           (M + 1) * (N + 3), ws.data_ptr() if work else None, work) == 0
        torch.cuda.synchronize()
        check_product(to_host(out[:, :M, :N]), x.astype(np.float64), w64, K, 3, f"workspace {work}")
        assert (out[:, M:] == 7.0).all() and (out[:, :, N:] == 7.0).all() and (ws[work // 4:] == 7.0).all()


def test_far_rows():
    """Rows of codes, of X and of C that lie more than 2^32 bytes apart."""
    import torch

    rng = np.random.default_rng(12)
    M, N, K = 5, 70, 200
    ld = (1 << 30) + 16
    a, w = ref.random_matrix(rng, (M,), K), ref.random_matrix(rng, (N,), K)
    far = torch.empty(M * ld, dtype=torch.uint8, device="cuda:0")
    codes = far.as_strided((M, a[0].shape[1]), (ld, 1))
    scales = far.as_strided((M, a[1].shape[1]), (ld, 1), 1024)
    codes.copy_(to_dev(a[0]))
    scales.copy_(to_dev(a[1]))
    A = b.Mxfp4(codes, scales, K)
    a64, w64 = ref.values(*a, K), ref.values(*w, K)
    check_product(to_host(b.gemm_mxfp4(A, held(*w, K))), a64, w64, K)
    check_product(to_host(b.gemm_mxfp4(held(*w, K), A)), w64, a64, K)
    assert np.array_equal(to_host(b.mxfp4_dequantize(A)), a64.astype(np.float32))
    xl = to_dev(wide_floats(rng, 3, K))
    check_product(to_host(b.gemm_mxfp4_weight(xl, A)), to_host(xl).astype(np.float64), a64, K, 3)
    x5 = to_dev(wide_floats(rng, 3, M))
    check_product(to_host(b.gemm_mxfp4_weight(x5, A, op=b.OP_N)), to_host(x5).astype(np.float64), a64.T, M, 3)
    del A, codes, scales, far
    fl = torch.empty(M * (1 << 28), device="cuda:0")
    X = fl.as_strided((M, K), (1 << 28, 1))
    x = wide_floats(rng, M, K)
    X.copy_(to_dev(x))
    W = held(*w, K)
    check_product(to_host(b.gemm_mxfp4_weight(X, W)), x.astype(np.float64), w64, K, 3)
    q, qt = b.mxfp4_quantize_both(X)
    assert np.array_equal(to_host(q.codes), ref.quantize(x)[0])
    assert np.array_equal(to_host(qt.codes), ref.quantize(np.ascontiguousarray(x.T))[0])
    out = fl.as_strided((M, N), (1 << 28, 1), 4096)
    b.gemm_mxfp4_weight(to_dev(x), W, out)
    check_product(to_host(out), x.astype(np.float64), w64, K, 3)


@pytest.mark.parametrize("op", ["T", "N"])
def test_tile_sized_products_of_far_rows(op):
    """Rows of W too far apart for a tile's 32-bit offsets, in a product that tiles would take."""
    import torch

    rng = np.random.default_rng(17)
    M, N, K = 3000, 300, 2000
    rows, cols = (N, K) if op == "T" else (K, N)
    ld = ((1 << 31) // (256 if op == "T" else K) + 4095) // 16 * 16
    w = ref.random_matrix(rng, (rows,), cols)
    far = torch.empty(rows * ld, dtype=torch.uint8, device="cuda:0")
    codes = far.as_strided((rows, w[0].shape[1]), (ld, 1))
    scales = far.as_strided((rows, w[1].shape[1]), (ld, 1), 2048)
    codes.copy_(to_dev(w[0]))
    scales.copy_(to_dev(w[1]))
    w64 = ref.values(*w, cols)
    x = wide_floats(rng, M, K)
    got = b.gemm_mxfp4_weight(to_dev(x), b.Mxfp4(codes, scales, cols), op=b.OP_T if op == "T" else b.OP_N)
    check_product(to_host(got), x.astype(np.float64), w64 if op == "T" else w64.T, K, 3)


@pytest.mark.parametrize("op", ["T", "N"])
def test_one_row_at_the_longest_stride(op):
    """A lone row's stride is never stepped over, however long it is."""
    import torch

    rng = np.random.default_rng(13)
    M, N, K, far = 1, 70, 200, 1 << 57
    w = ref.random_matrix(rng, (N,) if op == "T" else (K,), K if op == "T" else N)
    w64 = ref.values(*w, K if op == "T" else N)
    x = wide_floats(rng, M, K)
    X, W = to_dev(x), held(*w, K if op == "T" else N)
    out = torch.full((3, N), 7.0, device="cuda:0")
    wc = b.Mxfp4Matrix(W.codes.data_ptr(), W.codes.stride(0), 0, W.scales.data_ptr(), W.scales.stride(0), 0)
    rc = b.gemm_mxfp4_weight_product(b.OP_T if op == "T" else b.OP_N, 1, M, N, K, X.data_ptr(), far, 0, wc,
                                     out.data_ptr(), far, 0)
    assert rc == 0
    torch.cuda.synchronize()
    check_product(to_host(out[:1]), x.astype(np.float64), w64 if op == "T" else w64.T, K, 3)
    assert (out[1:] == 7.0).all()
    if op == "N":
        return
    q = b.mxfp4_empty((3, K))
    q.codes.fill_(9)
    q.scales.fill_(9)
    qc = b.Mxfp4Matrix(q.codes.data_ptr(), far, 0, q.scales.data_ptr(), far, 0)
    back = torch.full((3, K), 7.0, device="cuda:0")
    assert b.gemm_mxfp4_quantize(1, 1, K, X.data_ptr(), far, 0, qc, None) == 0
    assert b.gemm_mxfp4_dequantize(1, 1, K, qc, back.data_ptr(), far, 0) == 0
    assert b.gemm_mxfp4_product(1, 1, N, K, qc, wc, out.data_ptr(), far, 0) == 0
    torch.cuda.synchronize()
    codes, scales = ref.quantize(x)
    assert np.array_equal(to_host(q.codes[:1, : codes.shape[1]]), codes)
    assert (q.codes[1:] == 9).all() and (q.scales[1:] == 9).all()
    x64 = ref.values(codes, scales, K)
    assert np.array_equal(to_host(back[:1]), x64.astype(np.float32)) and (back[1:] == 7.0).all()
    check_product(to_host(out[:1]), x64, w64, K)
    assert (out[1:] == 7.0).all()


# ---- refusals of the tensor calls ---------------------------------------------------

def test_tensor_refusals():
    import torch

    dev = "cuda:0"
    A, W = b.mxfp4_empty((4, 64), dev), b.mxfp4_empty((6, 64), dev)
    x = torch.zeros(4, 64, device=dev)
    with pytest.raises(ValueError, match="shape mismatch"):
        b.gemm_mxfp4(A, b.mxfp4_empty((6, 96), dev))
    with pytest.raises(ValueError, match="shape mismatch"):
        b.gemm_mxfp4_weight(x, b.mxfp4_empty((6, 96), dev))
    with pytest.raises(ValueError, match="shape mismatch"):
        b.gemm_mxfp4_weight(x, W, op=b.OP_N)
    with pytest.raises(ValueError, match="op must"):
        b.gemm_mxfp4_weight(x, W, op=7)
    with pytest.raises(ValueError, match="row-major"):
        b.gemm_mxfp4_weight(torch.zeros(64, 4, device=dev).T, W)
    with pytest.raises(TypeError):
        b.gemm_mxfp4_weight(x.half(), W)
    with pytest.raises(ValueError, match="out has shape"):
        b.gemm_mxfp4(A, W, torch.empty(6, 4, device=dev))
    with pytest.raises(ValueError, match="row-major"):
        b.gemm_mxfp4(A, W, torch.empty(6, 4, device=dev).T)
    with pytest.raises(ValueError, match="expected shape"):
        b.mxfp4_quantize(x, b.mxfp4_empty((4, 32), dev))
    with pytest.raises(ValueError, match="row-major or a transposed"):
        b.mxfp4_quantize(torch.zeros(4, 64, 2, device=dev)[..., 0])
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8, device=dev), torch.zeros(4, 4, dtype=torch.uint8, device=dev)
    for c, s, cols in ((codes, scales, 65), (codes[:, ::2], scales, 32), (codes, scales[:3], 64),
                       (codes, scales[:, :2], 64), (codes[0], scales[0], 64)):
        with pytest.raises(ValueError):
            b.Mxfp4(c, s, cols)
    with pytest.raises(TypeError):
        b.Mxfp4(codes.float(), scales, 64)
    shifted = torch.zeros(4 * 32 + 8, dtype=torch.uint8, device=dev)[8:].view(4, 32)
    with pytest.raises(b.GemmError, match="multiples of 16"):
        b.gemm_mxfp4(b.Mxfp4(shifted, scales, 64), W)
    with pytest.raises(b.GemmError, match="overlap"):
        buf = torch.zeros(4096, device=dev)
        b.gemm_mxfp4_weight(buf[:256].view(4, 64), W, buf[128:152].view(4, 6))
    with pytest.raises(b.GemmError, match="overlap"):  # every product of the batch into one C
        nb = b.mxfp4_empty((3, 4, 64), dev)
        b.gemm_mxfp4(nb, nb, torch.empty(1, 4, 4, device=dev).expand(3, 4, 4))


# ---- a run of them together ------------------------------------------------------------

def linear_step(X, W, dY):
    x, xt = b.mxfp4_quantize_both(X)
    w, wt = b.mxfp4_quantize_both(W)
    dy, dyt = b.mxfp4_quantize_both(dY)
    return b.gemm_mxfp4(x, w), b.gemm_mxfp4(dy, wt), b.gemm_mxfp4(dyt, xt)


def rounded(x):
    q = ref.quantize(np.ascontiguousarray(x))
    return ref.values(*q, x.shape[1])


@pytest.mark.parametrize("shape", [(33, 65, 97), (200, 320, 256), (515, 129, 300)])
def test_linear_step(shape):
    M, N, K = shape
    rng = np.random.default_rng(13)
    x, w, dy = (rng.standard_normal(s).astype(np.float32) for s in ((M, K), (N, K), (M, N)))
    y, dx, dw = (to_host(t) for t in linear_step(to_dev(x), to_dev(w), to_dev(dy)))
    check_product(y, rounded(x), rounded(w), K, 1, "y")
    check_product(dx, rounded(dy), rounded(w.T), N, 1, "dx")
    check_product(dw, rounded(dy.T), rounded(x.T), M, 1, "dw")


@pytest.mark.parametrize("shape", [(9, 64, 96), (70, 130, 200)])
def test_gradient_against_differences(shape):
    """For L = sum(G * (X W^T)), linear in X: (L(X + D) - L(X - D)) / 2 is
    <dX, D> with dX = G W.  Both sides from the GPU's products, the sums in
    64 bits; each carries at most its products' bound."""
    M, N, K = shape
    rng = np.random.default_rng(14)
    x, d = rng.standard_normal((M, K)).astype(np.float32), rng.standard_normal((M, K)).astype(np.float32)
    g = rng.standard_normal((M, N)).astype(np.float32)
    q = ref.random_matrix(rng, (N,), K)
    W, w64 = held(*q, K), ref.values(*q, K)

    def L(v):
        return float((to_host(b.gemm_mxfp4_weight(to_dev(v), W)).astype(np.float64) * g).sum())

    plus, minus = x + d, x - d  # rounded once to FP32: the step is their difference
    step = (plus.astype(np.float64) - minus) / 2
    dx = to_host(b.gemm_mxfp4_weight(to_dev(g), W, op=b.OP_N)).astype(np.float64)
    got, want = (L(plus) - L(minus)) / 2, float((dx * step).sum())
    aw = np.abs(w64)
    S = ((np.abs(plus) + np.abs(minus)).astype(np.float64) @ aw.T * np.abs(g)).sum() / 2
    Sx = (np.abs(g).astype(np.float64) @ aw * np.abs(step)).sum()
    assert abs(got - want) <= (3 * K / 16 + 8) * ULP * S + (3 * N / 16 + 8) * ULP * Sx


def test_layer_served_token_by_token():
    """A stored layer applied to a prompt and then to single tokens: the rows
    of the one are the others', within the bound of each."""
    rng = np.random.default_rng(15)
    K, N = 512, 384
    q = ref.quantize((rng.standard_normal((N, K)) * 0.02).astype(np.float32))
    W, w64 = held(*q, K), ref.values(*q, K)
    x = rng.standard_normal((150, K)).astype(np.float32)
    X = to_dev(x)
    check_product(to_host(b.gemm_mxfp4_weight(X, W)), x.astype(np.float64), w64, K, 3)
    for i in (0, 77, 149):
        check_product(to_host(b.gemm_mxfp4_weight(X[i : i + 1], W)), x[i : i + 1].astype(np.float64), w64, K, 3)


# ---- streams, graphs, threads ------------------------------------------------------------

def test_runs_on_callers_stream_and_repeats_bit_for_bit():
    import torch

    rng = np.random.default_rng(16)
    x, w, dy = (to_dev(rng.standard_normal(s).astype(np.float32)) for s in ((300, 256), (512, 256), (300, 512)))
    want = [to_host(t) for t in linear_step(x, w, dy)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        q = b.mxfp4_quantize(x, stream=side)
        p = b.mxfp4_quantize(w, stream=side)
        y = b.gemm_mxfp4(q, p, stream=side)
        z = b.mxfp4_dequantize(q, stream=side)
        g = b.gemm_mxfp4_weight(dy, p, op=b.OP_N, stream=side)
        side.synchronize()
        assert np.array_equal(to_host(y), want[0])
        assert np.array_equal(to_host(z), rounded(to_host(x)).astype(np.float32))
        check_product(to_host(g), to_host(dy).astype(np.float64), rounded(to_host(w)).T, 512, 3)
    for _ in range(2):
        for u, v in zip(linear_step(x, w, dy), want):
            assert np.array_equal(to_host(u), v)


@pytest.mark.parametrize("shape", [(1, 256, 512), (70, 96, 640), (64, 64, 32768), (300, 520, 256)])
def test_graph_capture_replays(shape):
    import torch

    M, N, K = shape
    log(f"graph {shape}")
    rng = np.random.default_rng(17)
    X, W, dY = (to_dev(rng.standard_normal(s).astype(np.float32)) for s in ((M, K), (N, K), (M, N)))

    def step():
        y, dx, dw = linear_step(X, W, dY)
        q = b.mxfp4_quantize(W)
        return y, dx, dw, b.gemm_mxfp4_weight(X, q), b.gemm_mxfp4_weight(dY, q, op=b.OP_N), b.mxfp4_dequantize(q)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        for t in (X, W, dY):
            t.copy_(to_dev(rng.standard_normal(tuple(t.shape)).astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        got = [to_host(t).copy() for t in outs]
        for u, v in zip(got, step()):
            assert np.array_equal(u, to_host(v)), f"replay {i}"


def test_concurrent_calls_from_threads():
    import torch

    rng = np.random.default_rng(18)
    jobs = []
    for i in range(4):
        M, N, K = 40 + 50 * i, 100 + 30 * i, 200 + 64 * i
        x, w = to_dev(rng.standard_normal((M, K)).astype(np.float32)), to_dev(rng.standard_normal((N, K)).astype(np.float32))
        jobs.append((x, w, to_host(b.gemm_mxfp4(b.mxfp4_quantize(x), b.mxfp4_quantize(w)))))
    torch.cuda.synchronize()
    wrong = []

    def work(x, w, want):
        s = torch.cuda.Stream()
        for _ in range(5):
            y = b.gemm_mxfp4(b.mxfp4_quantize(x, stream=s), b.mxfp4_quantize(w, stream=s), stream=s)
            s.synchronize()
            if not np.array_equal(y.cpu().numpy(), want):
                wrong.append(tuple(x.shape))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# ---- large products, against float64 products on the GPU ------------------------------------

def random_on_gpu(rows, cols, seed):
    """(Mxfp4, its float64 values) of random codes, scales within 2^+-4."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = ref.blocks(cols)
    codes = torch.randint(0, 256, (rows, nb * 16), generator=g, device="cuda", dtype=torch.uint8)
    if cols % 32:
        keep = torch.arange(nb * 32, device="cuda") < cols
        mask = torch.where(keep, 15, 0).view(-1, 2)
        codes &= (mask[:, 0] | mask[:, 1] << 4).to(torch.uint8)
    scales = torch.randint(123, 132, (rows, ref.blocks(nb * 8) * 4), generator=g, device="cuda").to(torch.uint8)
    nib = torch.stack((codes & 15, codes >> 4), -1).view(rows, nb * 32)[:, :cols].long()
    table = torch.tensor(np.concatenate([ref.ELEMENTS, -ref.ELEMENTS]), device="cuda")
    v = table[nib] * torch.exp2(scales[:, :nb].double() - 127).repeat_interleave(32, 1)[:, :cols]
    return b.Mxfp4(codes, scales, cols), v


LARGE = [(4133, 4161, 1000), (4096, 4096, 2048), (8200, 2900, 515), (1100, 1024, 40000), (700, 9000, 1568),
         (2048, 2048, 512), (300, 2050, 1030), (200, 4000, 1029), (511, 1023, 2077), (100, 8193, 1500),
         (260, 520, 9000), (65, 14000, 1100)]


@pytest.mark.parametrize("shape", LARGE)
def test_large_products(shape):
    import torch

    M, N, K = shape
    log(f"large {shape}")
    A, a64 = random_on_gpu(M, K, 1)
    W, w64 = random_on_gpu(N, K, 2)
    x = torch.randn(M, K, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") * \
        torch.exp2(torch.arange(K, device="cuda") % 13 - 6.0)
    Wn, wn64 = random_on_gpu(K, N, 4)
    for name, got, p, q, parts in (("product", b.gemm_mxfp4(A, W), a64, w64.t(), 1),
                                   ("weight T", b.gemm_mxfp4_weight(x, W), x.double(), w64.t(), 3),
                                   ("weight N", b.gemm_mxfp4_weight(x, Wn, op=b.OP_N), x.double(), wn64, 3)):
        want, S = p @ q, p.abs() @ q.abs()
        over = (got.double() - want).abs() - (parts * K / 16 + 8) * ULP * S
        assert bool(torch.isfinite(got).all()) and float(over.max()) <= 0, (name, float(over.max()))


def test_large_batch():
    import torch

    A, a64 = random_on_gpu(20 * 520, 600, 5)
    W, w64 = random_on_gpu(20 * 530, 600, 6)
    A3 = b.Mxfp4(A.codes.view(20, 520, -1), A.scales.view(20, 520, -1), 600)
    W3 = b.Mxfp4(W.codes.view(20, 530, -1), W.scales.view(20, 530, -1), 600)
    x = torch.randn(20, 520, 600, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    w64 = w64.view(20, 530, 600).transpose(1, 2).contiguous()
    for got, p, parts in ((b.gemm_mxfp4(A3, W3), a64.view(20, 520, 600), 1),
                          (b.gemm_mxfp4_weight(x, W3), x.double(), 3)):
        over = (got.double() - p @ w64).abs() - (parts * 600 / 16 + 8) * ULP * (p.abs() @ w64.abs())
        assert float(over.max()) <= 0


def test_longest_rows():
    """The longest row there may be: 2^31 - 1024 values."""
    import torch

    K = (1 << 31) - 1024
    x = torch.zeros(3, K, device="cuda:0")
    for i in range(3):
        for v, k in ((1.0, 0), (2.0, K // 2 + 5 * i), (4.0, K - 1 - i)):
            x[i, k] = v
    ones = b.mxfp4_empty((2, K))
    ones.codes.fill_(0x22)
    ones.scales.fill_(127)
    want = torch.full((3, 2), 7.0, device="cuda:0")
    for M in (1, 2, 3):  # sums of powers of two and zeros: exact in any order
        assert torch.equal(b.gemm_mxfp4_weight(x[:M], ones), want[:M])
    q = b.mxfp4_quantize(x[2:])
    assert torch.equal(b.gemm_mxfp4(q, ones), want[:1])
    assert torch.equal(b.mxfp4_dequantize(q), x[2:])
    torch.cuda.empty_cache()


@pytest.mark.parametrize("shape", [(3, 100), (2, 3, 100), (1, 1), (0, 64), (3, 0), (0, 2, 40), (2, 0, 40), (2, 5, 0)])
def test_tensors_of_an_empty(shape):
    """codes and scales of an mxfp4_empty are its memory, also when asked for
    after a call has filled it."""
    import torch

    *lead, cols = shape
    nb = -(-cols // 32)
    x = torch.randn(shape, device="cuda:0")
    q = b.mxfp4_quantize(x)
    assert q.device == x.device and q.shape == shape
    assert q.codes.shape == (*lead, nb * 16) and q.scales.shape == (*lead, -(-nb // 4) * 4)
    again = b.Mxfp4(q.codes, q.scales, cols)
    assert torch.equal(b.mxfp4_dequantize(again), b.mxfp4_dequantize(q))
    e = b.mxfp4_empty(shape)
    e.codes.copy_(q.codes)
    e.scales.copy_(q.scales)
    assert torch.equal(b.mxfp4_dequantize(e), b.mxfp4_dequantize(q))
    assert e.codes.data_ptr() % 16 == 0 and e.scales.data_ptr() % 4 == 0
