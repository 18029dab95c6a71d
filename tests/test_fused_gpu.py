"""The fused operators (include/gemm_f32_fused.h) on the GPU, against the same
in 64 bits.  Tolerances: fused_oracle.py."""

from __future__ import annotations

import math

import pytest
import torch

from dense_fp32_gemm_row_amd import binding as b
from tests import fused_oracle as o

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GUARD = 12345.0


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV) * scale


def stored(seed, rows, cols, op, pad=0, scale=1.0):
    """A rows x cols operand of form `op`, in a wider allocation of NaN."""
    r, c = (rows, cols) if op == "N" else (cols, rows)
    wide = torch.full((r, c + pad), math.nan, device=DEV)
    wide[:, :c] = rnd(seed, r, c, scale=scale)
    v = wide[:, :c]
    return v if op == "N" else v.t()


class Guarded:
    """A rows x cols output inside a larger allocation whose other cells must stay."""

    def __init__(self, rows, cols, pad=3, op="N"):
        r, c = (rows, cols) if op == "N" else (cols, rows)
        self.all = torch.full((r + 2, c + pad), GUARD, device=DEV)
        v = self.all[1:r + 1, :c]
        self.inner = v
        self.out = v if op == "N" else v.t()

    def check(self):
        rest = self.all.clone()
        r, c = self.inner.shape
        rest[1:r + 1, :c] = GUARD
        assert bool((rest == GUARD).all()), "written outside the output"


SHAPES = [(1, 4, 1), (2, 5, 4097), (16, 6, 64), (15, 2100, 200), (33, 9000, 65), (49, 16500, 70), (64, 33000, 40),
          (7, 32801, 130), (48, 8193, 127), (17, 4, 3000),
          (1, 1, 1), (1, 2, 3), (3, 5, 7), (2, 64, 16), (64, 128, 32), (65, 129, 33), (63, 127, 31), (17, 300, 50),
          (128, 128, 128), (129, 257, 100), (256, 256, 64), (255, 254, 253), (300, 520, 96), (1, 1000, 333),
          (5, 4, 2000), (1000, 1, 77), (260, 3, 40), (4, 4, 4), (131, 66, 17), (257, 258, 15)]


@pytest.mark.parametrize("ops", ["NN", "NT", "TN", "TT"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, ops):
    A, B = stored(1, M, K, ops[0], 1), stored(2, K, N, ops[1], 5)
    g = Guarded(M, N)
    b.gemm_fused(A, B, g.out)
    want = o.layer(A, B)
    o.check(g.out, want["y"], want["y_tol"])
    g.check()


# whole and ragged tiles of every size: the last tile a row, a few, or all of it
LARGE = [(3584, 3840, 64), (3329, 3585, 47), (3331, 3842, 16), (3400, 3700, 130),
         (1792, 1920, 64), (1665, 1793, 47), (1667, 1922, 33), (1700, 1900, 400)]


@pytest.mark.parametrize("ops", ["NN", "NT", "TN", "TT"])
@pytest.mark.parametrize("M,N,K", LARGE)
def test_large_products(M, N, K, ops):
    A, B = stored(1, M, K, ops[0], 1), stored(2, K, N, ops[1], 2)
    bias, res = rnd(3, N), stored(4, M, N, "N", 5)
    c, z = Guarded(M, N), Guarded(M, N, 1)
    b.gemm_fused(A, B, c.out, bias=bias, activation="gelu_tanh", residual=res, pre=z.out)
    want = o.layer(A, B, bias, "gelu_tanh", res)
    o.check(c.out, want["y"], want["y_tol"])
    o.check(z.out, want["z"], want["z_tol"])
    c.check(), z.check()


@pytest.mark.parametrize("n,M,N,K", [(25, 700, 780, 48), (40, 260, 385, 50), (70, 100, 300, 33)])
@pytest.mark.parametrize("ops", ["NN", "TT"])
def test_large_batches(n, M, N, K, ops):
    A = rnd(1, n, *((M, K) if ops[0] == "N" else (K, M)))
    B = rnd(2, n, *((K, N) if ops[1] == "N" else (N, K)))
    A, B = (A if ops[0] == "N" else A.transpose(1, 2)), (B if ops[1] == "N" else B.transpose(1, 2))
    y = b.gemm_fused(A, B)
    want = o.layer(A, B)
    o.check(y, want["y"], want["y_tol"])


@pytest.mark.parametrize("M,N,K", [(33, 70, 20), (130, 200, 64), (1, 257, 500), (300, 300, 300)])
@pytest.mark.parametrize("kind", o.ACTS)
@pytest.mark.parametrize("with_bias,with_residual,keep", [(True, True, True), (False, False, False), (True, False, True),
                                                          (False, True, False)])
def test_epilogue(M, N, K, kind, with_bias, with_residual, keep):
    A, B = stored(3, M, K, "N"), stored(4, K, N, "T", 3, scale=2 / math.sqrt(K))
    bias = rnd(5, N) if with_bias else None
    residual = stored(6, M, N, "N", 2) if with_residual else None
    c, z = Guarded(M, N), Guarded(M, N, 1)
    b.gemm_fused(A, B, c.out, bias=bias, activation=kind, residual=residual, pre=z.out if keep else None)
    want = o.layer(A, B, bias, kind, residual)
    o.check(c.out, want["y"], want["y_tol"], "C")
    c.check(), z.check()
    if keep:
        o.check(z.out, want["z"], want["z_tol"], "Z")
    else:
        assert bool((z.out == GUARD).all())


@pytest.mark.parametrize("M,N,K", [(40, 60, 30), (260, 300, 700), (1, 500, 900), (3, 8201, 66), (20, 33001, 40)])
def test_residual_may_be_the_output(M, N, K):
    A, B, x = rnd(1, M, K), rnd(2, K, N), rnd(3, M, N)
    want = o.layer(A, B, None, "silu", x)
    b.gemm_fused(A, B, x, activation="silu", residual=x)
    o.check(x, want["y"], want["y_tol"])


@pytest.mark.parametrize("kind", o.ACTS)
def test_activation_over_its_range(kind):
    """A product with 1 leaves the operand: tails, zeros of both signs, infinities, NaN."""
    z = torch.cat([torch.linspace(-30, 30, 4001, device=DEV), torch.tensor(
        [0.0, -0.0, 1e-30, -1e-30, 1e30, -1e30, 88.0, -88.0, -104.0, -250.0, 3.4e38, -3.4e38, math.inf, -math.inf,
         math.nan], device=DEV)])
    y = b.gemm_fused(z[:, None], torch.ones(1, 1, device=DEV), activation=kind)[:, 0]
    d = z.double()
    want = o.activate(kind, d)
    if kind != "none":  # the limit, where the formula is infinity times zero, or its power overflows
        want = torch.where(d < -1000, 0.0, want)
        want = torch.where(d > 1000, d, want)
    o.check(y, want, torch.nan_to_num(o.activation_tolerance(kind, d.clamp(-1000, 1000)), nan=0.0) + 2e-38)
    dA = b.gemm_fused_grad(torch.ones_like(y)[:, None], z[:, None].contiguous(), torch.ones(1, 1, device=DEV),
                           pre=z[:, None].contiguous(), activation=kind, dB=False)[0][:, 0]
    slope = o.slope(kind, d)
    if kind != "none":
        slope = torch.where(d < -300, 0.0, torch.where(d > 300, 1.0, slope))
        slope = torch.where(torch.isnan(d), d, slope)
    o.check(dA, slope, torch.nan_to_num(o.slope_tolerance(kind, d.clamp(-300, 300)), nan=0.0) + 2e-38, "slope")


@pytest.mark.parametrize("ops", ["NN", "NT", "TN", "TT"])
def test_batch(ops):
    n, M, N, K = 5, 70, 90, 40
    A = rnd(1, n, *((M, K) if ops[0] == "N" else (K, M)))
    B = rnd(2, n, *((K, N) if ops[1] == "N" else (N, K)))
    A, B = (A if ops[0] == "N" else A.transpose(1, 2)), (B if ops[1] == "N" else B.transpose(1, 2))
    bias, res = rnd(3, n, N), rnd(4, n, M, N)
    z = torch.empty(n, M, N, device=DEV)
    y = b.gemm_fused(A, B, bias=bias, activation="gelu", residual=res, pre=z)
    want = o.layer(A, B, bias, "gelu", res)
    o.check(y, want["y"], want["y_tol"]), o.check(z, want["z"], want["z_tol"])
    shared = b.gemm_fused(A[:1].expand(n, M, K), B, bias=bias[0], residual=res[:1].expand(n, M, N))
    want = o.layer(A[:1].expand(n, M, K), B, bias[0], "none", res[:1].expand(n, M, N))
    o.check(shared, want["y"], want["y_tol"])


@pytest.mark.parametrize("kind", ["none", "gelu"])
def test_nothing_to_sum(kind):
    bias = rnd(1, 9)
    z = torch.empty(4, 9, device=DEV)
    y = b.gemm_fused(torch.empty(4, 0, device=DEV), torch.empty(0, 9, device=DEV), bias=bias, activation=kind, pre=z)
    want = bias.double().expand(4, 9)
    assert torch.equal(z.double(), want)
    o.check(y, o.activate(kind, want), o.activation_tolerance(kind, want))
    for M, N in ((0, 9), (4, 0)):
        assert b.gemm_fused(torch.empty(M, 3, device=DEV), torch.empty(3, N, device=DEV)).shape == (M, N)


SPECIAL = [math.inf, -math.inf, math.nan, 3.4028234663852886e38, -3.4028234663852886e38, 3.3961775292304e38, 1e-40, 0.0]


@pytest.mark.parametrize("M,N,K", [(70, 130, 48), (300, 300, 70), (2, 600, 64), (130, 140, 33), (3330, 3600, 40),
                                   (1700, 1900, 50), (3330, 3600, 100), (1700, 1900, 96)])
@pytest.mark.parametrize("ops", ["NN", "NT", "TN", "TT"])
def test_values_at_the_ends_of_the_range(M, N, K, ops):
    """One special value in a row of A, against columns of B that hold zeros,
    small numbers and specials: what the sum of FP32 products gives."""
    A, B = rnd(1, M, K), rnd(2, K, N, scale=1e-3)
    for i, v in enumerate(SPECIAL):
        A[(11 * i + 1) % M, (7 * i) % K] = v
    B[0, 3], B[7, 5], B[:, 9] = 0.0, math.inf, 0.0
    a = A if ops[0] == "N" else A.t().contiguous().t()
    w = B if ops[1] == "N" else B.t().contiguous().t()
    y = b.gemm_fused(a, w)
    want = o.layer(A, B)
    top = torch.finfo(torch.float32).max
    # within FP32's range the sums are exact enough; past it they are infinite
    want["y"] = torch.where(want["y"].abs() > top, want["y"].sign() * math.inf, want["y"])
    o.check(y, want["y"], torch.nan_to_num(want["y_tol"], nan=0.0, posinf=0.0))


@pytest.mark.parametrize("scale_a,scale_b", [(1e-30, 1e-3), (1e30, 1e-30), (1e18, 1e18), (1e-18, 1e-18)])
def test_scales(scale_a, scale_b):
    A, B = rnd(1, 130, 200, scale=scale_a), rnd(2, 200, 140, scale=scale_b)
    want = o.layer(A, B)
    o.check(b.gemm_fused(A, B), want["y"], want["y_tol"])


def test_scales_that_cancel_along_the_sum():
    """Columns of A from 1e-20 to 1e20, rows of B the inverse: every product counts the same."""
    K = 160
    s = torch.logspace(-20, 20, K, device=DEV)
    A, B = rnd(1, 140, K) * s, rnd(2, K, 150) / s[:, None]
    want = o.layer(A, B)
    o.check(b.gemm_fused(A, B), want["y"], want["y_tol"])


def uneven(name, M, N, K):
    """Operands on whose ranges it depends how their values may be held."""
    A, B = rnd(1, M, K), rnd(2, K, N)
    if name == "along the sum":
        s = torch.logspace(-15, 15, K, device=DEV)
        A, B = A * s, B / s[:, None]
    elif name == "rows":
        A, B = A * torch.logspace(-25, 25, M, device=DEV)[:, None], B * torch.logspace(-12, 12, N, device=DEV)
    elif name == "one large":  # met by zeros, but for one column
        A[:, 5], B[5] = 1e20, 0.0
        B[5, 7] = 1e-20
    elif name == "one large each":  # met by the other's small ones
        A[::3, 5], B[5] = 1e15, B[5] * 1e-15
        B[9, ::5], A[:, 9] = 1e12, A[:, 9] * 1e-12
    elif name == "outliers":
        A[:, ::50] *= 300.0
        B[:, ::7] *= 100.0
    elif name == "half zeros":
        A = A.clamp_min(0.0)
    elif name == "zeros in both":
        A, B = A.clamp_min(0.0), B * (rnd(3, K, N) > 0)
    elif name == "apart":  # nothing meets: the sum is exactly zero
        A[:, : K // 2], B[K // 2:] = 0.0, 0.0
    elif name == "zero rows":
        A[3::5], B[:, 2::3] = 0.0, 0.0
    elif name == "tiny":
        A, B = A * 1e-37, B * 1e30
    elif name == "one row of infinities":
        A[77] = math.inf
    elif name == "lowest":
        A[70, 3], B[3] = torch.finfo(torch.float32).min, 1e-30
    return A, B


UNEVEN = ["along the sum", "rows", "one large", "one large each", "outliers", "half zeros", "zeros in both", "apart",
          "zero rows", "tiny", "one row of infinities", "lowest"]


@pytest.mark.parametrize("ops", ["NN", "NT", "TN", "TT"])
@pytest.mark.parametrize("name", UNEVEN)
@pytest.mark.parametrize("M,N,K", [(3400, 3600, 150), (1700, 1900, 130), (130, 200, 128)])
def test_uneven_operands(M, N, K, name, ops):
    A, B = uneven(name, M, N, K)
    a = A if ops[0] == "N" else A.t().contiguous().t()
    w = B if ops[1] == "N" else B.t().contiguous().t()
    want = o.layer(A, B)
    top = torch.finfo(torch.float32).max
    want["y"] = torch.where(want["y"].abs() > top, want["y"].sign() * math.inf, want["y"])
    y = b.gemm_fused(a, w)
    o.check(y, want["y"], torch.nan_to_num(want["y_tol"], nan=0.0, posinf=0.0))
    if name == "apart":
        assert not y.any()


@pytest.mark.parametrize("M,N,K", [(1, 1, 1 << 20), (64, 64, 1 << 18), (3400, 3600, 8200)])
@pytest.mark.parametrize("uniform", [False, True])
def test_long_sums(M, N, K, uniform):
    """Whether roundings fall one way would show on sums of one sign."""
    A, B = rnd(1, M, K), rnd(2, K, N)
    if uniform:
        A, B = A.abs(), B.abs()
    want = o.layer(A, B)
    y = b.gemm_fused(A, B)
    o.check(y, want["y"], want["y_tol"])
    # the root of the mean square, too: sqrt(K) roundings of at most S / sqrt(3) u each
    err = (y.double() - want["y"]).square().mean().sqrt()
    S = o.product(A, B)[1].square().mean().sqrt()
    assert err <= math.sqrt(K + 16) * o.U * S


@pytest.mark.parametrize("M,N,K", [(64, 64, 64), (300, 260, 200), (1, 300, 1000)])
def test_whole_numbers_are_exact(M, N, K):
    g = torch.Generator(device=DEV).manual_seed(0)
    A = torch.randint(-4, 5, (M, K), generator=g, device=DEV).float()
    B = torch.randint(-4, 5, (K, N), generator=g, device=DEV).float()
    assert torch.equal(b.gemm_fused(A, B).double(), torch.matmul(A.double(), B.double()))
    big = torch.randint(-(1 << 23), 1 << 23, (M, 1), generator=g, device=DEV).float()  # all 24 bits
    assert torch.equal(b.gemm_fused(big, torch.ones(1, N, device=DEV)), big.expand(M, N))


@pytest.mark.parametrize("ops", ["NN", "NT", "TN", "TT"])
@pytest.mark.parametrize("M,N,K,kind", [(1, 1, 1, "relu"), (33, 65, 40, "gelu"), (130, 90, 257, "silu"),
                                        (300, 40, 64, "gelu_tanh"), (64, 128, 33, "none"), (5, 300, 3, "relu"),
                                        (260, 514, 130, "silu"), (2000, 3400, 1801, "gelu"), (1801, 1700, 1902, "relu")])
def test_grad(M, N, K, kind, ops):
    A, B = stored(1, M, K, ops[0], 2), stored(2, K, N, ops[1], 1)
    dC, z = stored(3, M, N, "N", 4), stored(4, M, N, "N", 1, scale=2.0)
    da, db = Guarded(M, K, op=ops[0]), Guarded(K, N, op=ops[1])
    bias = torch.full((N + 2,), GUARD, device=DEV)
    got = b.gemm_fused_grad(dC, A, B, pre=z, activation=kind, dA=da.out, dB=db.out, dbias=bias[1:N + 1])
    want = o.layer_grad(dC, A, B, z, kind)
    for name, t in zip(("dA", "dB", "dbias"), got):
        o.check(t, *want[name], name)
    da.check(), db.check()
    assert bias[0] == GUARD and bias[-1] == GUARD
    # one at a time, allocated: the same bits, laid out as the operand
    for i, name in enumerate(("dA", "dB", "dbias")):
        one = b.gemm_fused_grad(dC, A, B, pre=z, activation=kind,
                                **{k: k == name for k in ("dA", "dB", "dbias")})
        assert torch.equal(one[i], got[i]) and all(t is None for j, t in enumerate(one) if j != i)


def test_grad_of_a_batch():
    n, M, N, K = 3, 50, 70, 30
    A, B, dC, z = rnd(1, n, M, K), rnd(2, n, K, N), rnd(3, n, M, N), rnd(4, n, M, N)
    got = b.gemm_fused_grad(dC, A, B, pre=z, activation="silu", dbias=True)
    want = o.layer_grad(dC, A, B, z, "silu")
    for name, t in zip(("dA", "dB", "dbias"), got):
        o.check(t, *want[name], name)
    # a shared operand: its gradient per product
    got = b.gemm_fused_grad(dC, A[:1].expand(n, M, K), B, pre=z, activation="silu")
    want = o.layer_grad(dC, A[:1].expand(n, M, K), B, z, "silu")
    o.check(got[0], *want["dA"]), o.check(got[1], *want["dB"])


@pytest.mark.parametrize("M,N,K", [(0, 5, 4), (3, 0, 4), (3, 5, 0)])
def test_grad_of_empty_products(M, N, K):
    dA, dB, dbias = b.gemm_fused_grad(rnd(1, M, N), rnd(2, M, K), rnd(3, K, N), pre=rnd(4, M, N), activation="silu",
                                      dbias=True)
    assert dA.shape == (M, K) and dB.shape == (K, N) and dbias.shape == (N,)
    assert not dA.any() and not dB.any()
    if M == 0:
        assert not dbias.any()


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_grad_against_differences(kind):
    """sum(dC * C) along a direction D of A, by central differences with step h:
    they leave out h^2 / 6 |f'''|, with |f'''| below 2 for these activations; each
    value is off by the layer's tolerance, each step by its rounding."""
    M, N, K, h = 40, 50, 30, 2.0 ** -5
    A, B, bias, dC = rnd(1, M, K), rnd(2, K, N, scale=1 / math.sqrt(K)), rnd(3, N), rnd(4, M, N)
    D = rnd(5, M, K, scale=1 / math.sqrt(K))
    z = torch.empty(M, N, device=DEV)
    b.gemm_fused(A, B, bias=bias, activation=kind, pre=z)
    dA, dB, dbias = b.gemm_fused_grad(dC, A, B, pre=z, activation=kind, dbias=True)
    for grad, step in ((dA, "A"), (dB, "B"), (dbias, "bias")):
        dirs = {"A": D, "B": rnd(6, K, N, scale=1 / math.sqrt(K)), "bias": rnd(7, N)}[step]
        val, slack = [], 0.0
        for s in (h, -h):
            args = {"A": A, "B": B, "bias": bias}
            args[step] = args[step] + s * dirs
            y = b.gemm_fused(args["A"], args["B"], bias=args["bias"], activation=kind)
            want = o.layer(args["A"], args["B"], args["bias"], kind)
            val.append((dC.double() * y.double()).sum().item())
            slack += (dC.double().abs() * want["y_tol"]).sum().item()
        d = dirs.double()
        direction = (torch.matmul(d, B.double()) if step == "A" else
                     torch.matmul(A.double(), d) if step == "B" else d.expand(M, N))
        third = (dC.double().abs() * direction.abs() ** 3).sum().item() * 2 * h * h / 6
        start = {"A": A, "B": B, "bias": bias}[step].double().abs()  # whose sum with a step is rounded
        rounded = o.U * (grad.double().abs() * (start + h * d.abs())).sum().item() / h
        diff = (val[0] - val[1]) / (2 * h)
        assert abs(diff - (grad.double() * dirs.double()).sum().item()) <= slack / (2 * h) + third + rounded


# ---- cross entropy -----------------------------------------------------------

def tokens(T, V, K, seed=0, ignore=-100, scale=2.0):
    X, W = stored(seed, T, K, "N", 1), stored(seed + 1, V, K, "N", 3, scale=scale / math.sqrt(max(K, 1)))
    g = torch.Generator(device=DEV).manual_seed(seed + 2)
    target = torch.randint(0, V, (T,), generator=g, device=DEV)
    if T > 2:
        target[1::5] = ignore
    return X, W, target


LOSS_SHAPES = [(1, 4, 1), (2, 5, 4097), (16, 6, 64), (15, 2100, 200), (33, 9000, 65), (49, 16500, 70), (64, 33000, 40),
          (7, 32801, 130), (48, 8193, 127), (17, 4, 3000),
          (1, 1, 1), (1, 2, 5), (2, 64, 16), (3, 1000, 40), (64, 128, 32), (65, 129, 33), (100, 777, 65),
               (130, 64, 64), (1, 5000, 300), (17, 63, 8), (300, 2049, 100), (5, 1, 7), (257, 300, 48), (16, 4096, 64), (48, 700, 90),
               (64, 130, 1000), (33, 65, 64), (400, 9000, 300), (512, 20000, 700), (513, 4100, 130),
               (1700, 2000, 72), (3340, 3700, 50), (2000, 9001, 1800)]


@pytest.mark.parametrize("T,V,K", LOSS_SHAPES)
def test_cross_entropy(T, V, K):
    X, W, target = tokens(T, V, K)
    want = o.loss_grad(X, W, target)
    loss, lse = b.cross_entropy(X, W, target)
    o.check(loss, *want["loss"], "loss")
    o.check(lse, *want["lse"], "lse")


@pytest.mark.parametrize("T,V,K", LOSS_SHAPES)
@pytest.mark.parametrize("weights", [False, True])
def test_cross_entropy_grad(T, V, K, weights):
    X, W, target = tokens(T, V, K, seed=5, ignore=7 if V > 7 else -1)
    ignore = 7 if V > 7 else -1
    g = rnd(9, T) if weights else None
    want = o.loss_grad(X, W, target, g, ignore)
    dx, dw = Guarded(T, K), Guarded(V, K)
    loss, lse, dX, dW = b.cross_entropy_grad(X, W, target, g, ignore_index=ignore, dX=dx.out, dW=dw.out)
    for name, t in (("loss", loss), ("lse", lse), ("dX", dX), ("dW", dW)):
        o.check(t, *want[name], name)
    dx.check(), dw.check()
    assert not dX[target == ignore].any()
    alone = b.cross_entropy_grad(X, W, target, g, ignore_index=ignore, dX=False)
    assert alone[2] is None and torch.equal(alone[3], dW)
    alone = b.cross_entropy_grad(X, W, target, g, ignore_index=ignore, dW=False)
    assert alone[3] is None and torch.equal(alone[2], dX)


@pytest.mark.parametrize("T,rows", [(300, 64), (300, 100), (600, 256), (65, 64), (129, 65)])
def test_cross_entropy_grad_in_pieces(T, rows):
    """A workspace for `rows` tokens at a time."""
    V, K = 333, 50
    X, W, target = tokens(T, V, K, seed=3)
    want = o.loss_grad(X, W, target)
    least = b.gemm_f32_cross_entropy_grad_workspace_least(T, V, K)
    space = torch.full((-(-least * rows // 64) // 4 + 1 + 64,), GUARD, device=DEV)
    got = b.cross_entropy_grad(X, W, target, workspace=space[:-64])
    assert bool((space[-64:] == GUARD).all())
    for name, t in zip(("loss", "lse", "dX", "dW"), got):
        o.check(t, *want[name], name)


def test_every_token_ignored():
    X, W, target = tokens(70, 200, 32)
    target[:] = -100
    X[3] = math.nan
    loss, lse, dX, dW = b.cross_entropy_grad(X, W, target)
    assert not loss.any() and not dX.any() and not dW.any()
    assert not b.cross_entropy(X, W, target)[0].any()


@pytest.mark.parametrize("T,V,K", [(70, 200, 32), (300, 300, 64), (3, 500, 64), (70, 40, 32), (300, 7, 70),
                                   (512, 6000, 300), (700, 2000, 1)])
def test_ignored_rows_may_hold_anything(T, V, K):
    """Padding of NaN, infinities and huge values takes no part; the tokens
    beside it keep their values to the last bit."""
    X, W, target = tokens(T, V, K)
    target[0], target[2] = -100, -100
    clean = X.clone()
    clean[target == -100] = 0.0
    want = b.cross_entropy_grad(clean, W, target)
    X[0], X[2] = math.nan, math.inf
    X[1] = torch.finfo(torch.float32).min
    target[1] = -100
    clean[1] = 0.0
    want = b.cross_entropy_grad(clean, W, target)
    got = b.cross_entropy_grad(X, W, target)
    keep = target != -100
    assert torch.equal(got[0], want[0]) and torch.equal(got[1][keep], want[1][keep])
    assert torch.equal(got[2], want[2])
    oracle = o.loss_grad(clean, W, target)
    o.check(got[3], *oracle["dW"])
    assert torch.equal(b.cross_entropy(X, W, target)[0], want[0])


def test_targets_outside_the_vocabulary():
    X, W, target = tokens(40, 100, 16)
    target[4], target[5] = 100, -3
    loss, lse, dX, _ = b.cross_entropy_grad(X, W, target)
    bad = torch.zeros(40, dtype=torch.bool, device=DEV)
    bad[4:6] = True
    assert torch.isnan(loss[bad]).all() and torch.isfinite(loss[~bad]).all()
    assert torch.isfinite(lse).all()
    assert torch.isnan(dX[bad]).all() and torch.isfinite(dX[~bad]).all()
    assert torch.equal(torch.isnan(b.cross_entropy(X, W, target)[0]), bad)


def test_large_logits():
    """Logits of +-1e4: the maximum is taken out; and words masked by -inf."""
    X, W, target = tokens(80, 300, 64, scale=2000.0)
    want = o.loss_grad(X, W, target)
    got = b.cross_entropy_grad(X, W, target)
    for name, t in zip(("loss", "lse", "dX", "dW"), got):
        o.check(t, *want[name], name)
    X, W, target = tokens(80, 300, 64)
    X[:, 0] = 1.0
    W[10:200, 0] = -math.inf
    target[:] = 5
    loss, lse = b.cross_entropy(X, W, target)
    rest = torch.cat([W[:10], W[200:]])
    want = o.loss_grad(X, rest, target)
    o.check(loss, *want["loss"]), o.check(lse, *want["lse"])


# ---- how they are called ------------------------------------------------------

def everything():
    """One call of each operator, and its outputs."""
    X, W, target = tokens(150, 700, 64, seed=20)
    A, B, bias, R = rnd(1, 200, 96), rnd(2, 96, 300), rnd(3, 300), rnd(4, 200, 300)
    z = torch.empty(200, 300, device=DEV)

    def call(stream=None):
        y = b.gemm_fused(A, B, bias=bias, activation="gelu", residual=R, pre=z, stream=stream)
        grads = b.gemm_fused_grad(y, A, B, pre=z, activation="gelu", dbias=True, stream=stream)
        return [y, z, *grads, *b.cross_entropy(X, W, target, stream=stream),
                *b.cross_entropy_grad(X, W, target, stream=stream)]

    return call


def test_runs_repeat_to_the_last_bit():
    call = everything()
    first = [t.clone() for t in call()]
    for _ in range(3):
        assert all(torch.equal(a, c) for a, c in zip(first, call()))


def test_on_another_stream():
    call = everything()
    first = [t.clone() for t in call()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(stream=s)
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(first, got))


def test_captured_and_replayed():
    call = everything()
    first = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for _ in range(4):
        for t in outs:
            t.fill_(GUARD)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(first, outs))
        assert all(torch.equal(a, c) for a, c in zip(first, call()))


def test_a_network_learns_as_its_formulas_say():
    """Two layers and the loss, three steps of descent: gradients of every
    step against 64 bits (torch.autograd) at the same weights.  The bound:
    three products and two epilogues in a row, each off by its own tolerance
    of at most 8 sqrt(K + 16) u S and S below 20 times the product's own
    spread, so 1e-4 of a gradient's largest element."""
    T, D, H, V, ignore = 140, 72, 200, 501, -100
    x0 = rnd(1, T, D)
    ws = [rnd(2, H, D, scale=1 / math.sqrt(D)), rnd(3, D, H, scale=1 / math.sqrt(H)), rnd(4, V, D, scale=1 / math.sqrt(D))]
    bias = rnd(5, H, scale=0.1)
    target = torch.randint(0, V, (T,), generator=torch.Generator(device=DEV).manual_seed(6), device=DEV)
    target[::7] = ignore
    g = torch.full((T,), 1.0 / int((target != ignore).sum()), device=DEV)
    for _ in range(3):
        w1, w2, head = ws
        z = torch.empty(T, H, device=DEV)
        h = b.gemm_fused(x0, w1.t(), bias=bias, activation="gelu", pre=z)
        x1 = b.gemm_fused(h, w2.t(), residual=x0)
        loss, _, dx1, dhead = b.cross_entropy_grad(x1, head, target, g, ignore_index=ignore)
        dh, dw2, _ = b.gemm_fused_grad(dx1, h, w2.t())
        _, dw1, dbias = b.gemm_fused_grad(dh, x0, w1.t(), pre=z, activation="gelu", dA=False, dbias=True)
        params = [t.double().cpu().requires_grad_() for t in (w1, w2, head, bias)]
        p1, p2, p3, pb = params
        hidden = torch.nn.functional.gelu(x0.double().cpu() @ p1.t() + pb)
        x1d = x0.double().cpu() + hidden @ p2.t()
        total = torch.nn.functional.cross_entropy(x1d @ p3.t(), target.cpu(), ignore_index=ignore)
        total.backward()
        assert abs((loss * g).sum().item() - total.item()) <= 1e-5 * (1 + abs(total.item()))
        for got, p in ((dw1.t(), p1), (dw2.t(), p2), (dhead, p3), (dbias, pb)):
            err = (got.double().cpu() - p.grad).abs().max()
            assert err <= 1e-4 * p.grad.abs().max()
        ws = [w1 - 0.5 * dw1.t(), w2 - 0.5 * dw2.t(), head - 0.5 * dhead]
        bias = bias - 0.5 * dbias


# ---- large products, and what they share --------------------------------------

def test_ignored_rows_out_of_scale_take_no_part():
    """Padding many orders of magnitude above the tokens, in products large
    enough for parts scaled by a row's largest value."""
    T, V, K = 2048, 4096, 2048
    X, W, target = tokens(T, V, K, seed=30)
    target[torch.arange(T, device=DEV) % 16 != 3] = -100
    ignored = target == -100
    clean = torch.where(ignored[:, None], 0.0, X)
    X = torch.where(ignored[:, None], 1e30 * clean[3].abs() + 1e30, X)
    want = o.loss_grad(clean, W, target)
    loss, lse, dX, dW = b.cross_entropy_grad(X, W, target)
    o.check(loss, *want["loss"], "loss"), o.check(dX, *want["dX"], "dX"), o.check(dW, *want["dW"], "dW")


def test_words_out_of_scale():
    """A word that no token can take, with weights far above the others': its
    share of dX is an exact zero."""
    T, V, K = 2048, 4096, 2048
    X, W, target = tokens(T, V, K, seed=31)
    X[:, :64] = X[:, :64].abs() + 0.5
    W[V - 1] = 0.0
    W[V - 1, :64] = -1e9
    target[target == V - 1] = 0
    want = o.loss_grad(X, W[:-1], target)
    loss, lse, dX, dW = b.cross_entropy_grad(X, W, target)
    o.check(loss, *want["loss"], "loss"), o.check(dX, *want["dX"], "dX")
    o.check(dW[:-1], *want["dW"], "dW")
    assert not dW[-1].any()


def test_pieces_of_many_tokens():
    """Logits of more than one piece at the workspace that is quickest; the
    oracle goes by 250 tokens.  dW is a sum of the pieces', one rounding each."""
    T, V, K = 4000, 300_001, 24
    X, W, target = tokens(T, V, K, seed=32)
    loss, lse, dX, dW = b.cross_entropy_grad(X, W, target)
    sums = [torch.zeros(V, K, dtype=torch.float64, device=DEV) for _ in range(3)]
    for t in range(0, T, 250):
        rows = slice(t, t + 250)
        want = o.loss_grad(X[rows], W, target[rows])
        for name, got in (("loss", loss), ("lse", lse), ("dX", dX)):
            o.check(got[rows], *want[name], name)
        sums[0] += want["dW"][0]
        # the tolerance of a sum of 250 products covers that many roundings of its own share;
        # a sum of T has them relative to all that came before
        sums[1] += want["dW"][1] * math.sqrt(T / 250 + 1)
        sums[2] += want["dW"][0].abs()
    o.check(dW, sums[0], sums[1] + 4 * o.U * sums[2], "dW")


@pytest.mark.parametrize("stored_as", ["in_out", "out_in"])
@pytest.mark.parametrize("M,N,K", [(1000, 1023, 777), (160, 1373, 2000), (517, 2304, 400), (148, 1824, 1500),
                                   (2000, 160, 700)])
def test_gradients_that_share_a_launch(M, N, K, stored_as):
    A, B = rnd(1, M, K), stored(2, K, N, "N" if stored_as == "in_out" else "T", 1)
    dC = rnd(3, M, N)
    want = o.layer_grad(dC, A, B)
    got = b.gemm_fused_grad(dC, A, B, dbias=True)
    for name, t in zip(("dA", "dB", "dbias"), got):
        o.check(t, *want[name], name)
    assert torch.equal(b.gemm_fused_grad(dC, A, B, dB=False)[0], got[0])
    assert torch.equal(b.gemm_fused_grad(dC, A, B, dA=False)[1], got[1])


@pytest.mark.parametrize("M,N,K,ops", [(3, 40, 70, "NT"), (20, 40, 70, "NN"), (200, 300, 64, "NN"), (200, 300, 64, "NT"),
                                       (200, 72, 64, "TN"), (90, 300, 64, "TT")])
def test_offsets_past_32_bits(M, N, K, ops):
    """Rows 64 or 256 MiB apart."""
    def far(seed, rows, cols, op):
        r, c = (rows, cols) if op == "N" else (cols, rows)
        ld = 2 ** 24 if r > 64 else 2 ** 26
        wide = torch.empty(((r - 1) * ld + c,), device=DEV).as_strided((r, c), (ld, 1))
        wide.copy_(rnd(seed, r, c))
        return wide if op == "N" else wide.t()

    A, B = far(1, M, K, ops[0]), rnd(2, K, N)
    near = A.clone(memory_format=torch.contiguous_format)
    want = o.layer(near, B)
    B = B if ops[1] == "N" else B.t().contiguous().t()
    o.check(b.gemm_fused(A, B), want["y"], want["y_tol"])
    del A
    B2 = far(2, K, N, ops[1])
    want = o.layer(near, B2.clone(memory_format=torch.contiguous_format))
    o.check(b.gemm_fused(near, B2), want["y"], want["y_tol"])


def large_calls():
    A, B, dC = rnd(1, 1000, 777), rnd(2, 777, 1023), rnd(3, 1000, 1023)
    X, W, target = tokens(2048, 4096, 2048, seed=33)
    lib = b.load()

    def call(space=None, stream=None):
        """`space(bytes)` gives a workspace."""
        got = lambda n: space(n) if space is not None and n else None
        y = b.gemm_fused(A, B, activation="silu", stream=stream,
                         workspace=got(lib.gemm_f32_fused_workspace_size(0, 0, 1, 1000, 1023, 777)))
        grads = b.gemm_fused_grad(dC, A, B, pre=y, activation="silu", dbias=True, stream=stream, workspace=got(
            lib.gemm_f32_fused_grad_workspace_size(0, 0, 1, 1000, 1023, 777, 4, 1, 1, 1)))
        loss = b.cross_entropy(X, W, target, stream=stream,
                               workspace=got(lib.gemm_f32_cross_entropy_workspace_size(2048, 4096, 2048)))
        return [y, *grads, *loss, *b.cross_entropy_grad(X, W, target, stream=stream, workspace=got(
            lib.gemm_f32_cross_entropy_grad_workspace_size(2048, 4096, 2048)))]

    return call


def test_workspaces_start_anywhere():
    """4-byte aligned, of exactly the bytes asked for, holding NaN."""
    call = large_calls()
    kept = []

    def space(n):
        kept.append(torch.full((n // 4 + 2,), math.nan, device=DEV))
        kept[-1][0] = kept[-1][-1] = GUARD
        return kept[-1][1:-1]

    first, got = call(), call(space)
    assert all(torch.equal(a, c) for a, c in zip(first, got))
    assert all(t[0] == GUARD and t[-1] == GUARD for t in kept) and len(kept) == 4


def test_calls_at_once():
    """Two streams, a workspace for each call, several rounds."""
    call = large_calls()
    first = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[call(stream=s) for s in streams] for _ in range(3)]
    torch.cuda.synchronize()
    for pair in outs:
        for got in pair:
            assert all(torch.equal(a, c) for a, c in zip(first, got))


def test_large_calls_captured_and_replayed():
    call = large_calls()
    first = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call()
    for _ in range(3):
        for t in outs:
            t.fill_(GUARD)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(first, outs))
        assert all(torch.equal(a, c) for a, c in zip(first, call()))


@pytest.mark.parametrize("ops", ["NN", "NT", "TN", "TT"])
@pytest.mark.parametrize("M,N", [(700, 900), (1300, 2050), (2600, 4100)])
def test_sums_that_end_inside_a_stage(M, N, ops):
    """Whole numbers, whose sums are exact in any order and form: a k that is
    summed twice or left out shows.  An infinity near the end of K counts once, too."""
    for K in (15, 16, 17, 31, 33, 47, 48, 63, 65, 100, 127, 200, 399):
        A = stored(K, M, K, ops[0]).mul(3.0).round()
        B = stored(K + 1, K, N, ops[1]).mul(3.0).round()
        want = torch.matmul(A.double().contiguous(), B.double().contiguous()).float()
        got = b.gemm_fused(A, B)
        assert torch.equal(got, want), K
        A[:, max(K - 20, 0)] = 1.0
        B[max(K - 20, 0), 5] = math.inf
        got = b.gemm_fused(A, B)
        assert bool((got[:, 5] == math.inf).all()) and bool(torch.isfinite(got[:, 6:]).all()), K
