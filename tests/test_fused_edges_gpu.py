"""The fused operators (include/gemm_f32_fused.h) where a result hangs on small values
beside large ones, on infinities, or on an operand of one to three columns.
Tolerances: fused_oracle.py."""

from __future__ import annotations

import math

import pytest
import torch

from dense_fp32_gemm_row_amd import binding as b
from tests import fused_oracle as o
from tests.test_fused_gpu import DEV, Guarded, rnd, stored, tokens

pytestmark = pytest.mark.gpu


# ---- probabilities of any size -------------------------------------------------

def peaked(T, V, K, gap, seed=40):
    """A softmax peaked to exp(-gap): token t is of class t % 16, whose word has a logit
    of `gap`, all others' are about 1.  Every second token's target is another word, so
    that its P is -1 there, and its hidden values, and those words' weights, are zero in half
    of the features: gradients there are sums of the small probabilities alone."""
    X, W = rnd(seed, T, K), rnd(seed + 1, V, K, scale=1 / math.sqrt(K))
    t = torch.arange(T, device=DEV)
    X[:, :16], W[:, :16] = 0.0, 0.0
    X[t, t % 16] = 1.0
    W[torch.arange(16), torch.arange(16)] = gap
    g = torch.Generator(device=DEV).manual_seed(seed + 2)
    target = torch.where(t % 2 == 0, torch.randint(16, 16 + V // 4, (T,), generator=g, device=DEV), t % 16)
    X[::2, K // 2:] = 0.0
    W[:16 + V // 4, K // 2:] = 0.0
    return X, W, target


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("gap", [16.0, 24.0, 28.0])
@pytest.mark.parametrize("T,V,K", [(2048, 4096, 2048), (700, 9001, 1030), (300, 2000, 130), (60, 1000, 96)])
def test_small_probabilities_count(T, V, K, gap, weights):
    X, W, target = peaked(T, V, K, gap)
    # loss weights from 1e-9 to 1, in an order of their own
    g = torch.logspace(-9, 0, T, device=DEV)[torch.randperm(T, generator=torch.Generator().manual_seed(3))] if weights else None
    want = o.loss_grad(X, W, target, g)
    for name, got in zip(("loss", "lse", "dX", "dW"), b.cross_entropy_grad(X, W, target, g)):
        o.check(got, *want[name], name)


# ---- tokens that take no part ------------------------------------------------------

SIZES = [(3, 500, 64), (70, 200, 32), (300, 300, 64), (40, 9000, 65), (400, 9000, 300), (520, 40000, 40),
         (2048, 4096, 2048)]


@pytest.mark.parametrize("pieces", [False, True])
@pytest.mark.parametrize("T,V,K", SIZES)
def test_ignored_tokens_beside_masked_words(T, V, K, pieces):
    """Words whose logits are -inf have a probability of zero.  Times their weights, of
    which one is -inf, that is NaN, but not in an ignored token's row of dX."""
    X, W, target = tokens(T, V, K, seed=50)
    X[:, 0] = 1.0
    W[10:200:7, 0] = -math.inf
    target[target >= 0] = target[target >= 0] % 10
    target[T // 2] = -100
    rest = torch.ones(V, dtype=torch.bool, device=DEV)
    rest[10:200:7] = False
    space = None
    if pieces:
        space = torch.empty(-(-b.gemm_f32_cross_entropy_grad_workspace_least(T, V, K) // 4), device=DEV)
    loss, lse, dX, dW = b.cross_entropy_grad(X, W, target, workspace=space)
    want = o.loss_grad(X, W[rest], target)
    ignored = target == -100
    o.check(loss, *want["loss"], "loss"), o.check(lse, *want["lse"], "lse")
    assert not dX[ignored].any() and bool(torch.isnan(dX[~ignored, 0]).all())
    o.check(dX[:, 1:], *(t[:, 1:] for t in want["dX"]), "dX")
    o.check(dW[rest], *want["dW"], "dW")
    assert not dW[~rest].any()
    assert torch.equal(torch.nan_to_num(b.cross_entropy_grad(X, W, target, dW=False, workspace=space)[2]), torch.nan_to_num(dX))


# ---- logits past FP32's range -----------------------------------------------------

@pytest.mark.parametrize("T,V,K", SIZES + [(1, 700, 40)])
def test_logits_past_the_range(T, V, K):
    """A logit of +inf makes its token's lse infinite, as the formula does, and its
    loss, unless it is the target's; its probability alone is NaN.  A logit of -inf is no
    word at all."""
    X, W, target = tokens(T, V, K, seed=60)
    at, word = T // 2, V // 3
    X[:, :2], W[:, :2] = 0.0, 0.0
    X[at, 0], W[word, 0], W[word + 1, 0] = 1e30, 1e30, -1e30
    target[at] = word + 2
    want = o.loss_grad(torch.where(torch.arange(T, device=DEV)[:, None] == at, 0.0, X), W, target)
    others = torch.arange(T, device=DEV) != at
    for loss, lse in (b.cross_entropy(X, W, target), b.cross_entropy_grad(X, W, target)[:2]):
        assert lse[at] == math.inf and loss[at] == math.inf
        for name, got in (("loss", loss), ("lse", lse)):
            o.check(got[others], *(t[others] for t in want[name]), name)
    _, _, dX, dW = b.cross_entropy_grad(X, W, target)
    assert bool(torch.isnan(dX[at]).all()) and bool(torch.isnan(dW[word]).all())
    o.check(dX[others], *(t[others] for t in want["dX"]), "dX")
    # the token's own share of the other words: a probability of 0, less 1 at the target
    share = torch.zeros(V, K, dtype=torch.float64, device=DEV)
    share[word + 2] = -X[at].double()
    valid = others & (target != -100)
    tokens_left = o.loss_grad(X[others], W, target[others]) if bool(valid.any()) else {"dW": (share * 0, share * 0)}
    value, tol = tokens_left["dW"]
    value, tol = value + share, tol + 2 * o.U * share.abs()
    keep = torch.arange(V, device=DEV) != word
    o.check(dW[keep], value[keep], tol[keep], "dW")
    target[at] = word
    loss, lse = b.cross_entropy(X, W, target)
    assert lse[at] == math.inf and bool(torch.isnan(loss[at]))
    X[at, 1] = math.nan
    loss, lse = b.cross_entropy(X, W, target)
    assert bool(torch.isnan(lse[at])) and bool(torch.isnan(loss[at]))


# ---- one to three columns --------------------------------------------------------

@pytest.mark.parametrize("ops", ["NN", "TN", "NT", "TT"])
@pytest.mark.parametrize("N", [1, 2, 3])
@pytest.mark.parametrize("M,K", [(1, 70000), (16, 33), (31, 5), (32, 4096), (33, 17), (300, 1), (1000, 777), (8192, 4096),
                                 (70001, 130), (3, 1 << 20)])
def test_few_columns(M, N, K, ops):
    A, B = stored(1, M, K, ops[0], 1), stored(2, K, N, ops[1], 2)
    bias, res = rnd(3, N), stored(4, M, N, "N", 5)
    c, z = Guarded(M, N), Guarded(M, N, 1)
    b.gemm_fused(A, B, c.out, bias=bias, activation="silu", residual=res, pre=z.out)
    want = o.layer(A, B, bias, "silu", res)
    o.check(c.out, want["y"], want["y_tol"])
    o.check(z.out, want["z"], want["z_tol"])
    c.check(), z.check()


@pytest.mark.parametrize("ops", ["NN", "TN", "NT", "TT"])
@pytest.mark.parametrize("M,N,K", [(8192, 1, 4096), (5000, 2, 300), (4100, 3, 3), (64, 700, 1), (1, 500, 2), (2000, 1, 1)])
def test_gradients_of_few_columns(M, N, K, ops):
    A, B = stored(1, M, K, ops[0], 2), stored(2, K, N, ops[1], 1)
    dC, z = rnd(3, M, N), rnd(4, M, N)
    da, db = Guarded(M, K, op=ops[0]), Guarded(K, N, op=ops[1])
    got = b.gemm_fused_grad(dC, A, B, pre=z, activation="gelu", dA=da.out, dB=db.out, dbias=True)
    want = o.layer_grad(dC, A, B, z, "gelu")
    for name, t in zip(("dA", "dB", "dbias"), got):
        o.check(t, *want[name], name)
    da.check(), db.check()


@pytest.mark.parametrize("n,M,N,K", [(40, 70, 1, 33), (300, 5, 3, 64), (7, 33, 2, 2000)])
def test_batches_of_few_columns(n, M, N, K):
    A, B = rnd(1, n, M, K), rnd(2, n, K, N)
    want = o.layer(A, B)
    o.check(b.gemm_fused(A, B), want["y"], want["y_tol"])


@pytest.mark.parametrize("T,V,K", [(3, 1, 40), (100, 1, 33), (400, 3, 2000), (513, 2, 70), (2000, 3, 300), (600, 500, 1),
                                   (40, 3000, 2), (2100, 40, 3)])
def test_losses_of_few_words_or_features(T, V, K):
    X, W, target = tokens(T, V, K, seed=70)
    want = o.loss_grad(X, W, target)
    for name, got in zip(("loss", "lse"), b.cross_entropy(X, W, target)):
        o.check(got, *want[name], name)
    for name, got in zip(("loss", "lse", "dX", "dW"), b.cross_entropy_grad(X, W, target)):
        o.check(got, *want[name], name)


# ---- tails of the activations --------------------------------------------------------

def test_gelu_keeps_relative_precision():
    """Of z times the normal distribution, z <= 0, down to where its parts leave FP32's normal
    range: the share is off by 20 steps (its polynomial's argument 3, times 2.3; its Horner
    scheme 3, its coefficients 4, the exponential 2, two products, the fit 1) and by
    the exponential's argument's, z^2 / 2 times two roundings and a constant's 0.2; then a product."""
    z = -torch.linspace(0.001, 12.5, 40001, device=DEV)
    y = b.gemm_fused(z[:, None], torch.ones(1, 1, device=DEV), activation="gelu")[:, 0].double()
    d = z.double()
    want = d * 0.5 * torch.special.erfc(-d / math.sqrt(2))
    assert bool(((y - want).abs() <= (1.2 * d * d + 21) * o.U * want.abs()).all())


# ---- both products of a loss's gradient in one launch of tiles --------------------------

# in slices of V and of T, both (643 to 804 tokens), or of V alone
SHARED = [(643, 737, 1258), (643, 2807, 209), (804, 921, 643), (33, 3508, 1573), (53, 2246, 2459)]


@pytest.mark.parametrize("T,V,K", SHARED)
def test_loss_gradients_that_share_a_launch(T, V, K):
    X, W, target = tokens(T, V, K, seed=80)
    target[-1] = 5
    g = rnd(81, T)
    want = o.loss_grad(X, W, target, g)
    got = b.cross_entropy_grad(X, W, target, g)
    for name, t in zip(("loss", "lse", "dX", "dW"), got):
        o.check(t, *want[name], name)
    assert torch.equal(b.cross_entropy_grad(X, W, target, g, dW=False)[2], got[2])
    assert torch.equal(b.cross_entropy_grad(X, W, target, g, dX=False)[3], got[3])
    # padding of anything takes no part
    ignored = target == -100
    X[ignored] = math.nan
    X[1] = math.inf
    odd = b.cross_entropy_grad(X, W, target, g)
    assert torch.equal(odd[0], got[0]) and torch.equal(odd[2], got[2])
    o.check(odd[3], *want["dW"], "dW")


@pytest.mark.parametrize("T,V,K", SHARED)
def test_masked_words_in_a_shared_launch(T, V, K):
    test_ignored_tokens_beside_masked_words(T, V, K, False)


@pytest.mark.parametrize("T,V,K", SHARED[:2])
def test_a_shared_launch_captured_and_on_another_stream(T, V, K):
    X, W, target = tokens(T, V, K, seed=82)
    first = b.cross_entropy_grad(X, W, target)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = b.cross_entropy_grad(X, W, target, stream=s)
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = b.cross_entropy_grad(X, W, target)
    for _ in range(3):
        for t in outs:
            t.fill_(12345.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(first, outs))
        assert all(torch.equal(a, c) for a, c in zip(first, b.cross_entropy_grad(X, W, target)))
