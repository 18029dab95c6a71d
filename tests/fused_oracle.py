"""The fused operators (include/gemm_f32_fused.h) in 64 bits, and how far FP32
results may be from them.

Tolerances.  u = 2^-24 is half a step of FP32.  With S the sum of |a b|, a sum
of K products in FP32, in any order, is off by at most (K + 16) u S: K roundings
of partial sums, each at most u of S, and the 16 cover the terms that
the product of three parts leaves out (at most 2 u of each |a b|) and the joining
of slices.  Roundings of random data don't all fall one way: the error of
sqrt(K) independent ones exceeds 8 sqrt(K + 16) u S with probability below
1e-13, and the smaller of the two is the bound.  Values below 2^-110 are held to 2^-134.
"""

from __future__ import annotations

import math

import torch

U = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
C = math.sqrt(2 / math.pi)


def product(A, B):
    """(A B, S) in 64 bits; the operands may be any 2-D or 3-D float32 tensors."""
    a, b = A.double().contiguous(), B.double().contiguous()
    return torch.matmul(a, b), torch.matmul(a.abs(), b.abs())


def least_tolerance(A, B):
    """What the least place of the operands' parts amounts to (no NaN or infinities)."""
    a, b = (torch.nan_to_num(t.double().abs(), nan=0.0, posinf=0.0) for t in (A, B))
    return 2.0 ** -134 * (a.sum(-1)[..., :, None] + b.sum(-2)[..., None, :])


def product_tolerance(S, K: int):
    return min(K + 16, 8 * math.sqrt(K + 16)) * U * S + K * 2.0 ** -130


def _share(kind, z):
    """(q, u): act(z) = z q, and how much a rounding of q's argument moves q."""
    if kind == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)), z * z
    if kind == "gelu_tanh":
        v = 2 * C * (z + 0.044715 * z ** 3)
    else:
        v = z
    return 1 / (1 + torch.exp(-v)), v


def activate(kind, z):
    if kind == "none":
        return z
    if kind == "relu":
        return torch.where(z < 0, 0.0, z)
    return z * _share(kind, z)[0]


def slope(kind, z):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0).double()
    q, _ = _share(kind, z)
    if kind == "gelu":
        return q + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    dv = 2 * C * (1 + 3 * 0.044715 * z * z) if kind == "gelu_tanh" else 1.0
    return q + z * q * (1 - q) * dv


def activation_tolerance(kind, z):
    """Of act(z) for an exact z: q = z's share is an exponential or erfc of an
    argument that is itself rounded (4 roundings, relative to which q moves by
    |u| at most), the function is good to 4 steps, then a sum, a
    division and a product."""
    if kind in ("none", "relu"):
        return torch.zeros_like(z)
    q, u = _share(kind, z)
    return (z * q).abs() * (4 * u.abs() + 12) * U + 2.0 ** -126


def slope_tolerance(kind, z):
    """As activation_tolerance, for both terms of the slope; the second has up
    to 8 roundings more, and |z| <= 15 holds where it isn't 0 (its share of
    the sum is below 2, the factor of its argument's rounding below z^2)."""
    if kind in ("none", "relu"):
        return torch.zeros_like(z)
    q, u = _share(kind, z)
    lean = (q * (4 * u.abs() + 12)).abs()
    if kind == "gelu":
        second = (z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)).abs() * (2 * z * z + 12)
    else:
        dv = 2 * C * (1 + 3 * 0.044715 * z * z) if kind == "gelu_tanh" else 1.0
        # 1 - q has an error of q's, absolutely
        second = (z * q * (1 - q) * dv).abs() * (4 * u.abs() + 20) + (z * q * dv).abs() * q * 12
    return (lean + second) * U + 2.0 ** -126


def layer(A, B, bias=None, kind="none", residual=None):
    """{"y", "y_tol", "z", "z_tol"}"""
    z, S = product(A, B)
    K = A.shape[-1]
    tol = product_tolerance(S, K) + least_tolerance(A, B)
    if bias is not None:
        b = bias.double()
        b = b[:, None, :] if b.dim() == 2 else b
        z = z + b
        tol = tol + U * (z.abs() + tol)
    y = activate(kind, z)
    # no activation's slope is above 1.13
    y_tol = 1.13 * tol + activation_tolerance(kind, z)
    if residual is not None:
        y = y + residual.double()
        y_tol = y_tol + U * (y.abs() + y_tol)
    return {"y": y, "y_tol": y_tol, "z": z, "z_tol": tol}


def layer_grad(dC, A, B, z=None, kind="none"):
    """{"dA", "dB", "dbias"} each (value, tolerance), for one product."""
    g = dC.double()
    gt = torch.zeros_like(g)
    if kind != "none":
        z = z.double()
        gt = g.abs() * slope_tolerance(kind, z)
        g = g * slope(kind, z)
        gt = gt + U * g.abs()
    a, b = A.double(), B.double()
    bt, at = b.transpose(-1, -2).contiguous(), a.transpose(-1, -2).contiguous()
    N, M = g.shape[-1], g.shape[-2]
    dA = torch.matmul(g, bt)
    dB = torch.matmul(at, g)
    ab, aa, ag = bt.abs(), at.abs(), g.abs() + gt
    return {"dA": (dA, torch.matmul(gt, ab) + product_tolerance(torch.matmul(ag, ab), N)),
            "dB": (dB, torch.matmul(aa, gt) + product_tolerance(torch.matmul(aa, ag), M)),
            "dbias": (g.sum(-2), gt.sum(-2) + product_tolerance(ag.sum(-2), M))}


def loss_grad(X, W, target, g=None, ignore=-100):
    """{"loss", "lse", "dX", "dW"} each (value, tolerance), for targets that
    are in range or ignored."""
    x, w = X.double(), W.double()
    T, K = x.shape
    V = w.shape[0]
    logits, S = product(x, w.t())
    tol = product_tolerance(S, K)
    lse = torch.logsumexp(logits, 1)
    # A logit's error d moves exp(logit - m) by d relatively, and so the
    # weighted mean of the errors moves lse; then the difference, exponential
    # (4 steps and its argument's rounding) and the sum of V terms, of which
    # the logarithm is taken; the last sum rounds lse itself.
    p = torch.exp(logits - lse[:, None])
    small = 8 * U + 2 * U * logits.abs().amax(1)
    lse_tol = (p * tol).sum(1) + small + min(V, 8 * math.sqrt(V)) * U + 4 * U * (lse.abs() + 1)
    valid = target != ignore
    at = torch.where(valid, target, 0)[:, None]
    loss = torch.where(valid, lse - logits.gather(1, at)[:, 0], 0.0)
    loss_tol = torch.where(valid, lse_tol + tol.gather(1, at)[:, 0] + U * loss.abs(), 0.0)
    g = torch.ones(T, dtype=torch.float64, device=x.device) if g is None else g.double()
    g = torch.where(valid, g, 0.0)
    hot = torch.zeros_like(p).scatter_(1, at, 1.0)
    P = (p - hot) * g[:, None]
    p_tol = (p * (tol + lse_tol[:, None] + 8 * U + U * (logits - lse[:, None]).abs()) + 2 * U * (p - hot).abs()) \
        * g.abs()[:, None]
    xs = torch.where(valid[:, None], x, 0.0)  # (an ignored token's x takes no part)
    aP = P.abs() + p_tol
    Pt = P.t().contiguous()
    return {"loss": (loss, loss_tol), "lse": (lse, lse_tol),
            "dX": (torch.matmul(P, w), torch.matmul(p_tol, w.abs()) + product_tolerance(torch.matmul(aP, w.abs()), V)),
            "dW": (torch.matmul(Pt, xs), torch.matmul(p_tol.t().contiguous(), xs.abs())
                   + product_tolerance(torch.matmul(aP.t().contiguous(), xs.abs()), T + 16))}


def check(got, want, tol, what=""):
    """Every element within its tolerance; NaN and infinities where the oracle has them."""
    got = got.double()
    want, tol = want.to(got.device), tol.to(got.device)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    odd = ~torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    assert bool(same[odd].all()), f"{what}: infinities or NaN differ"
    err = torch.where(odd, 0.0, (got - want).abs())
    bad = ~(err <= tol) & ~odd
    if bool(bad.any()):
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got[i].item()!r} for {want[i].item()!r}, tolerance {tol[i].item():.3e}")
