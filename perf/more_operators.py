"""The operators of a linear layer with its epilogue, and of the loss that ends
a network, each with its gradient, for measurement.  Everything is FP32.

Kinds of case:
  linear       y = act(x W^T + bias) + residual, with z = x W^T + bias kept
               where a backward pass will need it
  linear_grad  of y's gradient dy: dz = dy act'(z), dx = dz W, dw = dz^T x,
               dbias = the sum of dz over rows
  loss         softmax cross entropy of tokens over a vocabulary, the logits
               being x W^T: loss_t = lse_t - logit_{t, target}, lse_t the
               logarithm of the sum of exponentials
  loss_grad    the same with dx and dw, the gradients of sum_t g_t loss_t

W is stored as layers hold it, a row an output (a word of the vocabulary), or
("stored": "in_out") a row an input.  A target of -100 takes no part: its loss
and gradient are zero.
"""

import math

import torch

own = False

ACTIVATIONS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
IGNORED = -100


def _linear(name, M, N, K, act, bias=True, residual=False, keep=False, stored="out_in"):
    return {"name": name, "kind": "linear", "M": M, "N": N, "K": K, "activation": act, "bias": bias,
            "residual": residual, "keep": keep, "stored": stored}


def _grad(name, M, N, K, act, stored="out_in"):
    return {"name": name, "kind": "linear_grad", "M": M, "N": N, "K": K, "activation": act, "stored": stored}


def _loss(name, kind, T, V, K):
    return {"name": name, "kind": kind, "T": T, "V": V, "K": K}


def listed():
    return [
        # one token through a feed-forward up-projection: reading W is the work
        _linear("linear_token", 1, 14336, 4096, "silu"),
        # a small batch of decoded tokens, an odd number, through the down-projection, added to its input
        _linear("linear_batch", 37, 4096, 14336, "none", residual=True),
        # no size a multiple of a tile, rows that no vector load divides
        _linear("linear_ragged", 1000, 1023, 777, "gelu_tanh", residual=True, stored="in_out"),
        # the feed-forward up-projection of 8192 tokens in training
        _linear("linear_ffn", 8192, 14336, 4096, "gelu", keep=True),
        # a small layer's backward pass: launches and latency
        _grad("linear_grad_small", 256, 256, 256, "relu"),
        # odd sizes in every direction
        _grad("linear_grad_ragged", 1000, 1023, 777, "silu", stored="in_out"),
        # a training step of a square layer
        _grad("linear_grad_square", 4096, 4096, 4096, "gelu"),
        # one token scored against a vocabulary: reading W is the work
        _loss("loss_token", "loss", 1, 32768, 4096),
        # a prompt scored: its perplexity
        _loss("loss_prompt", "loss", 2048, 32768, 4096),
        # a few rows of a small classifier in training
        _loss("loss_grad_small", "loss_grad", 64, 1000, 256),
        # odd sizes in every direction
        _loss("loss_grad_ragged", "loss_grad", 517, 32003, 1001),
        # a training step over a large vocabulary
        _loss("loss_grad_vocabulary", "loss_grad", 4096, 131072, 2048),
    ]


def _size(rng, lo, hi):
    """Log-uniform, odd sizes as likely as round ones."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 64:
        n = n // 32 * 32
    return max(lo, min(hi, n))


def draw(rng):
    kind = rng.choice(["linear", "linear_grad", "loss", "loss_grad"])
    while True:
        if kind.startswith("linear"):
            c = {"kind": kind, "M": _size(rng, 1, 8192), "N": _size(rng, 64, 14336), "K": _size(rng, 64, 14336),
                 "activation": rng.choice(ACTIVATIONS), "stored": rng.choice(["out_in", "in_out"])}
            most = 8192 * 14336 * 4096 if kind == "linear" else 4096 ** 3
            if c["M"] * c["N"] * c["K"] > most:
                continue
            if kind == "linear":
                c.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, keep=rng.random() < 0.3)
            return c
        c = {"kind": kind, "T": _size(rng, 1, 4096), "V": _size(rng, 500, 131072), "K": _size(rng, 64, 4096)}
        if c["T"] * c["V"] * c["K"] <= (2048 * 32768 * 4096 if kind == "loss" else 4096 * 131072 * 2048):
            return c


# ---- inputs ------------------------------------------------------------------

def _activations(g, rows, cols):
    """Normal, a few columns much larger than the rest, the last row of a
    batch padding (zeros)."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    gain = torch.exp(0.3 * torch.randn(cols, generator=g, device="cuda"))
    gain *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.005, 10.0, 1.0)
    x *= gain
    if rows >= 16:
        x[-1] = 0.0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    K = case["K"]
    if case["kind"] in ("linear", "linear_grad"):
        M, N = case["M"], case["N"]
        s["x"] = _activations(g, M, K)
        w = torch.randn(*((N, K) if case["stored"] == "out_in" else (K, N)), generator=g, device="cuda")
        s["w"] = w.mul_(1.0 / math.sqrt(K))
        if case["kind"] == "linear":
            s["bias"] = torch.randn(N, generator=g, device="cuda") * 0.1 if case["bias"] else None
            s["residual"] = torch.randn(M, N, generator=g, device="cuda") if case["residual"] else None
        else:
            s["z"] = torch.randn(M, N, generator=g, device="cuda") * 1.5
            s["dy"] = _activations(g, M, N) * 1e-3
        return s
    T, V = case["T"], case["V"]
    s["x"] = _activations(g, T, K)
    s["w"] = torch.randn(V, K, generator=g, device="cuda").mul_(1.5 / math.sqrt(K))
    s["target"] = torch.randint(0, V, (T,), generator=g, device="cuda")
    ignored = torch.rand(T, generator=g, device="cuda") < 0.1
    ignored[0] = False
    s["target"] = torch.where(ignored, IGNORED, s["target"])
    if case["kind"] == "loss_grad":  # the mean over the tokens that take part
        s["g"] = torch.full((T,), 1.0, device="cuda") / (~ignored).sum()
    return s


# ---- the plain forms: elementary operations in 32 bits -------------------------

_C = math.sqrt(2.0 / math.pi)


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_C * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z * _sigmoid(z)
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(_C * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C * (1.0 + 3.0 * 0.044715 * z * z)
    if name == "silu":
        p = _sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _plain(s):
    case, x, w = s["case"], s["x"], s["w"]
    kind = case["kind"]
    if kind == "linear":
        z = x @ (w.t() if case["stored"] == "out_in" else w)
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(case["activation"], z)
        if s["residual"] is not None:
            y = y + s["residual"]
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    if kind == "linear_grad":
        dz = s["dy"] * _act_slope(case["activation"], s["z"])
        if case["stored"] == "out_in":
            dx, dw = dz @ w, dz.t() @ x
        else:
            dx, dw = dz @ w.t(), x.t() @ dz
        return {"dx": dx, "dw": dw, "dbias": dz.sum(0)}
    logits = x @ w.t()
    top = logits.max(dim=1).values
    e = torch.exp(logits - top[:, None])
    total = e.sum(1)
    lse = top + torch.log(total)
    valid = s["target"] != IGNORED
    at = torch.where(valid, s["target"], 0)
    loss = torch.where(valid, lse - logits.gather(1, at[:, None])[:, 0], 0.0)
    if kind == "loss":
        return {"loss": loss, "lse": lse}
    g = torch.where(valid, s["g"], 0.0)
    p = e * (g / total)[:, None]
    p.scatter_add_(1, at[:, None], -g[:, None])
    return {"loss": loss, "lse": lse, "dx": p @ w, "dw": p.t() @ x}


# ---- the framework's calls ------------------------------------------------------

def _own(s):
    from dense_fp32_gemm_row_amd import binding as b

    case, x, w = s["case"], s["x"], s["w"]
    kind = case["kind"]
    if kind == "linear":
        z = torch.empty(case["M"], case["N"], device=x.device) if case["keep"] else None
        y = b.gemm_fused(x, w.t() if case["stored"] == "out_in" else w, bias=s["bias"],
                         activation=case["activation"], residual=s["residual"], pre=z)
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    if kind == "linear_grad":
        out_in = case["stored"] == "out_in"
        dx, dw, dbias = b.gemm_fused_grad(s["dy"], x, w.t() if out_in else w, pre=s["z"],
                                          activation=case["activation"], dbias=True)
        return {"dx": dx, "dw": dw.t() if out_in else dw, "dbias": dbias}
    if kind == "loss":
        loss, lse = b.cross_entropy(x, w, s["target"], ignore_index=IGNORED)
        return {"loss": loss, "lse": lse}
    loss, lse, dx, dw = b.cross_entropy_grad(x, w, s["target"], s["g"], ignore_index=IGNORED)
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    kind, K = case["kind"], case["K"]
    if kind in ("linear", "linear_grad"):
        M, N = case["M"], case["N"]
        if kind == "linear":
            sheets = 1 + case["residual"] + case["keep"]  # M x N matrices read or written
            return {"bytes": 4 * (M * K + N * K + sheets * M * N + case["bias"] * N), "flops": 2 * M * N * K}
        return {"bytes": 4 * (2 * M * K + 2 * N * K + 2 * M * N + N), "flops": 4 * M * N * K}
    T, V = case["T"], case["V"]
    if kind == "loss":
        return {"bytes": 4 * (T * K + V * K) + 16 * T, "flops": 2 * T * V * K}
    return {"bytes": 8 * (T * K + V * K) + 20 * T, "flops": 6 * T * V * K}


# ---- the definition in 64 bits -------------------------------------------------------

def _normal_cdf(z):
    return 0.5 * torch.special.erfc(-z / 2.0 ** 0.5)


def _value64(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp_min(0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return z * _normal_cdf(z)
    # (1 + tanh u) / 2 is the logistic function of 2 u
    return z / (1.0 + torch.exp(-2.0 * (2.0 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))


def _slope64(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, 1.0, 0.0).double()
    if name == "gelu":
        return _normal_cdf(z) + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    if name == "silu":
        u, du = z, 1.0
    else:
        u = 2.0 * (2.0 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)
        du = 2.0 * (2.0 / math.pi) ** 0.5 * (1.0 + 0.134145 * z ** 2)
    q = 1.0 / (1.0 + torch.exp(-u))
    return q + z * q * (1.0 - q) * du


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    x, w = s["x"].double(), s["w"].double()
    if kind in ("linear", "linear_grad") and case["stored"] == "out_in":
        w = w.t()  # K x N from here on
    if kind == "linear":
        z = torch.matmul(x, w)
        if case["bias"]:
            z += s["bias"].double()
        y = _value64(case["activation"], z)
        if case["residual"]:
            y = y + s["residual"].double()
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    if kind == "linear_grad":
        dz = s["dy"].double() * _slope64(case["activation"], s["z"].double())
        dw = torch.matmul(x.t(), dz)
        return {"dx": torch.matmul(dz, w.t()), "dw": dw.t() if case["stored"] == "out_in" else dw,
                "dbias": dz.sum(dim=0)}
    scores = torch.matmul(x, w.t())
    lse = torch.logsumexp(scores, dim=1)
    keep = s["target"] >= 0
    rows = torch.nonzero(keep)[:, 0]
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - scores[rows, s["target"][rows]]
    if kind == "loss":
        return {"loss": loss, "lse": lse}
    scores.sub_(lse[:, None]).exp_()
    scores[rows, s["target"][rows]] -= 1.0
    scores *= (s["g"].double() * keep)[:, None]
    return {"loss": loss, "lse": lse, "dx": torch.matmul(scores, w), "dw": torch.matmul(scores.t(), x)}
