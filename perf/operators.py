"""The operators of microscaled 4-bit floating point (MXFP4) as they are used, for measurement.

A matrix in this format holds, for every 32 values along a row, one power of
two (a byte e, 2^(e - 127)) and 32 four-bit codes (sign, two exponent bits,
one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6), two to a byte, low half first.

Kinds of case:
  round_trip   quantise an FP32 matrix and read it back, along its rows or
               along its rows and its columns
  product      C = A B^T, both operands in the format (a batch: experts)
  weight       C = X W^T, X in FP32, W in the format (W is N x K)
  weight_grad  dX = dY W, the gradient of `weight` with respect to X
  train        a linear layer's step: y = x w^T, dx = dy w, dw = dy^T x, with
               every operand quantised along the axis that the product sums
"""

import math

import torch

own = False

BLOCK = 32


def listed():
    return [
        # one token's activations on their way through the format: latency alone
        {"name": "round_trip_token", "kind": "round_trip", "rows": 1, "cols": 4096, "both": False},
        # the activations that enter a feed-forward layer, 8192 tokens
        {"name": "round_trip_ffn", "kind": "round_trip", "rows": 8192, "cols": 4096, "both": False},
        # an odd-sized matrix along both axes, as a training step needs it
        {"name": "round_trip_ragged", "kind": "round_trip", "rows": 1000, "cols": 777, "both": True},
        # the small square product
        {"name": "product_256", "kind": "product", "batch": 1, "M": 256, "N": 256, "K": 256},
        # no size a multiple of a tile or of a block of 32
        {"name": "product_ragged", "kind": "product", "batch": 1, "M": 1000, "N": 1023, "K": 777},
        # the feed-forward up-projection, 8192 tokens
        {"name": "product_ffn", "kind": "product", "batch": 1, "M": 8192, "N": 14336, "K": 4096},
        # 64 experts of 1024 tokens each
        {"name": "product_experts", "kind": "product", "batch": 64, "M": 1024, "N": 1024, "K": 1024},
        # few output tiles, long sums
        {"name": "product_deepk", "kind": "product", "batch": 1, "M": 1024, "N": 1024, "K": 65536},
        # one token through a stored layer: reading the weights is the work
        {"name": "weight_token", "kind": "weight", "M": 1, "N": 14336, "K": 4096},
        # a small batch of decoded tokens, an odd number
        {"name": "weight_batch", "kind": "weight", "M": 37, "N": 14336, "K": 4096},
        # a prompt through a stored layer, and its gradient
        {"name": "weight_grad_prompt", "kind": "weight_grad", "M": 4096, "N": 4096, "K": 14336},
        # a training step of one linear layer
        {"name": "train_step", "kind": "train", "M": 4096, "N": 4096, "K": 4096},
    ]


def _size(rng, lo, hi):
    """Log-uniform, odd sizes as likely as round ones."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 64:
        n = n // 32 * 32
    return max(lo, min(hi, n))


def draw(rng):
    kind = rng.choice(["round_trip", "product", "weight", "weight_grad", "train"])
    if kind == "round_trip":
        both = rng.random() < 0.5
        return {"kind": kind, "rows": _size(rng, 1, 8192 if not both else 5000),
                "cols": _size(rng, 32, 4096), "both": both}
    if kind == "product":
        batch = rng.choice([1, 1, 1, _size(rng, 2, 64)])
        while True:
            M, N, K = _size(rng, 1, 8192), _size(rng, 256, 14336), _size(rng, 256, 16384)
            if batch * M * N * K <= 8192 * 14336 * 4096 and batch * max(M * K, N * K, M * N) <= 1 << 28:
                return {"kind": kind, "batch": batch, "M": M, "N": N, "K": K}
    while True:
        M, N, K = _size(rng, 1, 8192), _size(rng, 256, 14336), _size(rng, 256, 14336)
        if kind == "train" and M >= 32 and M * N * K <= 4096 ** 3:
            return {"kind": kind, "M": M, "N": N, "K": K}
        if kind != "train" and M * N * K <= 4096 * 4096 * 14336:
            return {"kind": kind, "M": M, "N": N, "K": K}


# ---- inputs ------------------------------------------------------------------

def _activations(g, rows, cols):
    """Normal, a few columns much larger than the rest, the last row of a
    batch padding (zeros)."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    gain = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    gain = gain * torch.where(torch.rand(cols, generator=g, device="cuda") < 0.005, 30.0, 1.0)
    x *= gain
    if rows >= 16:
        x[-1] = 0.0
    return x


def _stored(g, batch, rows, cols, scale, outliers):
    """A matrix as a checkpoint holds it: (codes, scales).  A row of codes is
    whole blocks of 16 bytes, a row of scales whole words of 4 bytes."""
    nb = -(-cols // BLOCK)
    w = torch.randn(batch * rows, nb * BLOCK, generator=g, device="cuda") * scale
    if outliers:
        w *= torch.exp(0.5 * torch.randn(nb * BLOCK, generator=g, device="cuda"))
    w[:, cols:] = 0.0
    w = w.view(batch * rows, nb, BLOCK)
    e = torch.floor(torch.log2(w.abs().amax(-1).clamp_min(1e-30))) - 2
    v = w / torch.exp2(e)[..., None]
    m = torch.bucketize(v.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda"))
    codes = (m + 8 * (v < 0)).to(torch.uint8).view(batch * rows, nb * 16, 2)
    codes = codes[..., 0] | (codes[..., 1] << 4)
    scales = torch.zeros(batch * rows, -(-nb // 4) * 4, dtype=torch.uint8, device="cuda")
    scales[:, :nb] = (e + 127).to(torch.uint8)
    if batch > 1:
        return codes.view(batch, rows, -1), scales.view(batch, rows, -1)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    s = {"kind": kind, "case": case}
    if kind == "round_trip":
        s["x"] = _activations(g, case["rows"], case["cols"])
        s["both"] = case["both"]
        return s
    M, N, K = case["M"], case["N"], case["K"]
    if kind == "product":
        s["a"] = _stored(g, case["batch"], M, K, 1.0, True)
        s["b"] = _stored(g, case["batch"], N, K, 0.02, False)
    elif kind == "weight":
        s["x"] = _activations(g, M, K)
        s["w"] = _stored(g, 1, N, K, 0.02, False)
    elif kind == "weight_grad":
        s["x"] = _activations(g, M, K) * 1e-3
        s["w"] = _stored(g, 1, K, N, 0.02, False)
    else:
        s["x"] = _activations(g, M, K)
        s["w"] = torch.randn(N, K, generator=g, device="cuda") * 0.02
        s["dy"] = _activations(g, M, N) * 1e-3
    return s


# ---- the plain forms: elementary operations in 32 bits -------------------------

def _values(codes, scales, cols):
    """The FP32 values that (codes, scales) stand for."""
    nb = -(-cols // BLOCK)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=codes.device)
    c = codes[..., : nb * 16]
    v = torch.stack((table[(c & 15).int()], table[(c >> 4).int()]), dim=-1)
    v = v.reshape(*c.shape[:-1], nb, BLOCK)
    s = torch.ldexp(torch.ones((), device=codes.device), scales[..., :nb].int() - 127)
    return (v * s[..., None]).reshape(*c.shape[:-1], nb * BLOCK)[..., :cols]


def _rounded(x):
    """x as the format holds it, blocks along the last axis, in FP32."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    p = torch.zeros(rows, nb * BLOCK, device=x.device)
    p[:, :cols] = x
    p = p.view(rows, nb, BLOCK)
    amax = p.abs().amax(-1, keepdim=True)
    e = torch.frexp(amax).exponent - 3  # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, -127).clamp(-127, 127)
    v = torch.ldexp(p, -e)
    m = v.abs()
    q = torch.where(m < 2, torch.round(m * 2) / 2, torch.where(m < 4, torch.round(m), torch.round(m / 2) * 2))
    q = torch.copysign(q.clamp(max=6.0), v)
    return torch.ldexp(q, e).view(rows, nb * BLOCK)[:, :cols]


def _plain(s):
    kind, case = s["kind"], s["case"]
    if kind == "round_trip":
        if s["both"]:
            return {"values": _rounded(s["x"]), "values_t": _rounded(s["x"].t())}
        return {"values": _rounded(s["x"])}
    K = case["K"]
    if kind == "product":
        return {"c": _values(*s["a"], K) @ _values(*s["b"], K).transpose(-1, -2)}
    if kind == "weight":
        return {"c": s["x"] @ _values(*s["w"], K).t()}
    if kind == "weight_grad":
        return {"dx": s["x"] @ _values(*s["w"], case["N"])}
    x, w, dy = s["x"], s["w"], s["dy"]
    return {"y": _rounded(x) @ _rounded(w).t(),
            "dx": _rounded(dy) @ _rounded(w.t()).t(),
            "dw": _rounded(dy.t()) @ _rounded(x.t()).t()}


# ---- the framework's calls ------------------------------------------------------

def _own(s):
    from dense_fp32_gemm_row_amd import binding as b

    kind, case = s["kind"], s["case"]
    if kind == "round_trip":
        if s["both"]:
            q, qt = b.mxfp4_quantize_both(s["x"])
            return {"values": b.mxfp4_dequantize(q), "values_t": b.mxfp4_dequantize(qt)}
        return {"values": b.mxfp4_dequantize(b.mxfp4_quantize(s["x"]))}
    K = case["K"]
    if kind == "product":
        return {"c": b.gemm_mxfp4(b.Mxfp4(*s["a"], K), b.Mxfp4(*s["b"], K))}
    if kind == "weight":
        return {"c": b.gemm_mxfp4_weight(s["x"], b.Mxfp4(*s["w"], K))}
    if kind == "weight_grad":
        return {"dx": b.gemm_mxfp4_weight(s["x"], b.Mxfp4(*s["w"], case["N"]), op=b.OP_N)}
    x, xt = b.mxfp4_quantize_both(s["x"])
    w, wt = b.mxfp4_quantize_both(s["w"])
    dy, dyt = b.mxfp4_quantize_both(s["dy"])
    return {"y": b.gemm_mxfp4(x, w), "dx": b.gemm_mxfp4(dy, wt), "dw": b.gemm_mxfp4(dyt, xt)}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    kind = case["kind"]
    if kind == "round_trip":
        n = case["rows"] * case["cols"]
        forms = 2 if case["both"] else 1
        return {"bytes": 4 * n * (1 + forms), "flops": 2 * n * forms}
    M, N, K = case["M"], case["N"], case["K"]
    held = 17 / 32  # bytes of a value in the format, its share of the scale included
    if kind == "product":
        return {"bytes": case["batch"] * (held * (M + N) * K + 4 * M * N), "flops": 2 * case["batch"] * M * N * K}
    if kind == "train":
        return {"bytes": 8 * (M * K + N * K + M * N), "flops": 6 * M * N * K}
    return {"bytes": 4 * M * K + held * N * K + 4 * M * N, "flops": 2 * M * N * K}


# ---- the definition in 64 bits -------------------------------------------------------

def _read64(stored, cols):
    codes, scales = (t.long() for t in stored)
    k = torch.arange(cols, device=codes.device)
    nibble = (codes[..., k // 2] >> (4 * (k % 2))) & 15
    exponent, mantissa = (nibble >> 1) & 3, (nibble & 1).double()
    magnitude = torch.where(exponent == 0, 0.5 * mantissa, (1 + 0.5 * mantissa) * torch.exp2(exponent.double() - 1))
    sign = 1.0 - 2.0 * (nibble >> 3).double()
    return sign * magnitude * torch.exp2(scales[..., k // BLOCK].double() - 127)


def _round64(x):
    """Nearest value of the format, ties to the even code, blocks along the last axis."""
    x = x.double()
    rows, cols = x.shape
    pad = torch.nn.functional.pad(x, (0, -cols % BLOCK)).reshape(-1, BLOCK)
    top = pad.abs().max(dim=1).values
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.where(top > 0, top, 2.0 ** -130))) - 2, min=-127))
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device, dtype=torch.float64)
    middle = (grid[1:] + grid[:-1]) / 2
    v = pad.abs() / step[:, None]
    low, high = torch.bucketize(v, middle), torch.bucketize(v, middle, right=True)
    code = torch.where(low % 2 == 0, low, high)
    return (torch.sign(pad) * grid[code] * step[:, None]).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "round_trip":
        out = {"values": _round64(s["x"])}
        if case["both"]:
            out["values_t"] = _round64(s["x"].t())
        return out
    K = case["K"]
    if kind == "product":
        A, B = _read64(s["a"], K), _read64(s["b"], K)
        return {"c": torch.matmul(A, B.transpose(-1, -2).contiguous())}
    if kind == "weight":
        return {"c": torch.matmul(s["x"].double(), _read64(s["w"], K).t())}
    if kind == "weight_grad":
        return {"dx": torch.matmul(s["x"].double(), _read64(s["w"], case["N"]))}
    x, w, dy = s["x"], s["w"], s["dy"]
    return {"y": torch.matmul(_round64(x), _round64(w).t()),
            "dx": torch.matmul(_round64(dy), _round64(w.t()).t()),
            "dw": torch.matmul(_round64(dy.t()), _round64(x.t()).t())}
