"""Cases that measure the linear and layer-norm operators on block-quantized weights.

Four operators are measured, on the layer shapes this repository's workloads
use and on odd ones around them:

- ``linear``: y = x W^T, W block-quantized (int4 or int8 codes, one binary32
  scale per block of the flat weight buffer), from one token to a long prompt;
- ``linear_grad``: its input gradient dx = dy W from the same codes;
- ``layer_norm``: y = (x - mean) * rstd * weight + bias, with mean and rstd;
- ``layer_norm_grad``: dx, dweight and dbias.

``run`` computes them with elementary torch operations in binary32 when
``own`` is false, and with the library's calls when it is true. ``exact``
holds their definitions in binary64.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


# ---- cases ---------------------------------------------------------------------

def _linear(name, op, tokens, inf, outf, bits, block, x="bf16", y="bf16"):
    c = {"op": op, "tokens": tokens, "in": inf, "out": outf, "bits": bits, "block": block, "x": x, "y": y}
    return {"name": name, **c} if name else c


def _norm(name, op, rows, width, x="bf16", w="bf16"):
    c = {"op": op, "rows": rows, "width": width, "x": x, "w": w}
    return {"name": name, **c} if name else c


def listed():
    return [
        # decoding one token: the key projection of the 8192-wide grouped-query layer, the smallest call
        _linear("token key int4", "linear", 1, 8192, 1024, 4, 128),
        # decoding one token: the gate projection of the same layer, a stream of 117 MB of codes
        _linear("token gate int4", "linear", 1, 8192, 28672, 4, 128),
        # decoding 16 sequences at once: the down projection from 8-bit weights
        _linear("batch down int8", "linear", 16, 28672, 8192, 8, 512),
        # a ragged prompt through the 11008-wide layer, whose 2048-element blocks straddle rows; binary32 result
        _linear("ragged down int8 fp32", "linear", 333, 11008, 4096, 8, 2048, "bf16", "fp32"),
        # a training batch of 4096 tokens through the gate projection, the largest call
        _linear("prompt gate int4", "linear", 4096, 8192, 28672, 4, 128),
        # backward of a short sequence through the key projection: little work to spread over the GPU
        _linear("grad key int4", "linear_grad", 512, 8192, 1024, 4, 128),
        # backward in binary32 with an odd number of outputs
        _linear("grad ragged int4 fp32", "linear_grad", 77, 4096, 11007, 4, 256, "fp32", "fp32"),
        # backward of a training batch through the query projection from 8-bit weights
        _linear("grad query int8", "linear_grad", 4096, 8192, 8192, 8, 512),
        # one token's normalisation while decoding
        _norm("norm token", "layer_norm", 1, 8192),
        # a training batch's normalisation, forward and backward
        _norm("norm batch", "layer_norm", 8192, 8192),
        _norm("norm grad batch", "layer_norm_grad", 8192, 8192),
        # odd rows and width in binary32: no row starts on a vector boundary
        _norm("norm grad odd fp32", "layer_norm_grad", 1001, 4099, "fp32", "fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "layer_norm", "layer_norm_grad"])
    x = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("linear"):
        while True:
            tokens, inf, outf = _log(rng, 1, 4096), 32 * _log(rng, 4, 640), _log(rng, 64, 28672)
            if rng.random() < 0.5:
                outf = -(-outf // 64) * 64
            block = rng.choice([32, 64, 128, 256, 512, 2048])
            # no dearer than the largest listed case (binary32 products cost several times bf16 ones)
            if (inf * outf) % block == 0 and inf * outf <= 8192 * 28672 and \
                    tokens * inf * outf * (1 if x == "bf16" else 8) <= 4096 * 8192 * 28672:
                break
        y = "fp32" if x == "fp32" else rng.choice(["bf16", "bf16", "fp32"])
        return _linear(None, op, tokens, inf, outf, rng.choice([4, 8]), block, x, y)
    while True:
        rows, width = _log(rng, 1, 16384), _log(rng, 64, 28672)
        if rng.random() < 0.5:
            width = -(-width // 64) * 64
        if rows * width <= 8192 * 8192:
            break
    return _norm(None, op, rows, width, x, rng.choice([x, "fp32"]))


# ---- inputs --------------------------------------------------------------------

def _quantize(w, block, bits):
    """Symmetric absmax codes and scales of a flat binary32 tensor."""
    q = 127 if bits == 8 else 7
    b = w.view(-1, block)
    scales = b.abs().amax(1) / q
    codes = torch.round(b / torch.where(scales > 0, scales, torch.ones_like(scales))[:, None])
    codes = codes.clamp_(-q, q).to(torch.int8).view(-1)
    if bits == 8:
        return codes.view(torch.uint8), scales
    u = codes.view(torch.uint8) & 15
    return u[0::2] | (u[1::2] << 4), scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    xt = DTYPES[case["x"]]
    st = dict(case)
    if case["op"].startswith("linear"):
        outf, inf = case["out"], case["in"]
        # weights as a trained layer holds them: narrow, with a few large channels
        w = normal(outf, inf, std=0.02)
        w[:, :: max(inf // 16, 1)] *= 8.0
        st["codes"], st["scales"] = _quantize(w.view(-1), case["block"], case["bits"])
        del w
        grad = case["op"] == "linear_grad"
        width = outf if grad else inf
        # activations after a normalisation; gradients are smaller by orders of magnitude
        st["a"] = normal(case["tokens"], width, std=1e-3 if grad else 1.0, dtype=xt)
        return st
    rows, width, wt = case["rows"], case["width"], DTYPES[case["w"]]
    # a residual stream: a per-row offset and scale, and some wide channels
    x = normal(rows, width) * (0.5 + torch.rand(rows, 1, generator=g, device="cuda")) + normal(rows, 1, std=0.3)
    x[:, :: max(width // 8, 1)] *= 10.0
    st["a"] = x.to(xt)
    st["weight"], st["bias"] = (1.0 + normal(width, std=0.1)).to(wt), normal(width, std=0.1, dtype=wt)
    if case["op"] == "layer_norm_grad":
        st["dy"] = normal(rows, width, std=1e-2, dtype=xt)
        # what the forward pass kept
        xd = st["a"].double()
        mean = xd.mean(1)
        st["mean"] = mean.float()
        st["rstd"] = (((xd - mean[:, None]) ** 2).mean(1) + EPS).rsqrt().float()
    return st


# ---- one pass ------------------------------------------------------------------

def _plain_weight(st):
    """The weights in binary32, [out, in]."""
    c = st["codes"]
    if st["bits"] == 8:
        q = c.view(torch.int8).float()
    else:
        # bytes hold two's-complement nibbles, the even element in the low one
        n = torch.stack((c & 15, c >> 4), 1).view(-1).float()
        q = torch.where(n > 7, n - 16, n)
    return (q.view(-1, st["block"]) * st["scales"][:, None]).view(st["out"], st["in"])


def _plain_linear(st):
    return (st["a"].float() @ _plain_weight(st).t()).to(DTYPES[st["y"]])


def _plain_linear_grad(st):
    return (st["a"].float() @ _plain_weight(st)).to(DTYPES[st["y"]])


def _plain_norm(st):
    x = st["a"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + EPS)
    y = d * rstd[:, None] * st["weight"].float() + st["bias"].float()
    return {"y": y.to(st["a"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_grad(st):
    dy, rstd = st["dy"].float(), st["rstd"][:, None]
    xhat = (st["a"].float() - st["mean"][:, None]) * rstd
    g = dy * st["weight"].float()
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * rstd
    wt = st["weight"].dtype
    return {"dx": dx.to(st["a"].dtype), "dweight": (dy * xhat).sum(0).to(wt), "dbias": dy.sum(0).to(wt)}


def run(state):
    op = state["op"]
    if not own:
        plain = {"linear": _plain_linear, "linear_grad": _plain_linear_grad, "layer_norm": _plain_norm,
                 "layer_norm_grad": _plain_norm_grad}
        return plain[op](state)
    import block_quantization_codec_amd as z

    if op == "linear":
        return z.linear(state["a"], state["codes"], state["scales"], state["bits"], state["block"], state["out"],
                        dtype=DTYPES[state["y"]])
    if op == "linear_grad":
        return z.linear_grad(state["a"], state["codes"], state["scales"], state["bits"], state["block"],
                             state["in"], dtype=DTYPES[state["y"]])
    if op == "layer_norm":
        y, mean, rstd = z.layer_norm(state["a"], state["weight"], state["bias"], EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dw, db = z.layer_norm_grad(state["dy"], state["a"], state["weight"], state["mean"], state["rstd"])
    return {"dx": dx, "dweight": dw, "dbias": db}


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"].startswith("linear"):
        n = case["out"] * case["in"]
        a, b = (case["in"], case["out"]) if case["op"] == "linear" else (case["out"], case["in"])
        byt = n * case["bits"] // 8 + 4 * (n // case["block"]) + \
            case["tokens"] * (a * size[case["x"]] + b * size[case["y"]])
        return {"bytes": byt, "flops": 2 * case["tokens"] * n}
    r, w, xs, ws = case["rows"], case["width"], size[case["x"]], size[case["w"]]
    if case["op"] == "layer_norm":
        return {"bytes": 2 * r * w * xs + 2 * w * ws + 8 * r, "flops": 8 * r * w}
    return {"bytes": 3 * r * w * xs + 3 * w * ws + 8 * r, "flops": 14 * r * w}


# ---- definitions in binary64 ---------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    a = st["a"].to(torch.float64)
    if case["op"].startswith("linear"):
        outf, inf, bits = case["out"], case["in"], case["bits"]
        # element i of the flat buffer: its code's bits, as a signed number, times the scale of block i // block
        n = torch.arange(outf * inf, device="cuda", dtype=torch.int64)
        raw = st["codes"][n * bits // 8].to(torch.int16)
        if bits == 4:
            raw = torch.bitwise_right_shift(raw, (n % 2 * 4).to(torch.int16)).bitwise_and_(15)
        half = 1 << (bits - 1)
        raw = (raw + half).remainder_(2 * half) - half
        w = raw.double()
        del raw
        w *= st["scales"].double()[n // case["block"]]
        del n
        w = w.view(outf, inf)
        return torch.matmul(a, w.T if case["op"] == "linear" else w)
    weight = st["weight"].to(torch.float64)
    n = case["width"]
    if case["op"] == "layer_norm":
        mean = a.sum(-1) / n
        var = torch.square(a).sum(-1) / n - torch.square(mean)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(st["bias"].double(), (a - mean.unsqueeze(-1)) * rstd.unsqueeze(-1), weight)
        return {"y": y, "mean": mean, "rstd": rstd}
    dy, mean, rstd = st["dy"].double(), st["mean"].double(), st["rstd"].double()
    centred = a - mean.unsqueeze(-1)
    dw = torch.einsum("rw,rw,r->w", dy, centred, rstd)
    # dx_j = rstd (g_j - sum_i g_i / n - c_j rstd^2 sum_i g_i c_i / n),  g = dy * weight, c = x - mean
    g = dy * weight
    first = g.sum(-1) / n
    second = rstd * rstd * (g * centred).sum(-1) / n
    dx = rstd.unsqueeze(-1) * (g - first.unsqueeze(-1) - centred * second.unsqueeze(-1))
    return {"dx": dx, "dweight": dw, "dbias": dy.sum(0)}
