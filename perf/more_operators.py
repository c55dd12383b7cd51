"""Cases that measure the operators around a layer's block-quantized weights.

Three operators are measured with their gradients, on the layer shapes this
repository's workloads use and on odd ones around them:

- ``rms_norm``: the residual stream's sum h = x + residual, its root-mean-square
  norm, and that norm's block-quantized 8-bit codes; ``rms_norm_grad`` its
  backward pass;
- ``linear_adapters``: y = x W^T + s_g (x A_g^T) B_g^T for rows that each name a
  low-rank adapter g or none, W block-quantized; ``linear_adapters_grad`` the
  gradients of x and of every adapter;
- ``linear_grouped``: rows grouped by expert, each group through its own
  block-quantized weight; ``linear_grouped_grad`` its input gradient.

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

def _norm(name, op, rows, width, residual, bits=0, block=0, x="bf16", w="bf16"):
    """residual: whether a residual is added (forward), or a gradient of the sum arrives (backward).
    bits: codes of the norm are asked for in place of the norm itself."""
    c = {"op": op, "rows": rows, "width": width, "residual": residual, "bits": bits, "block": block, "x": x, "w": w}
    return {"name": name, **c} if name else c


def _adapters(name, op, rows, inf, outf, bits, block, adapters, rank, requests, x="bf16", w="bf16", y="bf16"):
    """requests: the rows are that many neighbouring runs, each with an adapter of its own choice (or none)."""
    c = {"op": op, "rows": rows, "in": inf, "out": outf, "bits": bits, "block": block, "adapters": adapters,
         "rank": rank, "requests": requests, "x": x, "w": w, "y": y}
    return {"name": name, **c} if name else c


def _grouped(name, op, rows, inf, outf, bits, block, groups, x="bf16", y="bf16"):
    c = {"op": op, "rows": rows, "in": inf, "out": outf, "bits": bits, "block": block, "groups": groups, "x": x,
         "y": y}
    return {"name": name, **c} if name else c


def listed():
    return [
        # decoding one token: the smallest call
        _norm("norm token", "rms_norm", 1, 8192, True),
        # a training batch whose normed activations go on as 8-bit codes
        _norm("norm batch codes", "rms_norm", 8192, 8192, True, 8, 128),
        # backward of that batch, with the gradient that skips the layer
        _norm("norm grad batch", "rms_norm_grad", 8192, 8192, True),
        # odd rows and width in binary32: no row starts on a vector boundary
        _norm("norm grad odd fp32", "rms_norm_grad", 1001, 4099, False, 0, 0, "fp32", "fp32"),
        # decoding 48 requests, which choose among 32 adapters, through the gate projection
        _adapters("adapters requests", "linear_adapters", 48, 8192, 28672, 4, 128, 32, 64, 48),
        # prompts of 5 requests side by side through the gate projection, the largest call
        _adapters("adapters prompts", "linear_adapters", 4096, 8192, 28672, 4, 128, 4, 64, 5),
        # training one adapter beside the query projection: backward of a batch of 4096 tokens
        _adapters("adapters grad train", "linear_adapters_grad", 4096, 8192, 8192, 8, 512, 1, 64, 1),
        # backward in binary32 with an odd number of outputs, three adapters and some rows without one
        _adapters("adapters grad ragged fp32", "linear_adapters_grad", 333, 4096, 11007, 4, 256, 3, 16, 7,
                  "fp32", "fp32", "fp32"),
        # decoding 32 tokens over 16 experts: few rows each, some experts with none
        _grouped("experts decode", "linear_grouped", 32, 4096, 11008, 4, 128, 16),
        # a prompt of 8192 tokens over 16 experts of unequal load
        _grouped("experts prompt", "linear_grouped", 8192, 4096, 11008, 4, 128, 16),
        # backward of a training batch over 8 experts from 8-bit weights
        _grouped("experts grad train", "linear_grouped_grad", 4096, 4096, 11008, 8, 512, 8),
        # backward in binary32, blocks that straddle rows, an odd number of outputs
        _grouped("experts grad odd fp32", "linear_grouped_grad", 300, 2080, 1407, 4, 32, 5, "fp32", "fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rms_norm", "rms_norm_grad", "linear_adapters", "linear_adapters_grad", "linear_grouped",
                     "linear_grouped_grad"])
    x = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("rms_norm"):
        bits = rng.choice([0, 8]) if op == "rms_norm" else 0
        block = rng.choice([32, 64, 128, 256]) if bits else 0
        while True:
            rows, width = _log(rng, 1, 16384), _log(rng, 64, 28672)
            if bits:
                width = -(-width // block) * block
            elif rng.random() < 0.5:
                width = -(-width // 64) * 64
            if rows * width <= 8192 * 8192:
                break
        return _norm(None, op, rows, width, rng.random() < 0.6, bits, block, x, rng.choice([x, "fp32"]))
    y = "fp32" if x == "fp32" else rng.choice(["bf16", "bf16", "fp32"])
    bits, block = rng.choice([4, 8]), rng.choice([32, 64, 128, 256, 512])
    # no dearer than the largest listed case (binary32 products cost several times bf16 ones)
    dear = 1 if x == "bf16" and y == "bf16" else 3 if x == "bf16" else 8
    if op.startswith("linear_adapters"):
        while True:
            rows, inf, outf = _log(rng, 1, 4096), 32 * _log(rng, 4, 320), _log(rng, 64, 28672)
            if rng.random() < 0.5:
                outf = -(-outf // 64) * 64
            adapters, rank = _log(rng, 1, 32), 8 * _log(rng, 1, 16)
            if (inf * outf) % block == 0 and inf * outf <= 8192 * 28672 and adapters * rank <= 2048 and \
                    rows * inf * outf * dear <= 4096 * 8192 * 28672:
                break
        requests = _log(rng, 1, rows)
        w = x if rng.random() < 0.7 else "fp32"
        return _adapters(None, op, rows, inf, outf, bits, block, adapters, rank, requests, x, w, y)
    while True:
        rows, inf, outf, groups = _log(rng, 1, 8192), 32 * _log(rng, 4, 256), _log(rng, 64, 11008), _log(rng, 1, 64)
        if rng.random() < 0.5:
            outf = -(-outf // 64) * 64
        if (inf * outf) % block == 0 and groups * inf * outf <= 16 * 4096 * 11008 and \
                rows * inf * outf * dear <= 8192 * 4096 * 11008:
            break
    return _grouped(None, op, rows, inf, outf, bits, block, groups, x, y)


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
    host = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    xt = DTYPES[case["x"]]
    st = dict(case)
    rows = case["rows"]
    grad = case["op"].endswith("_grad")
    if case["op"].startswith("rms_norm"):
        width, wt = case["width"], DTYPES[case["w"]]
        # a residual stream: rows of different scale, and some wide channels
        h = normal(rows, width) * (0.5 + torch.rand(rows, 1, generator=g, device="cuda"))
        h[:, :: max(width // 8, 1)] *= 10.0
        st["weight"] = (1.0 + normal(width, std=0.1)).to(wt)
        if not grad:
            st["a"] = normal(rows, width, std=0.5, dtype=xt) if case["residual"] else h.to(xt)
            st["h"] = h.to(xt) if case["residual"] else None
            return st
        st["a"] = h.to(xt)
        st["dy"] = normal(rows, width, std=1e-2, dtype=xt)
        st["dsum"] = normal(rows, width, std=1e-2, dtype=xt) if case["residual"] else None
        # what the forward pass kept
        st["rstd"] = (st["a"].double().square().mean(1) + EPS).rsqrt().float()
        return st
    outf, inf, bits, block = case["out"], case["in"], case["bits"], case["block"]
    groups = case.get("groups", 1)
    codes, scales = [], []
    for _ in range(groups):
        # weights as a trained layer holds them: narrow, with a few large channels
        w = normal(outf, inf, std=0.02)
        w[:, :: max(inf // 16, 1)] *= 8.0
        c, s = _quantize(w.view(-1), block, bits)
        codes.append(c)
        scales.append(s)
        del w
    st["codes"], st["scales"] = torch.cat(codes), torch.cat(scales)
    # activations after a normalisation; gradients are smaller by orders of magnitude
    if grad:
        st["dy"] = normal(rows, outf, std=1e-3, dtype=xt)
    if "groups" in case:
        if not grad:
            st["a"] = normal(rows, inf, dtype=xt)
        # experts of unequal load; with few rows some have none
        load = torch.softmax(0.8 * torch.randn(groups, generator=host), 0)
        count = torch.bincount(torch.multinomial(load, rows, True, generator=host), minlength=groups)
        st["offsets"] = torch.cat((torch.zeros(1, dtype=torch.int64), count.cumsum(0))).to(torch.int32).cuda()
        st["most"] = int(count.max())
        return st
    st["a"] = normal(rows, inf, dtype=xt)
    n, rank, wt = case["adapters"], case["rank"], DTYPES[case["w"]]
    st["A"], st["B"] = normal(n, rank, inf, std=inf ** -0.5, dtype=wt), normal(n, outf, rank, std=0.05, dtype=wt)
    st["scaling"] = 0.5 + 1.5 * torch.rand(n, generator=g, device="cuda")
    if n == 1 and case["requests"] == 1:
        st["ids"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    else:
        # each request chooses an adapter, or none (one choice in n + 1)
        chosen = torch.randint(-1, n, (case["requests"],), generator=host)
        ends = torch.sort(torch.randperm(rows - 1, generator=host)[:case["requests"] - 1] + 1).values
        which = torch.zeros(rows, dtype=torch.int64)
        which[ends] = 1
        st["ids"] = chosen[which.cumsum(0)].to(torch.int32).cuda()
    if grad:  # what the forward pass kept: s_g A_g x of each row
        every = (st["a"].double() @ st["A"].double().view(n * rank, inf).t()).view(rows, n, rank)
        at = st["ids"].long().clamp(min=0)
        t = every[torch.arange(rows, device="cuda"), at] * st["scaling"].double()[at, None]
        st["reduced"] = torch.where(st["ids"][:, None] >= 0, t, 0.0).float()
    return st


# ---- one pass ------------------------------------------------------------------

def _values(c, scales, bits, block):
    """Codes as the binary32 values they stand for, flat."""
    if bits == 8:
        q = c.view(torch.int8).float()
    else:
        # bytes hold two's-complement nibbles, the even element in the low one
        n = torch.stack((c & 15, c >> 4), 1).view(-1).float()
        q = torch.where(n > 7, n - 16, n)
    return (q.view(-1, block) * scales[:, None]).view(-1)


def _plain_weight(st):
    """The weights in binary32, [out, in], or [groups, out, in]."""
    w = _values(st["codes"], st["scales"], st["bits"], st["block"])
    return w.view(st.get("groups", 1), st["out"], st["in"]) if "groups" in st else w.view(st["out"], st["in"])


def _plain_norm(st):
    xt = st["a"].dtype
    h = st["a"] if st["h"] is None else (st["a"].float() + st["h"].float()).to(xt)
    f = h.float()
    rstd = torch.rsqrt((f * f).mean(1) + EPS)
    y = f * rstd[:, None] * st["weight"].float()
    out = {"rstd": rstd}
    if st["h"] is not None:
        out["sum"] = h
    if not st["bits"]:
        out["y"] = y.to(xt)
        return out
    b = y.view(-1, st["block"])
    scales = b.abs().amax(1) / 127
    codes = torch.round(b / torch.where(scales > 0, scales, 1.0)[:, None]).clamp_(-127, 127).to(torch.int8)
    out["scales"] = scales
    out["values"] = _values(codes.view(-1), scales, 8, st["block"]).to(torch.bfloat16)
    return out


def _plain_norm_grad(st):
    h, dy, rstd = st["a"].float(), st["dy"].float(), st["rstd"][:, None]
    xhat = h * rstd
    g = dy * st["weight"].float()
    dx = (g - xhat * (g * xhat).mean(1, keepdim=True)) * rstd
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return {"dx": dx.to(st["a"].dtype), "dweight": (dy * xhat).sum(0).to(st["weight"].dtype)}


def _chosen(st):
    """[rows, adapters]: whether the row's adapter is this one."""
    return st["ids"][:, None] == torch.arange(st["adapters"], device="cuda", dtype=torch.int32)


def _own_only(t, chosen):
    """[rows, rank] as [rows, adapters * rank], zeros but at the row's own adapter."""
    return torch.where(chosen[:, :, None], t[:, None, :], 0.0).view(t.shape[0], -1)


def _plain_adapters(st):
    n, rank, inf, outf = st["adapters"], st["rank"], st["in"], st["out"]
    x, chosen = st["a"].float(), _chosen(st)
    every = (x @ st["A"].float().view(n * rank, inf).t()).view(-1, n, rank)
    t = (torch.where(chosen[:, :, None], every, 0.0) * st["scaling"][:, None]).sum(1)
    y = x @ _plain_weight(st).t()
    y = y + _own_only(t, chosen) @ st["B"].float().transpose(1, 2).reshape(n * rank, outf)
    return {"y": y.to(DTYPES[st["y"]]), "reduced": t}


def _plain_adapters_grad(st):
    n, rank, inf, outf = st["adapters"], st["rank"], st["in"], st["out"]
    dy, chosen, wt = st["dy"].float(), _chosen(st), st["A"].dtype
    every = (dy @ st["B"].float().transpose(1, 2).reshape(n * rank, outf).t()).view(-1, n, rank)
    u = (torch.where(chosen[:, :, None], every, 0.0) * st["scaling"][:, None]).sum(1)
    u = _own_only(u, chosen)
    dx = dy @ _plain_weight(st) + u @ st["A"].float().view(n * rank, inf)
    da = (u.t() @ st["a"].float()).view(n, rank, inf)
    db = (_own_only(st["reduced"], chosen).t() @ dy).view(n, rank, outf).transpose(1, 2).contiguous()
    return {"dx": dx.to(DTYPES[st["y"]]), "da": da.to(wt), "db": db.to(wt)}


def _plain_grouped(st):
    """The groups as one batched product, each padded to the largest one's rows."""
    grad = "dy" in st
    a, w = st["dy"] if grad else st["a"], _plain_weight(st)
    row = torch.arange(st["rows"], device="cuda", dtype=torch.int32)
    group = torch.searchsorted(st["offsets"][1:], row, right=True)
    slot = row - st["offsets"][group]
    padded = torch.zeros(st["groups"], st["most"], a.shape[1], device="cuda")
    padded[group, slot] = a.float()
    y = torch.bmm(padded, w if grad else w.transpose(1, 2))
    return y[group, slot].to(DTYPES[st["y"]])


def run(state):
    op = state["op"]
    if not own:
        plain = {"rms_norm": _plain_norm, "rms_norm_grad": _plain_norm_grad, "linear_adapters": _plain_adapters,
                 "linear_adapters_grad": _plain_adapters_grad, "linear_grouped": _plain_grouped,
                 "linear_grouped_grad": _plain_grouped}
        return plain[op](state)
    import block_quantization_codec_amd as z

    st = state
    if op == "rms_norm":
        y, total, rstd, codes, scales = z.rms_norm(st["a"], st["weight"], st["h"], EPS, bits=st["bits"],
                                                   block=st["block"], want_y=not st["bits"])
        out = {"rstd": rstd}
        if st["h"] is not None:
            out["sum"] = total
        if not st["bits"]:
            out["y"] = y
            return out
        out["scales"] = scales
        # the receiver of the codes expands them
        out["values"] = z.dequantize(codes, scales, st["bits"], st["a"].numel(), st["block"])
        return out
    if op == "rms_norm_grad":
        dx, dw = z.rms_norm_grad(st["dy"], st["a"], st["weight"], st["rstd"], dsum=st["dsum"])
        return {"dx": dx, "dweight": dw}
    if op == "linear_adapters":
        y, reduced = z.linear_adapters(st["a"], st["codes"], st["scales"], st["bits"], st["block"], st["out"], st["A"],
                                       st["B"], st["ids"], st["scaling"], dtype=DTYPES[st["y"]])
        return {"y": y, "reduced": reduced}
    if op == "linear_adapters_grad":
        dx, da, db = z.linear_adapters_grad(st["dy"], st["a"], st["reduced"], st["codes"], st["scales"], st["bits"],
                                            st["block"], st["A"], st["B"], st["ids"], st["scaling"],
                                            dtype=DTYPES[st["y"]])
        return {"dx": dx, "da": da, "db": db}
    if op == "linear_grouped":
        return z.linear_grouped(st["a"], st["offsets"], st["codes"], st["scales"], st["bits"], st["block"], st["out"],
                                dtype=DTYPES[st["y"]])
    return z.linear_grouped_grad(st["dy"], st["offsets"], st["codes"], st["scales"], st["bits"], st["block"],
                                 st["in"], dtype=DTYPES[st["y"]])


# ---- what a pass cannot do without ---------------------------------------------

def work(case):
    size = {"bf16": 2, "fp32": 4}
    r, xs, grad = case["rows"], size[case["x"]], case["op"].endswith("_grad")
    if case["op"].startswith("rms_norm"):
        w, ws, more = case["width"], size[case["w"]], 1 if case["residual"] else 0
        if grad:
            return {"bytes": (3 + more) * r * w * xs + 2 * w * ws + 4 * r, "flops": 9 * r * w}
        # the codes and their scales are written, and expanded to bf16 again for the answer
        y = r * w * xs if not case["bits"] else 2 * (r * w + 4 * (r * w // case["block"])) + 2 * r * w
        return {"bytes": (1 + 2 * more) * r * w * xs + y + w * ws + 4 * r, "flops": 5 * r * w}
    n, a, b = case["out"] * case["in"], case["in"], case["out"]
    ys, weight = size[case["y"]], n * case["bits"] // 8 + 4 * (n // case["block"])
    if "groups" in case:
        i, o = (b, a) if grad else (a, b)
        return {"bytes": min(case["groups"], r) * weight + r * (i * xs + o * ys), "flops": 2 * r * n}
    rank, ws, used = case["rank"], size[case["w"]], min(case["adapters"], case["requests"])
    low = used * rank * (a + b) * ws + 4 * r * (rank + 1)
    if not grad:
        return {"bytes": weight + r * (a * xs + b * ys) + low, "flops": 2 * r * n + 2 * r * rank * (a + b)}
    return {"bytes": weight + r * (b * xs + a * xs + a * ys) + low + case["adapters"] * rank * (a + b) * ws,
            "flops": 2 * r * n + 4 * r * rank * (a + b)}


# ---- definitions in binary64 ---------------------------------------------------

def _exact_weight(st, group):
    """Group's [out, in]: element i of its flat buffer is its code's bits, as a signed number, times the scale of
    block i // block."""
    n, bits = st["out"] * st["in"], st["bits"]
    i = torch.arange(n, device="cuda", dtype=torch.int64)
    raw = st["codes"][group * n * bits // 8 + i * bits // 8].to(torch.int16)
    if bits == 4:
        raw = torch.bitwise_right_shift(raw, (i % 2 * 4).to(torch.int16)).bitwise_and_(15)
    half = 1 << (bits - 1)
    raw = (raw + half).remainder_(2 * half) - half
    w = raw.double()
    del raw
    w *= st["scales"].double()[group * (n // st["block"]) + i // st["block"]]
    return w.view(st["out"], st["in"])


def _exact_norm(st):
    xt, out = st["a"].dtype, {}
    h = st["a"].double()
    if st["h"] is not None:
        # the stream is kept in x's type, rounded once; the norm is that of what is kept
        h = (h + st["h"].double()).to(xt)
        out["sum"] = h
        h = h.double()
    n = st["width"]
    rstd = 1.0 / torch.sqrt(torch.einsum("rw,rw->r", h, h) / n + EPS)
    y = h * (rstd.unsqueeze(-1) * st["weight"].double())
    out["rstd"] = rstd
    if not st["bits"]:
        out["y"] = y
        return {k: out[k] for k in ("rstd", "sum", "y") if k in out}
    y = y.view(-1, st["block"])
    scales = y.abs().max(dim=1).values / 127
    safe = scales.masked_fill(scales == 0, 1.0).unsqueeze(-1)
    out["scales"], out["values"] = scales, ((y / safe).round() * safe).view(-1)
    return out


def _exact_norm_grad(st):
    h, dy, rstd, w = st["a"].double(), st["dy"].double(), st["rstd"].double(), st["weight"].double()
    dweight = torch.einsum("rw,rw,r->w", dy, h, rstd)
    # dx_j = rstd (g_j - h_j rstd^2 sum_i g_i h_i / n) + dsum_j,  g = dy * weight
    g = dy * w
    c = rstd * rstd * (g * h).sum(-1) / st["width"]
    dx = rstd.unsqueeze(-1) * (g - h * c.unsqueeze(-1))
    if st["dsum"] is not None:
        dx += st["dsum"].double()
    return {"dx": dx, "dweight": dweight}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rms_norm":
        return _exact_norm(st)
    if op == "rms_norm_grad":
        return _exact_norm_grad(st)
    if "groups" in case:
        grad = op.endswith("_grad")
        a = (st["dy"] if grad else st["a"]).double()
        y = torch.zeros(case["rows"], case["in"] if grad else case["out"], device="cuda", dtype=torch.float64)
        offsets = st["offsets"].tolist()
        for e in range(case["groups"]):
            b, t = offsets[e], offsets[e + 1]
            if t > b:
                w = _exact_weight(st, e)
                y[b:t] = a[b:t] @ (w if grad else w.T)
        return y
    w, A, B, s = _exact_weight(st, 0), st["A"].double(), st["B"].double(), st["scaling"].double()
    a, ids = st["a"].double(), st["ids"].long()
    if op == "linear_adapters":
        y, t = a @ w.T, a.new_zeros(case["rows"], case["rank"])
        for g in range(case["adapters"]):
            m = torch.nonzero(ids == g).flatten()
            t[m] = (a[m] @ A[g].T) * s[g]
            y[m] += t[m] @ B[g].T
        return {"y": y, "reduced": t}
    dy, t = st["dy"].double(), st["reduced"].double()
    dx, da, db = dy @ w, torch.zeros_like(A), torch.zeros_like(B)
    for g in range(case["adapters"]):
        m = torch.nonzero(ids == g).flatten()
        u = (dy[m] @ B[g]) * s[g]
        dx[m] += u @ A[g]
        da[g], db[g] = u.T @ a[m], dy[m].T @ t[m]
    return {"dx": dx, "da": da, "db": db}
