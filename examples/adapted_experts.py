"""A layer of frozen codes that is trained through adapters, and its experts:
residual + RMS norm -> projection with low-rank adapters -> experts, forward and
back, then a few requests of one token each.

    python examples/adapted_experts.py [--rows 4096] [--width 4096] [--out 11008] [--experts 8] [--bits 4] [--block 128]

The projection and the experts' weights stay as codes. Rows are sorted by expert, as a
router would leave them, each request's rows name its adapter, and some have none. The
normed rows also go out as 8-bit codes, what a gather over GPUs would send. Each result is
compared with the same formula in binary64 on the dequantized weights, the gradients with
autograd's, and the relative errors are printed.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantization_codec_amd as z  # noqa: E402

EPS = 1e-5


def off(got, want) -> float:
    return ((got.double() - want).norm() / want.norm()).item()


def run(rows=4096, width=4096, out=11008, experts=8, adapters=3, rank=16, bits=4, block=128,
        dtype=torch.bfloat16) -> dict[str, float]:
    """Relative error of each result against binary64."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def codes_of(n, k, count=1):
        w = normal(count * n, k, std=k ** -0.5)
        c, s = z.quantize(w, block, bits)
        return c, s, z.dequantize(c, s, bits, w.numel(), block, dtype=torch.float32).view(count, n, k).double()

    projection, p_scales, p = codes_of(out, width)
    expert, e_scales, e = codes_of(width, out, experts)
    gamma = 1 + normal(width) / 8
    a, b = normal(adapters, rank, width, std=width ** -0.5), normal(adapters, out, rank, std=0.2)
    scaling = torch.full((adapters,), 2.0, device="cuda")
    x, residual, dy, d_stream = normal(rows, width), normal(rows, width), normal(rows, width), normal(rows, width)
    # requests side by side, each with an adapter, the last without; rows already in the experts' order
    request = torch.arange(rows, device="cuda") * (adapters + 1) // rows
    ids = torch.where(request < adapters, request, -1).to(torch.int32)
    ends = torch.sort(torch.randint(0, rows + 1, (experts - 1,), generator=g, device="cuda")).values
    offsets = torch.cat((ends.new_zeros(1), ends, ends.new_full((1,), rows))).to(torch.int32)

    # forward
    h, stream, rstd, sent, sent_scales = z.rms_norm(x, gamma, residual, EPS, bits=8, block=32)
    q, reduced = z.linear_adapters(h, projection, p_scales, bits, block, out, a, b, ids, scaling)
    y = z.linear_grouped(q, offsets, expert, e_scales, bits, block, width)
    # backward: of the experts' input, of the adapters and their input, of the norm
    dq = z.linear_grouped_grad(dy, offsets, expert, e_scales, bits, block, out)
    dh, da, db = z.linear_adapters_grad(dq, h, reduced, projection, p_scales, bits, block, a, b, ids, scaling)
    dx, dgamma = z.rms_norm_grad(dh, stream, gamma, rstd, dsum=d_stream)
    # serving: the last row of each request at once
    last = torch.arange(1, adapters + 2, device="cuda") * rows // (adapters + 1) - 1
    token, _ = z.linear_adapters(h[last], projection, p_scales, bits, block, out, a, b, ids[last], scaling)

    # binary64, step by step as above, each step from what the one before gives in binary64
    leaves = [t.double().requires_grad_() for t in (x, residual, gamma, a, b)]
    x64, r64, g64, a64, b64 = leaves
    s64 = x64 + r64
    h64 = s64 * (s64.square().mean(-1, keepdim=True) + EPS).rsqrt() * g64
    parts = []
    for i in range(adapters + 1):
        here = h64[request == i]
        part = here @ p[0].t()
        parts.append(part + 2.0 * (here @ a64[i].t()) @ b64[i].t() if i < adapters else part)
    q64 = torch.cat(parts)
    bounds = offsets.tolist()
    y64 = torch.cat([q64[s:t] @ e[i].t() for i, (s, t) in enumerate(zip(bounds, bounds[1:]))])
    q64.retain_grad()
    h64.retain_grad()
    ((y64 * dy.double()).sum() + (s64 * d_stream.double()).sum()).backward()
    values = z.dequantize(sent, sent_scales, 8, rows * width, 32, dtype=torch.float32).view(rows, width)
    return {"stream": off(stream, s64.detach()), "h": off(h, h64.detach()), "sent": off(values, h64.detach()),
            "q": off(q, q64.detach()), "y": off(y, y64.detach()), "dq": off(dq, q64.grad), "dh": off(dh, h64.grad),
            "dx": off(dx, x64.grad), "dgamma": off(dgamma, g64.grad), "da": off(da, a64.grad), "db": off(db, b64.grad),
            "token": off(token, q64.detach()[last])}


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--rows", type=int, default=4096)
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--out", type=int, default=11008)
    p.add_argument("--experts", type=int, default=8)
    p.add_argument("--bits", type=int, default=4, choices=(4, 8))
    p.add_argument("--block", type=int, default=128)
    p.add_argument("--dtype", default="bf16", choices=("bf16", "f32"))
    c = p.parse_args()
    dtype = torch.bfloat16 if c.dtype == "bf16" else torch.float32
    for name, e in run(c.rows, c.width, c.out, c.experts, bits=c.bits, block=c.block, dtype=dtype).items():
        print(f"{name:7s} relative error {e:.1e}")


if __name__ == "__main__":
    main()
