"""A layer whose weight stays as codes and scales: norm -> linear, forward and
back, then one token at a time.

    python examples/quantized_layer.py [--rows 4096] [--width 4096] [--out 11008] [--bits 4] [--block 128]

The weight is quantized once, as a shard would be before the all-gather, and
is never expanded: the product, its input gradient and the single-token product
read the codes. Each result is compared with the same formula in binary64 on
the dequantized weight, and the relative errors are printed.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantization_codec_amd as z  # noqa: E402


def off(got, want) -> float:
    return ((got.double() - want).norm() / want.norm()).item()


def run(rows=4096, width=4096, out=11008, bits=4, block=128, dtype=torch.bfloat16) -> dict[str, float]:
    """Relative error of each result against binary64."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    weight = normal(out, width) * width ** -0.5
    codes, scales = z.quantize(weight, block, bits)
    gamma, beta = 1 + normal(width) / 8, normal(width) / 8
    x, dy = normal(rows, width), normal(rows, out)

    # training: forward and the gradients of x, gamma and beta
    h, mean, rstd = z.layer_norm(x, gamma, beta)
    y = z.linear(h, codes, scales, bits, block, out)
    dh = z.linear_grad(dy, codes, scales, bits, block, width)
    dx, dgamma, dbeta = z.layer_norm_grad(dh, x, gamma, mean, rstd)

    # serving: the last row by itself, on a workspace kept from token to token
    code = z.ZPP_BF16 if dtype == torch.bfloat16 else z.ZPP_FP32
    workspace = torch.empty(max(z.zpp_linear_blocks_workspace(0, code, width, code, 1, out, width), 16),
                            dtype=torch.uint8, device="cuda")
    one, _, _ = z.layer_norm(x[-1:], gamma, beta)
    token = z.linear(one, codes, scales, bits, block, out, workspace=workspace)

    w = z.dequantize(codes, scales, bits, out * width, block, dtype=torch.float32).view(out, width).double()
    hat = (x.double() - x.double().mean(-1, keepdim=True)) / (x.double().var(-1, unbiased=False, keepdim=True)
                                                               + 1e-5).sqrt()
    h64 = hat * gamma.double() + beta.double()
    dh64 = dy.double() @ w
    t = dh64 * gamma.double()
    dx64 = (t - t.mean(-1, keepdim=True) - hat * (t * hat).mean(-1, keepdim=True)) / (
        x.double().var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    return {"h": off(h, h64), "y": off(y, h64 @ w.t()), "dh": off(dh, dh64), "dx": off(dx, dx64),
            "dgamma": off(dgamma, (dh64 * hat).sum(0)), "dbeta": off(dbeta, dh64.sum(0)),
            "token": off(token, h64[-1:] @ w.t())}


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--rows", type=int, default=4096)
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--out", type=int, default=11008)
    p.add_argument("--bits", type=int, default=4, choices=(4, 8))
    p.add_argument("--block", type=int, default=128)
    p.add_argument("--dtype", default="bf16", choices=("bf16", "f32"))
    a = p.parse_args()
    dtype = torch.bfloat16 if a.dtype == "bf16" else torch.float32
    for name, e in run(a.rows, a.width, a.out, a.bits, a.block, dtype).items():
        print(f"{name:7s} relative error {e:.1e}")


if __name__ == "__main__":
    main()
