"""The short helpers on a stream that is not torch's current one, and is behind it.

The side stream first waits, so that when a helper returns none of its kernels
has run. Memory that is free for the current stream by then, temporaries and
dropped inputs, is taken and overwritten there; the results must not notice.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def z():
    need_gpu()
    import block_quantization_codec_amd as z

    return z


def cases(z):
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, dtype=BF):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    n, k, block = 4160, 256, 64
    codes, scales = z.quantize(normal(n * k), block, 4)
    x, dy, w = normal(700, 20001), normal(700, 20001), normal(20001, dtype=F32)
    _, mean, rstd = z.layer_norm(x, w, w)
    return {
        "quantize": (z.quantize, (normal(1 << 20), 128, 8)),
        "dequantize": (z.dequantize, (codes, scales, 4, n * k, block)),
        "dequant_reduce_requant": (z.dequant_reduce_requant, (codes, scales, 2, 4, n * k // 2, block, 8)),
        "linear": (z.linear, (normal(300, k, dtype=F32), codes, scales, 4, block, n)),  # packed activations
        "linear_grad": (z.linear_grad, (normal(70, n), codes, scales, 4, block, k)),    # split sums
        "layer_norm": (z.layer_norm, (x, w, w)),
        "layer_norm_grad": (z.layer_norm_grad, (dy, x, w, mean, rstd)),                 # shares and row sums
    }


NAMES = ["quantize", "dequantize", "dequant_reduce_requant", "linear", "linear_grad", "layer_norm", "layer_norm_grad"]


def tensors(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("handle", [False, True], ids=["object", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_a_stream_that_is_behind(z, name, handle):
    helper, args = cases(z)[name]
    want = tensors(helper(*args))
    torch.cuda.synchronize()
    sizes = {t.numel() * t.element_size() for t in (*want, *(a for a in args if isinstance(a, torch.Tensor)))}
    sizes |= {1 << 16, 1 << 20, 1 << 22, 1 << 24}
    side = torch.cuda.Stream()
    mine = [a.clone() if isinstance(a, torch.Tensor) else a for a in args]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # about 20 ms
    got = tensors(helper(*mine, stream=side.cuda_stream if handle else side))
    del mine
    taken = [torch.full((s,), 255, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want, strict=True):
        assert torch.equal(a, b)
    assert len(taken) == 4 * len(sizes)


def test_the_null_stream_by_its_handle(z):
    helper, args = cases(z)["linear_grad"]
    want = helper(*args)
    torch.cuda.synchronize()
    got = helper(*args, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
