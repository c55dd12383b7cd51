"""Rows and weights so far apart that offsets pass 32 bits, on paths that smaller cases do not take."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402
from test_gpu_linear import gen, weights  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def z():
    need_gpu()
    import block_quantization_codec_amd as z

    return z


def apart(t, stride):
    """t's rows, `stride` elements apart in memory of their own."""
    rows, width = t.shape
    far = torch.empty(rows * stride, dtype=t.dtype, device="cuda").view(rows, stride)[:, :width]
    far.copy_(t)
    return far


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
@pytest.mark.parametrize("stride", [(1 << 22), (1 << 22) + 8, (1 << 23) + 64])
def test_activations_in_far_rows(z, grad, stride):
    """Strides up to 2^22 elements are read in place by the tiled products, longer ones packed first."""
    g = gen(1)
    rows, n, k = 300, 1000, 1024
    codes, scales, w = weights(g, n, k, 4, 128, lambda m: torch.ones(m, device="cuda"))
    a = torch.randint(-4, 5, (rows, n if grad else k), generator=g, device="cuda").to(BF)
    f, m = (z.linear_grad, w) if grad else (z.linear, w.t())
    want = (a.double() @ m).to(BF)
    for r in (1, 4, 40, rows):  # every kernel
        assert torch.equal(f(apart(a[:r], stride), codes, scales, 4, 128, m.shape[1]), want[:r])
    out = torch.full((rows, stride), 77.0, dtype=BF, device="cuda")[:, :m.shape[1]]
    assert torch.equal(f(a, codes, scales, 4, 128, m.shape[1], out=out), want)


def test_8_bit_codes_past_32_bits(z):
    n, k, block = (1 << 21) + 3, 2048, 2048
    codes = torch.zeros(n * k, dtype=torch.uint8, device="cuda")
    scales = torch.ones(n * k // block, device="cuda")
    codes.view(n, k)[n - 1, ::2] = 255  # the last feature: -1, 2, -1, 2, ...
    codes.view(n, k)[n - 1, 1::2] = 2
    for rows in (3, 20, 300):
        y = z.linear(torch.ones(rows, k, dtype=BF, device="cuda"), codes, scales, 8, block, n)
        assert bool((y[:, n - 1] == k // 2).all()) and int(torch.count_nonzero(y)) == rows
        del y
    for rows in (5, 70):
        dy = torch.zeros(rows, n, dtype=BF, device="cuda")
        dy[:, n - 1] = 3
        dx = z.linear_grad(dy, codes, scales, 8, block, k)
        assert torch.equal(dx, torch.tensor([-3.0, 6.0], device="cuda").to(BF).repeat(rows, k // 2))


@pytest.mark.parametrize("width", [512, 4099, 8192, 20001, 32768, 40000])
@pytest.mark.parametrize("types", [(BF, F32), (F32, F32)], ids=["bf", "ff"])
def test_norm_rows_past_32_bits(z, types, width):
    """The same bits as from rows side by side in strides that keep the same alignment."""
    xt, wt = types
    g = gen(width)
    rows, stride, near = 4200, 1 << 20, -(-width // 8) * 8
    x, dy = (torch.randn(rows, near, generator=g, device="cuda").to(xt)[:, :width] for _ in range(2))
    w, b = (torch.randn(width, generator=g, device="cuda").to(wt) for _ in range(2))
    def like(t, fill):
        return torch.full((rows, t), fill, dtype=xt, device="cuda")[:, :width]

    y, mean, rstd = z.layer_norm(x, w, b, out=like(near, 5.0))
    dx, dw, db = z.layer_norm_grad(dy, x, w, mean, rstd, out=like(near, 5.0))
    fx, fdy = apart(x, stride), apart(dy, stride)
    out = like(stride, 7.0)
    y2, mean2, rstd2 = z.layer_norm(fx, w, b, out=out)
    assert torch.equal(y2, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    out.fill_(7.0)
    dx2, dw2, db2 = z.layer_norm_grad(fdy, fx, w, mean, rstd, out=out)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
