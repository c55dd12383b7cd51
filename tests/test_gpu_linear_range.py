"""Linear products on block codes where activations are far apart, or far out, in size.

Calls of up to 64 rows multiply by the codes themselves, so nothing but the
binary32 sums and the result is rounded, and an activation that meets a code of
zero has no part in a result, however large it is.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402
from test_gpu_linear import gen, pack, rounding_bound, weights  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EXACT = [1, 2, 3, 4, 5, 16, 17, 33, 64]  # rows of each kernel that multiplies by the codes


@pytest.fixture(scope="module")
def z():
    need_gpu()
    import block_quantization_codec_amd as z

    return z


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("ot", [BF, F32], ids=["b", "f"])
def test_weights_of_few_rows_are_not_rounded(z, bits, block, ot):
    n, k = 320, 1024
    for rows in EXACT:
        g = gen(rows)
        codes, scales, w = weights(g, n, k, bits, block, lambda m: torch.rand(m, generator=g, device="cuda") * 0.01)
        x = (torch.randn(rows, k, generator=g, device="cuda") * 3).to(BF)
        got = z.linear(x, codes, scales, bits, block, n, dtype=ot)
        want = x.double() @ w.t()
        off = (got.double() - want).abs()
        tol = rounding_bound(x, w.t(), want, BF, ot, False)
        assert bool((off <= tol).all()), (rows, (off / tol).max().item())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32)], ids=["bb", "bf", "ff"])
def test_a_large_activation_that_meets_zero_codes(z, types, block, bits):
    n, k = 320, 1024
    for rows in EXACT:
        g = gen(rows)
        half = 1 << (bits - 1)
        c = torch.randint(-half, half, (n, k), generator=g, device="cuda")
        far = torch.randperm(k, generator=g, device="cuda")[:8]
        c[:, far] = 0
        s = torch.rand(n * k // block, generator=g, device="cuda") * 0.01
        w = (c.double().view(-1, block) * s.double()[:, None]).view(n, k)
        x = torch.randn(rows, k, generator=g, device="cuda")
        x[:, far] *= 2.0 ** 18
        x = x.to(types[0])
        got = z.linear(x, pack(c, bits), s, bits, block, n, dtype=types[1])
        want = x.double() @ w.t()
        off = (got.double() - want).abs()
        tol = rounding_bound(x, w.t(), want, *types, False)
        assert bool((off <= tol).all()), (rows, (off / tol).max().item())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=["bb", "bf", "ff", "fb"])
def test_activations_far_out(z, types, bits):
    """Whole numbers times powers of two, exact in every order, whose sums without the scales
    would pass the largest binary32 value; other rows are of the usual size."""
    it, ot = types
    for rows, n, k, block in [(1, 96, 1024, 128), (2, 40, 96, 32), (4, 33, 2048, 2048), (5, 75, 1024, 128),
                              (17, 300, 160, 32), (33, 96, 4096, 64), (64, 130, 2176, 128), (70, 96, 512, 128),
                              (300, 140, 1024, 32), (333, 300, 2048, 256)]:
        g = gen(rows)
        codes, scales, w = weights(g, n, k, bits, block, lambda m: torch.pow(
            2.0, torch.randint(-31, -29, (m,), generator=g, device="cuda").float()))
        x = torch.randint(-3, 4, (rows, k), generator=g, device="cuda").to(it)
        x[:, : k // 2] = x[:, : k // 2].abs() + 1  # sums of one sign, so that they grow
        x[::3] *= 2.0 ** 125
        got = z.linear(x, codes, scales, bits, block, n, dtype=ot)
        want = x.double() @ w.t()
        assert bool((want.abs() < 2.0 ** 120).all())
        assert torch.equal(got, want.to(ot)), (rows, n, k, block, (got != want.to(ot)).sum().item())
        dy = torch.randint(-3, 4, (rows, n), generator=g, device="cuda").to(it)
        dy[::3] *= 2.0 ** 125
        got, want = z.linear_grad(dy, codes, scales, bits, block, k, dtype=ot), dy.double() @ w
        assert torch.equal(got, want.to(ot)), ("grad", rows, n, k, block)


@pytest.mark.parametrize("rows", [1, 4, 30, 64, 100])
def test_non_finite_activations_still_show(z, rows):
    g = gen(rows)
    codes, scales, _ = weights(g, 96, 1024, 8, 128, lambda m: torch.rand(m, generator=g, device="cuda"))
    x = torch.randn(rows, 1024, generator=g, device="cuda").to(BF)
    x[0, 1023] = float("inf")
    if rows > 1:
        x[rows - 1, 0] = float("nan")
    y = z.linear(x, codes, scales, 8, 128, 96, dtype=F32)
    bad = [0, rows - 1]
    assert not bool(torch.isfinite(y[bad]).any())
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert bool(torch.isfinite(y[keep]).all())
