"""Linear products on block codes, and their input gradient, on the GPU.

Most cases use small whole numbers and power-of-two scales, for which every
product and every partial sum is exact in binary32 (and every weight exact in
bf16): whatever the order of the sum, the result must equal the 64-bit one,
rounded once. A mistake in any index, scale or mask changes it. Random
real-valued cases bound the roundings that such numbers do not show.
"""
from __future__ import annotations

import itertools

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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def pack(codes, bits):
    """Signed codes (int, any shape) as the codec's bytes."""
    c = codes.reshape(-1).to(torch.int64)
    if bits == 8:
        return (c & 255).to(torch.uint8)
    n = (c & 15).view(-1, 2)
    return (n[:, 0] | (n[:, 1] << 4)).to(torch.uint8)


def weights(g, n, k, bits, block, scale_of):
    """(codes, scales, W in 64 bits): every code value occurs, -8 and -128 too."""
    half = 1 << (bits - 1)
    c = torch.randint(-half, half, (n * k,), generator=g, device="cuda")
    s = scale_of(n * k // block)
    w = (c.double().view(-1, block) * s.double()[:, None]).view(n, k)
    return pack(c, bits), s, w


def whole_case(z, seed, grad, rows, n, k, bits, block, it, ot, pad_in=0, pad_out=0):
    """A case of whole numbers: the call's result, the exact one, and the guard around the result."""
    g = gen(seed)
    codes, scales, w = weights(g, n, k, bits, block, lambda m: torch.pow(
        2.0, torch.randint(-1, 2, (m,), generator=g, device="cuda").float()))
    al, ol = (n, k) if grad else (k, n)
    # binary32 inputs take more than 8 bits; sums stay below 2^23 halves by 5 standard deviations or more
    top = 300 if it == F32 else 4
    a = torch.randint(-top, top + 1, (rows, al + pad_in), generator=g, device="cuda").to(it)
    out = torch.full((rows, ol + pad_out), 77.0, dtype=ot, device="cuda")
    f = z.linear_grad if grad else z.linear
    f(a[:, :al], codes, scales, bits, block, ol, out=out[:, :ol])
    want = a[:, :al].double() @ (w if grad else w.t())
    return out[:, :ol], want.to(ot), out[:, ol:]


# the rows of each kernel's tiles and one more or less; widths that are no multiple of any tile
ROWS = [1, 2, 15, 16, 17, 31, 33, 64, 65, 129, 257, 300]
SHAPES = [(1, 32, 32), (3, 64, 32), (16, 96, 64), (31, 128, 128), (64, 160, 32), (100, 256, 256), (257, 224, 32),
          (300, 1056, 32), (129, 384, 128), (8, 1024, 1024), (259, 128, 64)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=["bb", "bf", "ff", "fb"])
@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_whole_numbers(z, grad, types, bits):
    for i, (rows, (n, k, block)) in enumerate(itertools.product(ROWS, SHAPES)):
        got, want, _ = whole_case(z, i, grad, rows, n, k, bits, block, *types)
        assert torch.equal(got, want), (rows, n, k, block, (got != want).sum().item())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
@pytest.mark.parametrize("rows,n,k,block", [
    (1, 4096, 1056, 2048),    # blocks straddle rows: in_features = 33 * 32
    (5, 33, 4096 - 32, 32),
    (40, 64, 2080, 1024),
    (200, 96, 160, 512),
    (333, 2048, 352, 2048),
])
def test_blocks_that_straddle_rows(z, grad, bits, rows, n, k, block):
    assert n * k % block == 0
    got, want, _ = whole_case(z, 5, grad, rows, n, k, bits, block, BF, F32)
    assert torch.equal(got, want)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32)], ids=["bb", "bf", "ff"])
def test_many_tiles_and_split_sums(z, grad, types, bits):
    """Enough tiles for the largest ones, and long contractions with few tiles, which are split."""
    for rows, n, k, block in [(2100, 5120, 320, 64), (2100, 320, 5120, 256), (70, 4160, 192, 64), (70, 192, 4160, 64),
                              (13, 8200, 96, 32), (600, 1001, 1024, 128)]:
        got, want, _ = whole_case(z, 9, grad, rows, n, k, bits, block, *types)
        assert torch.equal(got, want), (rows, n, k, block)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("ot", [BF, F32], ids=["fb", "ff"])
@pytest.mark.parametrize("rows,n,k,block", [
    # on either side of the choice between exact codes and tiles of 16, 64 and 128 rows, split and not
    (129, 1056, 96, 32), (260, 8200, 352, 32), (200, 4100, 1056, 32), (333, 1001, 2080, 32), (520, 4100, 1056, 32),
    (700, 1000, 4128, 32), (300, 4096, 992, 64), (600, 1001, 1024, 128), (300, 96, 160, 64), (129, 8192, 1184, 512),
])
def test_many_rows_of_binary32(z, rows, n, k, block, ot, bits):
    got, want, _ = whole_case(z, 11, False, rows, n, k, bits, block, F32, ot)
    assert torch.equal(got, want)


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
@pytest.mark.parametrize("rows", [1, 3, 20, 70, 300])
def test_row_strides_leave_gaps_alone(z, grad, rows):
    for it, ot in [(BF, BF), (F32, F32)]:
        # the side of in_features in whole 16-byte pieces, the other with any stride
        for pad_in, pad_out in ([(1, 8), (5, 16), (8, 8)] if grad else [(8, 1), (16, 3), (8, 8)]):
            for n in (72, 75):
                got, want, gap = whole_case(z, 3, grad, rows, n, 128, 4, 32, it, ot, pad_in, pad_out)
                assert torch.equal(got, want) and bool((gap == 77).all()), (it, pad_in, pad_out, n)


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
@pytest.mark.parametrize("rows", [4, 40, 100, 300])
def test_non_finite_rows_stay_their_own(z, grad, rows):
    g = gen(1)
    codes, scales, w = weights(g, 96, 160, 4, 32, lambda m: torch.ones(m, device="cuda"))
    for it in (BF, F32):
        a = torch.randint(-4, 5, (rows, 96 if grad else 160), generator=g, device="cuda").to(it)
        want = (a.double() @ (w if grad else w.t())).to(it)
        bad = a.clone()
        bad[1, 7], bad[2, 0], bad[rows - 1, -1] = float("inf"), float("nan"), float("-inf")
        got = (z.linear_grad if grad else z.linear)(bad, codes, scales, 4, 32, 160 if grad else 96)
        keep = torch.ones(rows, dtype=torch.bool, device="cuda")
        keep[[1, 2, rows - 1]] = False
        assert torch.equal(got[keep], want[keep])
        assert not bool(torch.isfinite(got[~keep]).any())


def rounding_bound(a, w, want, it, ot, weights_rounded):
    """How far a result may be from the exact one. With v the products of one
    sum and c their number: the result's own rounding; where weights enter as
    bf16, c independent errors of at most 2^-8 |v| (their sum is within 6 times
    2^-8 |v|_2 by far more than the number of results); and the binary32 sum: c
    roundings of partial sums that stay below 4 |v|_2, of 2^-24 each, as a
    random walk (20 sqrt(c) covers 8 standard deviations), plus, in case the
    matrix instruction's own sums round one way, c / 8."""
    v2 = ((a.double() ** 2) @ (w ** 2)).sqrt()
    c = w.shape[0]
    tol = want.abs() * torch.finfo(ot).eps / 2 + 2.0 ** -24 * (20 * c ** 0.5 + c / 8) * v2
    if weights_rounded:
        tol = tol + 6 * 2.0 ** -8 * v2
    return tol * (1 + 2.0 ** -7) + 2.0 ** -130  # the last rounding is of the value with the other errors in it


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=["bb", "bf", "ff", "fb"])
@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_real_numbers(z, grad, types, bits):
    it, ot = types
    for i, (rows, n, k, block) in enumerate([(1, 1024, 2048, 128), (9, 555, 512, 64), (50, 640, 1024, 32),
                                             (150, 1027, 768, 256), (1030, 1024, 4096, 128)]):
        g = gen(100 + i)
        codes, scales, w = weights(g, n, k, bits, block, lambda m: torch.rand(m, generator=g, device="cuda") * 0.01)
        a = (torch.randn(rows, n if grad else k, generator=g, device="cuda") * 3).to(it)
        m = w if grad else w.t()
        got = (z.linear_grad if grad else z.linear)(a, codes, scales, bits, block, m.shape[1], dtype=ot)
        want = a.double() @ m
        off = (got.double() - want).abs()
        tol = rounding_bound(a, m, want, it, ot, types == (BF, BF))
        assert bool((off <= tol).all()), ((rows, n, k), (off / tol).max().item())


def test_gradient_is_the_slope_of_the_product(z):
    """dx . d against the difference of y along d, both from the library. Whole numbers: both exact."""
    g = gen(4)
    for bits, rows, n, k, block in [(4, 3, 70, 128, 32), (8, 90, 200, 320, 64)]:
        codes, scales, _ = weights(g, n, k, bits, block, lambda m: torch.ones(m, device="cuda"))
        x, d = (torch.randint(-3, 4, (rows, k), generator=g, device="cuda").float() for _ in range(2))
        dy = torch.randint(-3, 4, (rows, n), generator=g, device="cuda").float()
        up, down = (z.linear(x + s * d, codes, scales, bits, block, n) for s in (1, -1))
        slope = ((up - down).double() * dy.double()).sum(1) / 2
        dx = z.linear_grad(dy, codes, scales, bits, block, k)
        assert torch.equal((dx.double() * d.double()).sum(1), slope)


def test_codes_from_the_codec_multiply_as_they_dequantize(z):
    g = gen(8)
    for bits, n, k, block in [(4, 512, 1024, 128), (8, 320, 11008, 2048)]:
        w = (torch.randn(n, k, generator=g, device="cuda") * 0.02).to(BF)
        codes, scales = z.quantize(w.view(-1), block, bits)
        eye = torch.eye(k, dtype=BF, device="cuda")
        back = z.dequantize(codes, scales, bits, n * k, block).view(n, k)
        assert torch.equal(z.linear(eye, codes, scales, bits, block, n).t(), back)
        assert torch.equal(z.linear_grad(torch.eye(n, dtype=BF, device="cuda"), codes, scales, bits, block, k), back)
        full = z.dequantize(codes, scales, bits, n * k, block, dtype=F32).view(n, k)
        assert torch.equal(z.linear(eye[:48], codes, scales, bits, block, n, dtype=F32).t(), full[:, :48])


def test_leading_dimensions_and_no_rows(z):
    g = gen(2)
    codes, scales, w = weights(g, 48, 64, 8, 32, lambda m: torch.ones(m, device="cuda"))
    x = torch.randint(-4, 5, (2, 3, 64), generator=g, device="cuda").to(BF)
    y = z.linear(x, codes, scales, 8, 32, 48)
    assert y.shape == (2, 3, 48) and torch.equal(y, (x.double() @ w.t()).to(BF))
    assert z.linear(x[:0], codes, scales, 8, 32, 48).shape == (0, 3, 48)
    assert z.linear_grad(y[0, :0], codes, scales, 8, 32, 64).shape == (0, 64)


def test_same_bits_every_time_and_on_another_stream(z):
    g = gen(6)
    codes, scales, _ = weights(g, 4160, 256, 4, 64, lambda m: torch.rand(m, generator=g, device="cuda"))
    dy = torch.randn(70, 4160, generator=g, device="cuda").to(BF)  # split sums, joined in order
    first = z.linear_grad(dy, codes, scales, 4, 64, 256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = z.linear_grad(dy, codes, scales, 4, 64, 256)
    torch.cuda.current_stream().wait_stream(side)
    for got in (second, z.linear_grad(dy, codes, scales, 4, 64, 256)):
        assert torch.equal(got, first)


def test_offsets_past_32_bits(z):
    """More than 2^32 weights and results whose byte offsets pass 2^32."""
    n, k, block = (1 << 21) + 3, 2048, 2048
    codes = torch.zeros(n * k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.ones(n * k // block, device="cuda")
    codes.view(n, k // 2)[n - 1] = 0x21         # the last feature: 1, 2, 1, 2, ...
    x = torch.ones(3, k, dtype=BF, device="cuda")
    y = z.linear(x, codes, scales, 4, block, n, dtype=F32)
    assert bool((y[:, n - 1] == 1.5 * k).all()) and bool((y[:, : n - 1] == 0).all())
    dy = torch.zeros(70, n, dtype=BF, device="cuda")
    dy[:, n - 1] = 2
    dx = z.linear_grad(dy, codes, scales, 4, block, k)
    assert torch.equal(dx, torch.tensor([2.0, 4.0], device="cuda").to(BF).repeat(70, k // 2))
    many = z.linear(torch.ones(600, k, dtype=BF, device="cuda"), codes, scales, 4, block, n)  # 2.5 GB of results
    assert bool((many[:, n - 1] == 1.5 * k).all()) and int(torch.count_nonzero(many[:, : n - 1])) == 0
