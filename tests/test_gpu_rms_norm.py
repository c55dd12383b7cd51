"""RMS norm with residual and codes, forward and backward, on the GPU against its definition in 64 bits."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
U = 2.0 ** -24

# each kernel's widths and one more or less, odd ones, and rows beyond the registers
WIDTHS = [1, 2, 7, 64, 255, 512, 513, 1000, 2048, 2049, 2056, 4099, 8192, 8200, 8193, 16384, 16385, 20000, 40004]


@pytest.fixture(scope="module")
def z():
    need_gpu()
    import block_quantization_codec_amd as z

    return z


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def inputs(seed, rows, width, xt, wt, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, res, dy, ds = ((normal(g, rows, width + pad) * s).to(xt)[:, :width] for s in (2, 3, 1, 1))
    return x, res, dy, ds, (1 + 0.2 * normal(g, width)).to(wt)


def adds(width):
    """Most binary32 additions one value goes through in a row's sum: a thread's own, then the tree."""
    return (32 if width <= 16384 else -(-width // 1024)) + 6 + 16


def values(codes, scales, bits, block):
    c = codes.view(-1)
    if bits == 8:
        q = c.view(torch.int8).double()
    else:
        n = torch.stack((c & 15, c >> 4), 1).view(-1).to(torch.int64)
        q = torch.where(n > 7, n - 16, n).double()
    return q, (q.view(-1, block) * scales.double()[:, None]).view(-1)


def check_forward(z, x, res, w, bits=0, block=0, **kw):
    y, total, rstd, codes, scales = z.rms_norm(x, w, res, EPS, bits, block, **kw)
    if res is not None:
        # one binary32 addition, which is exact or rounded as torch's, then the rounding to x's type
        assert torch.equal(total, (x.float() + res.float()).to(x.dtype))
    else:
        assert total is None
    h = (x if res is None else total).double()
    width = h.shape[-1]
    ms = (h * h).mean(-1, keepdim=True)
    r = 1 / (ms + EPS).sqrt()
    # the sum of squares: a rounding each addition, relative to a sum of positive terms; the product with
    # 1 / width (2 roundings), the addition of eps; half of that through the root, whose own rounding and the
    # division's come on top
    er = ((adds(width) + 3) / 2 + 2) * U
    assert bool(((rstd.double() - r[..., 0]).abs() <= er * r[..., 0]).all())
    want = h * r * (1.0 if w is None else w.double())
    ey = er + 2 * U  # and two products
    if y is not None:
        tol = want.abs() * (ey + torch.finfo(x.dtype).eps / 2) * (1 + 2.0 ** -7) + 1e-37
        assert bool(((y.double() - want).abs() <= tol).all()), (tuple(x.shape), x.dtype)
    if bits:
        top = 127 if bits == 8 else 7
        q, v = values(codes, scales, bits, block)
        peak = want.reshape(-1, block).abs().amax(1) / top
        assert bool(((scales.double() - peak).abs() <= peak * (ey + U) * (1 + 2.0 ** -7)).all())
        assert bool((q.abs() <= top).all())
        # a code is the nearest to its value (off by ey) over the scale; the quotient is rounded, by at most
        # top * U of a step
        off = (v - want.reshape(-1)).abs()
        step = scales.double()[:, None].expand(-1, block).reshape(-1)
        assert bool((off <= step * (0.5 + top * U) + want.reshape(-1).abs() * ey + 1e-37).all())
        # and the largest of a block is coded by the largest code
        assert bool((q.view(-1, block).abs().amax(1)[scales > 0] == top).all())
    return y, total, rstd, codes, scales


def check_backward(z, dy, h, w, rstd, ds, out=None):
    rows, width = h.shape
    dx, dw = z.rms_norm_grad(dy, h, w, rstd, ds, out=out)
    r, g0 = rstd.double()[:, None], dy.double()
    xh = h.double() * r
    g = g0 * (1.0 if w is None else w.double())
    c = (g * xh).mean(1, keepdim=True)
    d = 0.0 if ds is None else ds.double()
    want = (g - xh * c) * r + d
    n = adds(width)
    # xh and g round once each, their products' sum n times, the mean's product with 1 / width 2
    ec = (n + 5) * U * (g * xh).abs().mean(1, keepdim=True)
    # g (1 rounding), xh c (xh's, the product's), the difference's own
    tol = (2 * U * g.abs() + 3 * U * (xh * c).abs() + ec * xh.abs()) * r
    tol = tol + ((g - xh * c) * r).abs() * U + want.abs() * (U + torch.finfo(h.dtype).eps / 2) + 1e-37
    off = (dx.double() - want).abs()
    assert bool((off <= tol * (1 + 2.0 ** -7)).all()), ((rows, width), (off / tol).max().item())
    # over rows: at most all of them in one thread's sum, plus the units' join
    k = min(rows, 4096) + 72 + 3
    v = g0 * xh
    tol = k * U * v.abs().sum(0) + v.sum(0).abs() * torch.finfo(dw.dtype).eps / 2 + 1e-37
    off = (dw.double() - v.sum(0)).abs()
    assert bool((off <= tol * (1 + 2.0 ** -7)).all()), ((rows, width), (off / tol).max().item())
    return dx, dw


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=["bb", "bf", "ff", "fb"])
@pytest.mark.parametrize("width", WIDTHS)
def test_against_64_bits(z, width, types):
    for rows in (1, 3, 67):
        x, res, dy, ds, w = inputs(rows, rows, width, *types)
        for residual, arriving in ((res, ds), (None, None)):
            _, total, rstd, _, _ = check_forward(z, x, residual, w)
            check_backward(z, dy, x if residual is None else total, w, rstd, arriving)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("xt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("width,block", [
    (32, 32), (96, 32), (256, 256), (512, 512), (512, 128), (1024, 1024), (1536, 512), (2048, 2048), (4096, 4096),
    (4160, 64), (4096, 1024), (8192, 4096), (8192, 32), (6144, 2048), (16384, 4096), (10240, 512), (20480, 4096),
    (32768, 64), (17408, 1024)])
def test_codes(z, width, block, xt, bits):
    for rows in (1, 5, 33):
        x, res, _, _, w = inputs(rows, rows, width, xt, F32)
        for residual in (None, res):
            got = check_forward(z, x, residual, w, bits, block)
            # the same codes whether y is asked for or not, and in binary32 those of y itself
            _, _, rstd, codes, scales = z.rms_norm(x, w, residual, EPS, bits, block, want_y=False)
            assert torch.equal(codes, got[3]) and torch.equal(scales, got[4]) and torch.equal(rstd, got[2])
            if xt == F32:
                c, s = z.quantize(got[0], block, bits)
                assert torch.equal(codes, c) and torch.equal(scales, s)


@pytest.mark.parametrize("rows,width", [(5000, 64), (9001, 100), (2500, 4096), (2500, 4097), (700, 16384), (600, 17000)])
def test_more_rows_than_units(z, rows, width):
    x, res, dy, ds, w = inputs(1, rows, width, BF, F32)
    block = width & -width
    bits, block = (8, min(block, 4096)) if block >= 32 else (0, 0)
    _, total, rstd, _, _ = check_forward(z, x, res, w, bits, block)
    check_backward(z, dy, total, w, rstd, ds)


@pytest.mark.parametrize("width", [96, 2052, 9024, 33000])
def test_row_strides_and_no_weights(z, width):
    for xt in (BF, F32):
        for pad in (0, 3, 8):
            x, res, dy, ds, _ = inputs(2, 9, width, xt, xt, pad)
            y, total, dx = (torch.full((9, width + 5), 77.0, dtype=xt, device="cuda") for _ in range(3))
            bits, block = (8, 32) if width % 32 == 0 else (0, 0)
            _, _, rstd, _, _ = check_forward(z, x, res, None, bits, block, out=y[:, :width], total=total[:, :width])
            check_backward(z, dy, total[:, :width], None, rstd, ds, out=dx[:, :width])
            for t in (y, total, dx):
                assert bool((t[:, width:] == 77).all())


def test_results_passed_in_are_used(z):
    x, res, _, _, w = inputs(3, 6, 256, BF, BF)
    want = z.rms_norm(x, w, res, EPS, 8, 64)
    mine = [torch.empty_like(t) for t in want]
    got = z.rms_norm(x, w, res, EPS, 8, 64, out=mine[0], total=mine[1], rstd=mine[2], codes=mine[3], scales=mine[4])
    for a, b, c in zip(want, mine, got):
        assert torch.equal(a, b) and c.data_ptr() == b.data_ptr()
    x3 = x.view(2, 3, 256)
    y, total, rstd, _, _ = z.rms_norm(x3, w, res.view(2, 3, 256), EPS)
    assert y.shape == total.shape == x3.shape and rstd.shape == (2, 3)
    assert torch.equal(y.view(6, 256), want[0]) and torch.equal(total.view(6, 256), want[1])


@pytest.mark.parametrize("width", [64, 1024, 8192, 20480])
def test_non_finite_rows_stay_their_own_and_zero_rows_are_zero(z, width):
    for xt in (BF, F32):
        x, res, dy, ds, w = inputs(4, 9, width, xt, F32)
        want = z.rms_norm(x, w, res, EPS, 8, 64)
        dwant, _ = z.rms_norm_grad(dy, want[1], w, want[2], ds)
        bad, rbad = x.clone(), res.clone()
        bad[2, 5], bad[4, width - 1], bad[6] = float("inf"), float("nan"), 0
        rbad[6] = 0
        y, total, rstd, codes, scales = z.rms_norm(bad, w, rbad, EPS, 8, 64)
        dx, _ = z.rms_norm_grad(dy, total, w, rstd, ds)
        ok = [0, 1, 3, 5, 7, 8]
        for a, b in ((y, want[0]), (total, want[1]), (rstd, want[2]), (codes.view(9, -1), want[3].view(9, -1)),
                     (scales.view(9, -1), want[4].view(9, -1)), (dx, dwant)):
            assert torch.equal(a[ok], b[ok])
        assert bool(torch.isnan(y[4].float()).all()) and bool((y[6] == 0).all())
        assert bool((codes.view(9, -1)[6] == 0).all()) and bool((scales.view(9, -1)[6] == 0).all())


def test_no_rows(z):
    x = torch.empty(0, 128, dtype=BF, device="cuda")
    y, total, rstd, codes, scales = z.rms_norm(x, None, x.clone(), EPS, 8, 32)
    assert y.shape == total.shape == (0, 128) and rstd.numel() == codes.numel() == scales.numel() == 0
    dx, dw = z.rms_norm_grad(x, x, None, rstd)
    assert dx.shape == (0, 128) and bool((dw == 0).all())


def test_gradient_against_differences(z):
    """dx . d and dweight . e against central differences of the definition in 64 bits."""
    x, res, dy, ds, w = inputs(5, 7, 300, F32, F32)
    _, total, rstd, _, _ = z.rms_norm(x, w, res, EPS)
    dx, dw = z.rms_norm_grad(dy, total, w, rstd, ds)
    g = torch.Generator(device="cuda").manual_seed(6)
    d, e = normal(g, 7, 300).double(), normal(g, 300).double()

    def loss(h, weight):
        y = h / ((h * h).mean(1, keepdim=True) + EPS).sqrt() * weight
        return ((y * dy.double()).sum() + (h * ds.double()).sum()).item()

    # the norm of the rounded sum: differentiate at what was kept
    h64, w64 = total.double(), w.double()

    def slope(s):
        return (loss(h64 + s * d, w64 + s * e) - loss(h64 - s * d, w64 - s * e)) / (2 * s)

    first, second = slope(2.0 ** -8), slope(2.0 ** -9)
    got = (dx.double() * d).sum().item() + (dw.double() * e).sum().item()
    # the differences' own error falls fourfold from step to step, so the second's is about a third of their
    # difference; the kernels' is at most 64 roundings of each term (see check_backward), rstd's of 27 among them
    terms = (dx.double() * d).abs().sum().item() + (dw.double() * e).abs().sum().item()
    mags = (dy.double() * w64 * rstd.double()[:, None]).abs() + ds.double().abs()
    terms += 2 * (mags * d.abs()).sum().item()
    assert abs(got - second) <= abs(first - second) + 64 * U * terms


def test_far_rows(z):
    rows, width, stride = 5, 512, (1 << 30) + 8  # the last row's offset passes 32 bits in bytes and in elements
    x, res, dy, ds, w = inputs(7, rows, width, BF, F32)

    def apart(t):
        far = torch.empty(rows * stride, dtype=BF, device="cuda").view(rows, stride)[:, :width]
        return far.copy_(t)

    y, total, rstd, codes, _ = z.rms_norm(apart(x), w, apart(res), EPS, 4, 64, out=apart(x), total=apart(x))
    want = z.rms_norm(x, w, res, EPS, 4, 64)
    assert torch.equal(y, want[0]) and torch.equal(total, want[1]) and torch.equal(codes, want[3])
    del y
    dx, dw = z.rms_norm_grad(apart(dy), total, w, rstd, apart(ds), out=apart(x))
    wx, ww = z.rms_norm_grad(dy, want[1], w, rstd, ds)
    assert torch.equal(dx, wx) and torch.equal(dw, ww)


def test_a_captured_pass_replays(z):
    x, res, dy, ds, w = inputs(8, 300, 2048, BF, F32)
    ws = torch.empty(z.zpp_rms_norm_grad_workspace(300, 2048), dtype=torch.uint8, device="cuda")

    def step():
        y, total, rstd, codes, scales = z.rms_norm(x, w, res, EPS, 8, 128)
        dx, dw = z.rms_norm_grad(dy, total, w, rstd, ds, workspace=ws)
        return y, total, rstd, codes, scales, dx, dw

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    g = torch.Generator(device="cuda").manual_seed(9)
    for _ in range(4):
        for t in (x, res, dy, ds):
            t.copy_(normal(g, 300, 2048))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for a, b in zip(kept, step()):
            assert torch.equal(a, b)


def test_on_a_stream_that_is_behind(z):
    x, res, dy, ds, w = inputs(10, 300, 20480, BF, F32)
    want = z.rms_norm(x, w, res, EPS, 8, 64)
    dwant = z.rms_norm_grad(dy, want[1], w, want[2], ds)
    side = torch.cuda.Stream()
    mine = [t.clone() for t in (x, res, dy, ds, w)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = z.rms_norm(mine[0], mine[4], mine[1], EPS, 8, 64, stream=side)
    dgot = z.rms_norm_grad(mine[2], got[1], mine[4], got[2], mine[3], stream=side)
    del mine
    taken = [torch.full((s,), 255, dtype=torch.uint8, device="cuda")
             for s in (x.numel() * 2, 4 * 20480, z.zpp_rms_norm_grad_workspace(300, 20480)) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((*got, *dgot), (*want, *dwant)):
        assert torch.equal(a, b)
    assert len(taken) == 12
