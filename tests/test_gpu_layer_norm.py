"""Layer norm, forward and backward, on the GPU against its definition in 64 bits."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5

# each kernel's widths and one more or less, odd ones, and rows beyond the registers
WIDTHS = [1, 2, 7, 64, 255, 256, 1000, 2047, 2048, 2049, 2056, 4099, 8192, 8200, 8193, 20000, 32768, 32769, 40004]


@pytest.fixture(scope="module")
def z():
    need_gpu()
    import block_quantization_codec_amd as z

    return z


def inputs(seed, rows, width, xt, wt, pad=0, offset=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = (normal(rows, width + pad) * 2 + offset).to(xt)[:, :width]
    dy = normal(rows, width + pad).to(xt)[:, :width]
    return x, dy, (1 + 0.2 * normal(width)).to(wt), (0.3 * normal(width)).to(wt)


def adds(width):
    """Most binary32 additions one value goes through in a row's sum: a thread's own, then the tree."""
    return (32 if width <= 32768 else -(-width // 1024)) + 6 + 16


def check_forward(z, x, w, b, out=None):
    y, mean, rstd = z.layer_norm(x, w, b, EPS, out=out)
    u = 2.0 ** -24
    xd = x.double()
    m = xd.mean(1, keepdim=True)
    d = xd - m
    r = 1 / ((d * d).mean(1, keepdim=True) + EPS).sqrt()
    wd = 1.0 if w is None else w.double()
    bd = 0.0 if b is None else b.double()
    want = d * r * wd + bd
    n = adds(x.shape[1])
    # sum of a row: n roundings, of at most the sum of magnitudes each; then the product with 1 / width
    dm = (n + 2) * u * xd.abs().mean(1, keepdim=True)
    # squares: the same sum again, of values off by the mean's error (which only adds its square) and 3 roundings
    dr = r * ((n + 8) * u + 0.5 * (dm * r) ** 2)
    assert bool(((mean.double() - m[:, 0]).abs() <= dm[:, 0]).all())
    assert bool(((rstd.double() - r[:, 0]).abs() <= dr[:, 0]).all())
    # y: the errors of mean and rstd, 3 roundings of the product, one of the sum, one to y's type
    tol = (dm * r + (d * r).abs() * (3 * u + dr / r)) * abs(wd) + u * want.abs() + want.abs() * torch.finfo(
        x.dtype).eps / 2 + 1e-37
    off = (y.double() - want).abs()
    assert bool((off <= tol * (1 + 2.0 ** -7)).all()), (tuple(x.shape), (off / tol).max().item())
    return y, mean, rstd


def check_backward(z, dy, x, w, mean, rstd, out=None):
    rows, width = x.shape
    dx, dw, db = z.layer_norm_grad(dy, x, w, mean, rstd, out=out)
    u = 2.0 ** -24
    xd, g0 = x.double(), dy.double()
    m, r = mean.double()[:, None], rstd.double()[:, None]
    xh = (xd - m) * r
    wd = 1.0 if w is None else w.double()
    g = g0 * wd
    a, c = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    want = (g - a - xh * c) * r
    n = adds(width)
    exh = 2 * u * xh.abs()  # x - mean and the product, a rounding each
    ea = (n + 3) * u * g.abs().mean(1, keepdim=True)
    ec = (n + 6) * u * (g * xh).abs().mean(1, keepdim=True)
    # each of the two differences rounds a value of at most the magnitudes' sum
    mag = g.abs() + a.abs() + (xh * c).abs()
    tol = (4 * u * mag + ea + ec * xh.abs() + exh * c.abs()) * r + want.abs() * (u + torch.finfo(x.dtype).eps / 2) + 1e-37
    off = (dx.double() - want).abs()
    assert bool((off <= tol * (1 + 2.0 ** -7)).all()), ((rows, width), (off / tol).max().item())
    # over rows: at most all of them in one thread's sum, plus the units' join
    k = min(rows, 4096) + 72 + 3
    eps = torch.finfo(dw.dtype).eps / 2
    for got, v in ((dw, g0 * xh), (db, g0)):
        want = v.sum(0)
        tol = k * u * v.abs().sum(0) + want.abs() * eps + 1e-37
        off = (got.double() - want).abs()
        assert bool((off <= tol * (1 + 2.0 ** -7)).all()), ((rows, width), (off / tol).max().item())
    return dx, dw, db


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=["bb", "bf", "ff", "fb"])
@pytest.mark.parametrize("width", WIDTHS)
def test_against_64_bits(z, width, types):
    for rows in (1, 3, 67):
        x, dy, w, b = inputs(rows, rows, width, *types)
        _, mean, rstd = check_forward(z, x, w, b)
        check_backward(z, dy, x, w, mean, rstd)


@pytest.mark.parametrize("rows,width", [(5000, 64), (9001, 100), (2500, 4096), (2500, 4097), (700, 16384)])
def test_more_rows_than_units(z, rows, width):
    x, dy, w, b = inputs(1, rows, width, BF, F32)
    _, mean, rstd = check_forward(z, x, w, b)
    check_backward(z, dy, x, w, mean, rstd)


@pytest.mark.parametrize("width", [96, 2052, 9000, 33000])
def test_row_strides_and_no_weights(z, width):
    for xt in (BF, F32):
        for pad in (0, 3, 8):
            x, dy, w, b = inputs(2, 9, width, xt, xt, pad)
            big = torch.full((9, width + 5), 77.0, dtype=xt, device="cuda")
            _, mean, rstd = check_forward(z, x, None, None, out=big[:, :width])
            assert bool((big[:, width:] == 77).all())
            check_backward(z, dy, x, None, mean, rstd, out=big[:, :width])
            assert bool((big[:, width:] == 77).all())
            check_forward(z, x, w, None)
            check_forward(z, x, None, b)


def test_far_mean_and_constant_rows(z):
    """A mean far above the spread: a difference of squares would lose the variance."""
    x, dy, w, b = inputs(3, 8, 4096, F32, F32, offset=3000.0)
    _, mean, rstd = check_forward(z, x, w, b)
    check_backward(z, dy, x, w, mean, rstd)
    x = torch.full((3, 512), 2.0, device="cuda")
    y, mean, rstd = z.layer_norm(x, w[:512].contiguous(), b[:512].contiguous(), EPS)
    assert torch.equal(y, b[:512].expand(3, 512)) and torch.equal(mean, torch.full((3,), 2.0, device="cuda"))
    assert bool((rstd == torch.tensor(EPS, dtype=F32).rsqrt().cuda()).all()) or bool(
        ((rstd.double() * EPS ** 0.5 - 1).abs() < 2.0 ** -22).all())


def test_non_finite_rows_stay_their_own(z):
    x, dy, w, b = inputs(4, 6, 3000, BF, BF)
    y0, _, _ = z.layer_norm(x, w, b, EPS)
    bad = x.clone()
    bad[1, 5], bad[4, 2999] = float("nan"), float("inf")
    y, _, _ = z.layer_norm(bad, w, b, EPS)
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], y0[keep]) and bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[4]).any())


def test_no_rows_gives_zero_weight_gradients(z):
    x = torch.empty(0, 300, dtype=BF, device="cuda")
    w = torch.ones(300, device="cuda")
    y, mean, rstd = z.layer_norm(x, w, w)
    dx, dw, db = z.layer_norm_grad(y, x, w, mean, rstd)
    assert dx.shape == (0, 300) and not dw.any() and not db.any() and dw.dtype == F32


def test_weight_gradient_can_be_left_out(z):
    x, dy, w, b = inputs(5, 33, 512, BF, F32)
    _, mean, rstd = z.layer_norm(x, w, b, EPS)
    dx, dw, db = z.layer_norm_grad(dy, x, w, mean, rstd)
    ws = torch.empty(z.zpp_layer_norm_grad_workspace(33, 512), dtype=torch.uint8, device="cuda")
    for want_w, want_b in ((True, False), (False, True), (False, False)):
        o, ow, ob = torch.empty_like(dx), torch.full_like(dw, 5), torch.full_like(db, 5)
        z.zpp_layer_norm_grad(dy, 512, x, z.ZPP_BF16, 512, 33, 512, w, z.ZPP_FP32, mean, rstd, o, 512,
                              ow if want_w else None, ob if want_b else None, ws, ws.numel())
        assert torch.equal(o, dx)
        assert torch.equal(ow, dw) if want_w else bool((ow == 5).all())
        assert torch.equal(ob, db) if want_b else bool((ob == 5).all())


def test_gradients_against_differences(z):
    """Central differences of the 64-bit forward pass."""
    x, dy, w, b = inputs(6, 5, 48, F32, F32)
    _, mean, rstd = z.layer_norm(x, w, b, EPS)
    dx, dw, db = z.layer_norm_grad(dy, x, w, mean, rstd)

    def loss(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return ((d / ((d * d).mean(1, keepdim=True) + EPS).sqrt() * w + b) * dy.double()).sum()

    at = [t.double() for t in (x, w, b)]
    h = 1e-6
    for i, got in enumerate((dx, dw, db)):
        v = torch.randn(at[i].shape, dtype=torch.float64, device="cuda")
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * v, at[i] - h * v
        slope = ((loss(*up) - loss(*down)) / (2 * h)).item()
        # truncation h^2 and cancellation 2^-53 / h of a loss of order 10^2, and the kernel's 2^-24
        assert abs((got.double() * v).sum().item() - slope) <= 1e-4


def test_linear_and_norm_in_a_graph(z):
    """A step of norm, projection and their backward passes, captured once and
    replayed on new inputs with eager work in between."""
    g = torch.Generator(device="cuda").manual_seed(7)
    k, n, rows, block = 512, 640, 70, 64
    wt = (torch.randn(n, k, generator=g, device="cuda") * 0.02).to(BF)
    codes, scales = z.quantize(wt.view(-1), block, 4)
    x, dy, w, b = inputs(8, rows, k, BF, F32)
    x = x.contiguous()
    dout = torch.randn(rows, n, generator=g, device="cuda").to(BF)

    def step():
        h, mean, rstd = z.layer_norm(x, w, b, EPS)
        y = z.linear(h, codes, scales, 4, block, n)
        one = z.linear(h[:1], codes, scales, 4, block, n, dtype=F32)
        dh = z.linear_grad(dout, codes, scales, 4, block, k)
        return (y, one, *z.layer_norm_grad(dh, x, w, mean, rstd))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        x.copy_(torch.randn(rows, k, generator=g, device="cuda"))
        dout.copy_(torch.randn(rows, n, generator=g, device="cuda"))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, t in zip(outs, want):
            assert torch.equal(got, t), i
