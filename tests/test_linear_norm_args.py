"""Refusals of the linear and layer-norm entry points, in the pure host checks
(fake addresses: no GPU call is made), their workspace queries, and the
binding's own checks."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

A = 1 << 40  # fake device addresses, 16-byte aligned, far apart
G = 1 << 36


@pytest.fixture(scope="module")
def z():
    import block_quantization_codec_amd as z

    return z


def _linear(z, grad=False, a=A, adt=1, astr=None, rows=4, codes=A + G, scales=A + 2 * G, bits=4, n=64, k=128, block=32,
            out=A + 3 * G, odt=1, ostr=None, ws=None, wsb=0):
    f = z.library().zpp_linear_blocks_grad if grad else z.library().zpp_linear_blocks
    al, ol = (n, k) if grad else (k, n)
    return f(a, adt, al if astr is None else astr, rows, codes, scales, bits, n, k, block, out, odt,
             ol if ostr is None else ostr, ws, wsb, None)


@pytest.mark.parametrize("grad", [False, True])
def test_linear_argument_errors(z, grad):
    def call(**kw):
        kw.setdefault("ws", A + 4 * G)
        kw.setdefault("wsb", 1 << 30)
        return _linear(z, grad, **kw)

    big = (1 << 22) + 32
    for bad in (dict(adt=0), dict(adt=3), dict(odt=0), dict(odt=-1), dict(bits=2), dict(bits=16), dict(rows=-1),
                dict(rows=(1 << 30) + 1), dict(n=0), dict(n=-1), dict(n=big), dict(k=0), dict(k=16), dict(k=48),
                dict(k=-32), dict(k=big), dict(n=1 << 22, k=1 << 22), dict(block=16), dict(block=8192),
                dict(block=96), dict(n=3, k=32, block=64), dict(astr=8), dict(ostr=8), dict(astr=-128),
                dict(astr=(1 << 40) + 8), dict(astr=1 << 40, rows=3), dict(ostr=1 << 40, rows=3), dict(wsb=-1)):
        assert call(**bad) == z.ZPP_ERR_ARG, bad
    for bad in (dict(a=None), dict(codes=None), dict(scales=None), dict(out=None)):
        assert call(**bad) == z.ZPP_ERR_NULL, bad
    for bad in (dict(a=A + 8), dict(codes=A + G + 4), dict(scales=A + 2 * G + 2), dict(out=A + 3 * G + 2),
                dict(ostr=132, odt=1) if grad else dict(astr=132, adt=1),
                dict(ostr=130, odt=2) if grad else dict(astr=130, adt=2)):
        assert call(**bad) == z.ZPP_ERR_ALIGN, bad
    for bad in (dict(out=A), dict(out=A + 256), dict(out=A + G), dict(out=A + 2 * G), dict(a=A + 3 * G + 16)):
        assert call(**bad) == z.ZPP_ERR_OVERLAP, bad
    assert call(rows=0, a=None, codes=None, out=None) == z.ZPP_OK


def test_linear_workspace_is_asked_for_and_checked(z):
    w = z.zpp_linear_blocks_workspace
    need = w(1, 1, 8192, 1, 16, 8192, 1024)  # one row of tiles, a long contraction: split
    assert need > 0 and need % 16 == 0
    kw = dict(grad=True, rows=16, n=8192, k=1024)
    assert _linear(z, ws=A + 4 * G, wsb=need - 1, **kw) == z.ZPP_ERR_ARG
    assert _linear(z, ws=None, wsb=need, **kw) == z.ZPP_ERR_NULL
    assert _linear(z, ws=A + 4 * G + 8, wsb=need, **kw) == z.ZPP_ERR_ALIGN
    for at in (A, A + G, A + 2 * G, A + 3 * G):  # on the input, the codes, the scales, the output
        assert _linear(z, ws=at, wsb=need, **kw) == z.ZPP_ERR_OVERLAP
    assert w(0, 1, 8192, 1, 1, 8192, 8192) == 0      # one token
    assert w(0, 1, 8192, 1, 0, 8192, 8192) == 0      # no rows
    assert w(1, 1, 8192, 1, 4096, 8192, 8192) == 0   # enough tiles, rows on 16-byte pieces
    # odd strides, odd lengths and binary32 are packed: rows of whole 64s, two bytes an element and part
    assert w(1, 1, 8193, 1, 4096, 8192, 8192) == 4096 * 8192 * 2
    assert w(1, 1, 8131, 1, 4096, 8131, 8192) == 4096 * 8192 * 2
    assert w(1, 2, 8192, 1, 4096, 8192, 8192) == 4096 * 8192 * 2 * 3
    for bad in ((0, 7, 64, 1, 4, 64, 64), (0, 1, 64, 7, 4, 64, 64), (0, 1, 64, 1, -1, 64, 64), (0, 1, 64, 1, 4, 0, 64),
                (0, 1, 64, 1, 4, 64, 33), (0, 1, 63, 1, 4, 64, 64)):
        assert w(*bad) == 0


def _norm(z, x=A, xdt=1, xs=128, rows=4, width=128, w=A + G, b=A + 2 * G, wdt=2, eps=1e-5, y=A + 3 * G, ys=128,
          mean=A + 4 * G, rstd=A + 5 * G):
    return z.library().zpp_layer_norm(x, xdt, xs, rows, width, w, b, wdt, eps, y, ys, mean, rstd, None)


def test_layer_norm_argument_errors(z):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(xdt=0), dict(wdt=9), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(width=0), dict(width=-4),
                dict(width=(1 << 22) + 1), dict(xs=127), dict(ys=127), dict(xs=(1 << 40) + 1),
                dict(xs=1 << 40, rows=3), dict(eps=-1e-9), dict(eps=nan), dict(eps=inf)):
        assert _norm(z, **bad) == z.ZPP_ERR_ARG, bad
    for bad in (dict(x=None), dict(y=None), dict(mean=None), dict(rstd=None)):
        assert _norm(z, **bad) == z.ZPP_ERR_NULL, bad
    for bad in (dict(x=A + 2), dict(w=A + G + 4), dict(b=A + 2 * G + 8), dict(y=A + 3 * G + 4), dict(mean=A + 4 * G + 2),
                dict(rstd=A + 5 * G + 1)):
        assert _norm(z, **bad) == z.ZPP_ERR_ALIGN, bad
    for bad in (dict(y=A), dict(y=A + G), dict(y=A + 2 * G + 16), dict(mean=A + 4), dict(rstd=A + 4 * G + 8),
                dict(mean=A + 3 * G + 8)):
        assert _norm(z, **bad) == z.ZPP_ERR_OVERLAP, bad
    assert _norm(z, rows=0, x=None, y=None, mean=None, rstd=None) == z.ZPP_OK


def _norm_grad(z, dy=A, dys=128, x=A + G, xdt=1, xs=128, rows=4, width=128, w=A + 2 * G, wdt=2, mean=A + 3 * G,
               rstd=A + 4 * G, dx=A + 5 * G, dxs=128, dw=A + 6 * G, db=A + 7 * G, ws=A + 8 * G, wsb=1 << 20):
    return z.library().zpp_layer_norm_grad(dy, dys, x, xdt, xs, rows, width, w, wdt, mean, rstd, dx, dxs, dw, db, ws,
                                           wsb, None)


def test_layer_norm_grad_argument_errors(z):
    need = z.zpp_layer_norm_grad_workspace(4, 128)
    assert need > 0
    for bad in (dict(xdt=0), dict(wdt=0), dict(rows=-1), dict(width=0), dict(dys=100), dict(xs=100), dict(dxs=100),
                dict(xs=1 << 40, rows=3), dict(wsb=need - 1), dict(wsb=-1)):
        assert _norm_grad(z, **bad) == z.ZPP_ERR_ARG, bad
    for bad in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(ws=None)):
        assert _norm_grad(z, **bad) == z.ZPP_ERR_NULL, bad
    for bad in (dict(dy=A + 2), dict(x=A + G + 2), dict(w=A + 2 * G + 4), dict(dx=A + 5 * G + 8), dict(dw=A + 6 * G + 4),
                dict(db=A + 7 * G + 4), dict(ws=A + 8 * G + 4), dict(mean=A + 3 * G + 2), dict(rstd=A + 4 * G + 2)):
        assert _norm_grad(z, **bad) == z.ZPP_ERR_ALIGN, bad
    for bad in (dict(dx=A), dict(dx=A + G), dict(dw=A + 2 * G), dict(db=A + 3 * G), dict(ws=A + 4 * G), dict(dw=A + 5 * G),
                dict(db=A + 6 * G), dict(ws=A + 7 * G)):
        assert _norm_grad(z, **bad) == z.ZPP_ERR_OVERLAP, bad
    assert _norm_grad(z, rows=0, dw=None, db=None, dy=None, x=None, dx=None, mean=None, rstd=None, ws=None,
                      wsb=0) == z.ZPP_OK
    assert z.zpp_layer_norm_grad_workspace(0, 128) == 0
    assert z.zpp_layer_norm_grad_workspace(4, 0) == 0


def test_binding_refuses_what_the_kernels_would_misread(z):
    codes, scales = torch.zeros(64 * 16, dtype=torch.uint8), torch.ones(64)  # 64 x 32 weights, 4 bits, block 32
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        z.linear(x, codes, scales, 4, 32, 32)                      # as many weights as half the codes
    with pytest.raises(ValueError):
        z.linear(x, codes, scales[:32], 4, 32, 64)                 # too few scales
    with pytest.raises(ValueError):
        z.linear(x.t().contiguous().t(), codes, scales, 4, 32, 64)  # columns, not rows, contiguous
    with pytest.raises(ValueError):
        z.linear(x, codes[::2], scales, 4, 32, 64)                 # strided codes
    with pytest.raises(TypeError):
        z.linear(x.half(), codes, scales, 4, 32, 64)
    with pytest.raises(TypeError):
        z.linear(x, codes, scales.double(), 4, 32, 64)
    with pytest.raises(ValueError):
        z.linear(x, codes, scales, 4, 32, 64, out=torch.zeros(4, 63, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        z.linear_grad(x, codes, scales, 4, 32, 32)                 # dy must have 64 columns
    with pytest.raises(ValueError):
        z.layer_norm(x, torch.ones(31))
    with pytest.raises(TypeError):
        z.layer_norm(x, torch.ones(32), torch.zeros(32, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        z.layer_norm(x[:, ::2])
    with pytest.raises(ValueError):
        z.layer_norm(x, out=torch.zeros(4, 32))
    with pytest.raises(ValueError):
        z.layer_norm_grad(x[:2], x, None, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError):
        z.layer_norm_grad(x, x, None, torch.zeros(3), torch.zeros(4))
    assert z._rows(torch.zeros(2, 3, 8)[:, :, :4], "x") == (6, 4, 8)
    assert z._rows(torch.zeros(5, 8)[::2], "x") == (3, 8, 16)
    with pytest.raises(ValueError):
        z._rows(torch.zeros(2, 3, 8)[:, :2], "x")                  # two strides
