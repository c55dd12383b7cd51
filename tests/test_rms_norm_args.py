"""Refusals of the RMS norm's entry points, in the pure host checks (fake
addresses: no GPU call is made), and the binding's own."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

A = 1 << 40  # fake device addresses, 16-byte aligned, far apart
G = 1 << 36
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def z():
    import block_quantization_codec_amd as z

    return z


def _norm(z, x=A, xdt=1, xs=128, res=A + G, rs=128, rows=4, width=128, w=A + 2 * G, wdt=2, eps=1e-5, total=A + 3 * G,
          ts=128, y=A + 4 * G, ys=128, codes=A + 5 * G, scales=A + 6 * G, bits=8, block=32, rstd=A + 7 * G):
    return z.library().zpp_rms_norm(x, xdt, xs, res, rs, rows, width, w, wdt, eps, total, ts, y, ys, codes, scales,
                                    bits, block, rstd, None)


def test_argument_errors(z):
    nan, inf, far = float("nan"), float("inf"), 1 << 40
    for bad in (dict(xdt=0), dict(wdt=9), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(width=0), dict(width=-4),
                dict(width=(1 << 22) + 1), dict(xs=127), dict(rs=127), dict(ts=127), dict(ys=127), dict(xs=far + 1),
                dict(xs=far, rows=3), dict(rs=far, rows=3), dict(ts=far, rows=3), dict(ys=far, rows=3),
                dict(eps=-1e-9), dict(eps=nan), dict(eps=inf), dict(bits=2), dict(bits=16), dict(block=0),
                dict(block=16), dict(block=48), dict(block=256), dict(block=8192), dict(bits=0),
                dict(bits=0, codes=None), dict(bits=0, scales=None), dict(res=None),
                dict(y=None, bits=0, codes=None, scales=None)):
        assert _norm(z, **bad) == z.ZPP_ERR_ARG, bad
    for bad in (dict(x=None), dict(rstd=None), dict(codes=None), dict(scales=None)):
        assert _norm(z, **bad) == z.ZPP_ERR_NULL, bad
    for name, at, off in (("x", A, 8), ("res", A + G, 2), ("w", A + 2 * G, 4), ("total", A + 3 * G, 8),
                          ("y", A + 4 * G, 4), ("codes", A + 5 * G, 8), ("scales", A + 6 * G, 2),
                          ("rstd", A + 7 * G, 1)):
        assert _norm(z, **{name: at + off}) == z.ZPP_ERR_ALIGN, name
    outs = ("total", "y", "codes", "scales", "rstd")
    for o in outs:
        for at in (A, A + 16, A + G, A + 2 * G):  # on x, the residual, the weight
            assert _norm(z, **{o: at}) == z.ZPP_ERR_OVERLAP, (o, at)
        for i, other in enumerate(outs):
            if other != o:
                assert _norm(z, **{o: A + (3 + i) * G}) == z.ZPP_ERR_OVERLAP, (o, other)
    assert _norm(z, rows=0, x=None, res=None, total=None, y=None, codes=None, scales=None, rstd=None) == z.ZPP_OK


def _grad(z, dy=A, dys=128, h=A + G, xdt=1, hs=128, ds=A + 2 * G, dss=128, rows=4, width=128, w=A + 3 * G, wdt=2,
          rstd=A + 4 * G, dx=A + 5 * G, dxs=128, dw=A + 6 * G, ws=A + 7 * G, wsb=1 << 20):
    return z.library().zpp_rms_norm_grad(dy, dys, h, xdt, hs, ds, dss, rows, width, w, wdt, rstd, dx, dxs, dw, ws, wsb,
                                         None)


def test_grad_argument_errors(z):
    need = z.zpp_rms_norm_grad_workspace(4, 128)
    assert need > 0
    for bad in (dict(xdt=0), dict(wdt=0), dict(rows=-1), dict(width=0), dict(dys=100), dict(hs=100), dict(dxs=100),
                dict(dss=100), dict(hs=1 << 40, rows=3), dict(wsb=need - 1), dict(wsb=-1)):
        assert _grad(z, **bad) == z.ZPP_ERR_ARG, bad
    for bad in (dict(dy=None), dict(h=None), dict(rstd=None), dict(dx=None), dict(ws=None)):
        assert _grad(z, **bad) == z.ZPP_ERR_NULL, bad
    for bad in (dict(dy=A + 2), dict(h=A + G + 2), dict(ds=A + 2 * G + 4), dict(w=A + 3 * G + 4), dict(dx=A + 5 * G + 8),
                dict(dw=A + 6 * G + 4), dict(ws=A + 7 * G + 4), dict(rstd=A + 4 * G + 2)):
        assert _grad(z, **bad) == z.ZPP_ERR_ALIGN, bad
    for o, me in (("dx", 5), ("dw", 6), ("ws", 7)):
        for i in range(8):
            if i != me:
                assert _grad(z, **{o: A + i * G}) == z.ZPP_ERR_OVERLAP, (o, i)
    assert _grad(z, rows=0, dw=None, dy=None, h=None, ds=None, dx=None, rstd=None, ws=None, wsb=0) == z.ZPP_OK
    assert z.zpp_rms_norm_grad_workspace(0, 128) == 0
    assert z.zpp_rms_norm_grad_workspace(4, 0) == 0
    assert z.zpp_rms_norm_grad_workspace(4, (1 << 22) + 1) == 0


def test_binding_refuses_what_the_kernels_would_misread(z):
    x, w, r = torch.zeros(4, 96, dtype=BF), torch.ones(96), torch.ones(4)
    for kw in (dict(weight=torch.ones(95)), dict(weight=torch.ones(192)[::2]), dict(residual=x.float()),
               dict(residual=x[:2]), dict(residual=torch.zeros(96, 4, dtype=BF).t()), dict(bits=8, block=64),
               dict(bits=8), dict(bits=3, block=32), dict(total=x), dict(want_y=False, out=x), dict(codes=x),
               dict(out=x.float()), dict(rstd=torch.ones(3)), dict(rstd=torch.ones(4, dtype=BF)),
               dict(bits=8, block=32, codes=torch.zeros(4 * 95, dtype=torch.uint8)),
               dict(bits=8, block=32, scales=torch.zeros(11))):
        with pytest.raises(ValueError):
            z.rms_norm(x, **kw)
    with pytest.raises(TypeError):
        z.rms_norm(x.half())
    with pytest.raises(TypeError):
        z.rms_norm(x, w.double())
    for kw in (dict(dy=x.float()), dict(dy=x[:2]), dict(rstd=r[:3]), dict(rstd=r.double()), dict(dsum=x[:3]),
               dict(weight=w[:95]), dict(out=x.float()), dict(dweight=w.to(BF))):
        with pytest.raises(ValueError):
            z.rms_norm_grad(**{"dy": x, "x": x, "weight": w, "rstd": r, **kw})
