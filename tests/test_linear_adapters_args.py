"""Refusals of the linear products with adapters, in the pure host checks (fake
addresses: no GPU call is made), their workspace query, and the binding's own."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

A = 1 << 40  # fake device addresses, 16-byte aligned, far apart
G = 1 << 36
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def z():
    import block_quantization_codec_amd as z

    return z


def _forward(z, x=A, xdt=1, xs=None, rows=4, codes=A + G, scales=A + 2 * G, bits=4, n=64, k=128, block=32, a=A + 3 * G,
             b=A + 4 * G, wdt=1, adapters=3, rank=16, ids=A + 5 * G, scaling=A + 6 * G, reduced=A + 7 * G, y=A + 8 * G,
             ydt=1, ys=None, ws=A + 9 * G, wsb=1 << 30):
    return z.library().zpp_linear_adapters(x, xdt, k if xs is None else xs, rows, codes, scales, bits, n, k, block, a, b,
                                           wdt, adapters, rank, ids, scaling, reduced, y, ydt, n if ys is None else ys,
                                           ws, wsb, None)


def _grad(z, dy=A, dydt=1, dys=None, x=A + G, xs=None, reduced=A + 2 * G, rows=4, codes=A + 3 * G, scales=A + 4 * G,
          bits=4, n=64, k=128, block=32, a=A + 5 * G, b=A + 6 * G, wdt=1, adapters=3, rank=16, ids=A + 7 * G,
          scaling=A + 8 * G, dx=A + 9 * G, dxdt=1, dxs=None, da=A + 10 * G, db=A + 11 * G, ws=A + 12 * G, wsb=1 << 30):
    return z.library().zpp_linear_adapters_grad(dy, dydt, n if dys is None else dys, x, k if xs is None else xs, reduced,
                                                rows, codes, scales, bits, n, k, block, a, b, wdt, adapters, rank, ids,
                                                scaling, dx, dxdt, k if dxs is None else dxs, da, db, ws, wsb, None)


SIZES = [dict(bits=2), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(n=0), dict(n=(1 << 22) + 32), dict(k=0), dict(k=48),
         dict(block=16), dict(block=96), dict(n=3, k=32, block=64), dict(wdt=0), dict(wdt=3), dict(adapters=0),
         dict(adapters=-1), dict(adapters=4097), dict(rank=0), dict(rank=-8), dict(rank=4), dict(rank=12), dict(rank=264),
         dict(adapters=4096, rank=256, n=(1 << 20) + 32, k=32), dict(wsb=-1)]


def test_forward_argument_errors(z):
    for bad in SIZES + [dict(xdt=0), dict(ydt=9), dict(xs=120), dict(ys=60), dict(xs=1 << 40, rows=3)]:
        assert _forward(z, **bad) == z.ZPP_ERR_ARG, bad
    for name in ("x", "codes", "scales", "a", "b", "reduced", "y"):
        assert _forward(z, **{name: None}) == z.ZPP_ERR_NULL, name
    for bad in (dict(x=A + 8), dict(codes=A + G + 4), dict(scales=A + 2 * G + 2), dict(a=A + 3 * G + 8),
                dict(b=A + 4 * G + 8), dict(ids=A + 5 * G + 2), dict(scaling=A + 6 * G + 1), dict(reduced=A + 7 * G + 8),
                dict(y=A + 8 * G + 2), dict(xs=132)):
        assert _forward(z, **bad) == z.ZPP_ERR_ALIGN, bad
    for o, me in (("reduced", 7), ("y", 8)):
        for i in range(9):
            if i != me:
                assert _forward(z, **{o: A + i * G}) == z.ZPP_ERR_OVERLAP, (o, i)
    assert _forward(z, rows=0, x=None, codes=None, a=None, b=None, reduced=None, y=None, ws=None, wsb=0) == z.ZPP_OK


def test_grad_argument_errors(z):
    for bad in SIZES + [dict(dydt=0), dict(dxdt=9), dict(dys=60), dict(xs=120), dict(dxs=120), dict(dys=1 << 40, rows=3)]:
        assert _grad(z, **bad) == z.ZPP_ERR_ARG, bad
    for name in ("dy", "x", "reduced", "codes", "scales", "a", "b", "dx", "ws"):
        assert _grad(z, **{name: None}) == z.ZPP_ERR_NULL, name
    for bad in (dict(dy=A + 8), dict(x=A + G + 8), dict(reduced=A + 2 * G + 4), dict(codes=A + 3 * G + 4),
                dict(scales=A + 4 * G + 2), dict(a=A + 5 * G + 8), dict(b=A + 6 * G + 8), dict(ids=A + 7 * G + 2),
                dict(scaling=A + 8 * G + 1), dict(dx=A + 9 * G + 2), dict(da=A + 10 * G + 4), dict(db=A + 11 * G + 4),
                dict(ws=A + 12 * G + 8), dict(dxs=132)):
        assert _grad(z, **bad) == z.ZPP_ERR_ALIGN, bad
    for o, me in (("dx", 9), ("da", 10), ("db", 11), ("ws", 12)):
        for i in range(13):
            if i != me:
                assert _grad(z, **{o: A + i * G}) == z.ZPP_ERR_OVERLAP, (o, i)
    need = z.zpp_linear_adapters_workspace(1, 1, 64, 1, 4, 64, 128, 3, 16)
    assert need >= 4 * 16 * 4 and _grad(z, wsb=need - 1) == z.ZPP_ERR_ARG
    nothing = dict(rows=0, dy=None, x=None, reduced=None, codes=None, a=None, b=None, dx=None, da=None, db=None)
    assert _grad(z, **nothing) == z.ZPP_OK


def test_grad_without_x_takes_any_stride_of_it(z):
    for xs in (0, -1, 120, 1 << 41):
        # past the arguments: dx on dy is what is refused
        assert _grad(z, x=None, da=None, xs=xs, dx=A) == z.ZPP_ERR_OVERLAP, xs
        assert _grad(z, da=None, xs=xs, dx=A) == z.ZPP_ERR_ARG, xs
        assert _grad(z, x=None, xs=xs) == z.ZPP_ERR_NULL, xs


def test_workspace_is_asked_for_and_checked(z):
    w = z.zpp_linear_adapters_workspace
    need = w(0, 1, 8192, 1, 16, 8192, 8192, 2, 64)
    assert need > 0 and need % 16 == 0
    kw = dict(rows=16, n=8192, k=8192, adapters=2, rank=64)
    assert _forward(z, wsb=need - 1, **kw) == z.ZPP_ERR_ARG
    assert _forward(z, ws=None, wsb=need, **kw) == z.ZPP_ERR_NULL
    assert _forward(z, ws=A + 9 * G + 8, wsb=need, **kw) == z.ZPP_ERR_ALIGN
    for i in range(9):
        assert _forward(z, ws=A + i * G, wsb=need, **kw) == z.ZPP_ERR_OVERLAP
    for bad in ((0, 7, 64, 1, 4, 64, 64, 1, 8), (0, 1, 64, 7, 4, 64, 64, 1, 8), (0, 1, 64, 1, -1, 64, 64, 1, 8),
                (0, 1, 64, 1, 4, 64, 33, 1, 8), (0, 1, 63, 1, 4, 64, 64, 1, 8), (0, 1, 64, 1, 4, 64, 64, 0, 8),
                (0, 1, 64, 1, 4, 64, 64, 1, 7), (0, 1, 64, 1, 4, 64, 64, 1, 512), (0, 1, 64, 1, 0, 64, 64, 1, 8)):
        assert w(*bad) == 0


def test_binding_refuses_what_the_kernels_would_misread(z):
    codes, scales = torch.zeros(64 * 16, dtype=torch.uint8), torch.ones(64)  # 64 x 32, 4 bits, block 32
    x, dy = torch.zeros(4, 32, dtype=BF), torch.zeros(4, 64, dtype=BF)
    a, b = torch.zeros(3, 8, 32, dtype=BF), torch.zeros(3, 64, 8, dtype=BF)
    ids, s, t = torch.zeros(4, dtype=I32), torch.ones(3), torch.zeros(4, 8)

    def forward(**kw):
        v = dict(x=x, a=a, b=b, ids=ids, scaling=s) | kw
        z.linear_adapters(v.pop("x"), codes, scales, 4, 32, 64, v.pop("a"), v.pop("b"), **v)

    def back(**kw):
        v = dict(dy=dy, x=x, reduced=t, a=a, b=b, ids=ids, scaling=s) | kw
        z.linear_adapters_grad(v.pop("dy"), v.pop("x"), v.pop("reduced"), codes, scales, 4, 32, v.pop("a"), v.pop("b"),
                               **v)

    for f in (forward, back):
        for kw in (dict(a=a[:2]), dict(a=a[:, :4]), dict(a=a[..., :16]), dict(b=b[:, :32]), dict(a=a[0]),
                   dict(b=b.transpose(1, 2)), dict(b=b.transpose(1, 2).contiguous().transpose(1, 2)),
                   dict(ids=ids[:3]), dict(ids=ids.long()), dict(ids=torch.zeros(8, dtype=I32)[::2]),
                   dict(scaling=s[:2]), dict(scaling=s.double())):
            with pytest.raises(ValueError):
                f(**kw)
        with pytest.raises(TypeError):
            f(a=a.float())
        with pytest.raises(TypeError):
            f(a=a.half(), b=b.half())
    for kw in (dict(out=torch.zeros(4, 63, dtype=BF)), dict(reduced=t[:, :4]), dict(reduced=t.to(BF))):
        with pytest.raises(ValueError):
            forward(**kw)
    for kw in (dict(out=dy), dict(x=x.float()), dict(x=x[:2]), dict(reduced=t[:2]), dict(reduced=t.double()),
               dict(da=b), dict(db=b.float()), dict(want_adapters=False, da=a)):
        with pytest.raises(ValueError):
            back(**kw)
