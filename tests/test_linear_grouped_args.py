"""Refusals of the grouped linear entry points, in the pure host checks (fake
addresses: no GPU call is made), their workspace query, and the binding's own."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

A = 1 << 40  # fake device addresses, 16-byte aligned, far apart
G = 1 << 36
BF = torch.bfloat16


@pytest.fixture(scope="module")
def z():
    import block_quantization_codec_amd as z

    return z


def _grouped(z, grad=False, a=A, adt=1, astr=None, rows=4, offsets=A + G, groups=3, codes=A + 2 * G, scales=A + 3 * G,
             bits=4, n=64, k=128, block=32, out=A + 4 * G, odt=1, ostr=None, ws=A + 5 * G, wsb=1 << 30):
    f = z.library().zpp_linear_grouped_grad if grad else z.library().zpp_linear_grouped
    al, ol = (n, k) if grad else (k, n)
    return f(a, adt, al if astr is None else astr, rows, offsets, groups, codes, scales, bits, n, k, block, out, odt,
             ol if ostr is None else ostr, ws, wsb, None)


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_argument_errors(z, grad):
    def call(**kw):
        return _grouped(z, grad, **kw)

    big = (1 << 22) + 32
    for bad in (dict(groups=0), dict(groups=-1), dict(groups=4097), dict(groups=4096, n=1 << 15, k=1 << 14), dict(adt=0),
                dict(odt=3), dict(bits=2), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(n=0), dict(n=-1), dict(n=big),
                dict(k=0), dict(k=48), dict(k=-32), dict(block=16), dict(block=96), dict(n=3, k=32, block=64),
                dict(astr=8), dict(ostr=8), dict(astr=1 << 40, rows=3), dict(wsb=-1)):
        assert call(**bad) == z.ZPP_ERR_ARG, bad
    for bad in (dict(a=None), dict(offsets=None), dict(codes=None), dict(scales=None), dict(out=None)):
        assert call(**bad) == z.ZPP_ERR_NULL, bad
    for bad in (dict(a=A + 8), dict(offsets=A + G + 2), dict(codes=A + 2 * G + 4), dict(scales=A + 3 * G + 2),
                dict(out=A + 4 * G + 2), dict(ostr=132) if grad else dict(astr=132)):
        assert call(**bad) == z.ZPP_ERR_ALIGN, bad
    # the last matrix's codes and scales count, and the last offset
    last = 2 * 64 * 128
    for bad in (dict(out=A), dict(out=A + G), dict(out=A + 2 * G), dict(out=A + 3 * G), dict(out=A + 2 * G + last // 2 + 16),
                dict(scales=A + 4 * G - 4 * (last // 32) - 16), dict(offsets=A + 4 * G - 12)):
        assert call(**bad) == z.ZPP_ERR_OVERLAP, bad
    assert call(rows=0, a=None, codes=None, out=None, offsets=None) == z.ZPP_OK


def test_workspace_is_asked_for_and_checked(z):
    w = z.zpp_linear_grouped_workspace
    need = w(1, 1, 8192, 1, 16, 2, 8192, 1024)
    assert need > 0 and need % 16 == 0
    kw = dict(grad=True, rows=16, groups=2, n=8192, k=1024)
    assert _grouped(z, wsb=need - 1, **kw) == z.ZPP_ERR_ARG
    assert _grouped(z, ws=None, wsb=need, **kw) == z.ZPP_ERR_NULL
    assert _grouped(z, ws=A + 5 * G + 8, wsb=need, **kw) == z.ZPP_ERR_ALIGN
    for at in (A, A + G, A + 2 * G, A + 3 * G, A + 4 * G):
        assert _grouped(z, ws=at, wsb=need, **kw) == z.ZPP_ERR_OVERLAP
    for bad in ((0, 7, 64, 1, 4, 2, 64, 64), (0, 1, 64, 7, 4, 2, 64, 64), (0, 1, 64, 1, -1, 2, 64, 64),
                (0, 1, 64, 1, 4, 0, 64, 64), (0, 1, 64, 1, 4, 4097, 64, 64), (0, 1, 64, 1, 4, 2, 64, 33),
                (0, 1, 63, 1, 4, 2, 64, 64), (0, 1, 64, 1, 0, 2, 64, 64)):
        assert w(*bad) == 0


def test_binding_refuses_what_the_kernels_would_misread(z):
    codes, scales = torch.zeros(2 * 64 * 16, dtype=torch.uint8), torch.ones(2 * 64)  # two of 64 x 32, 4 bits, block 32
    x, o = torch.zeros(4, 32, dtype=BF), torch.tensor([0, 1, 4], dtype=torch.int32)
    for bad in (o.float(), o.long()):
        with pytest.raises(TypeError):
            z.linear_grouped(x, bad, codes, scales, 4, 32, 64)
    for bad in (o[:2], o[:1], o.view(1, 3), torch.zeros(6, dtype=torch.int32)[::2],
                torch.zeros(4, dtype=torch.int32)):                 # too few groups, none, a matrix, strides, too many
        with pytest.raises(ValueError):
            z.linear_grouped(x, bad, codes, scales, 4, 32, 64)
    with pytest.raises(ValueError):
        z.linear_grouped_grad(x, o, codes, scales, 4, 32, 32)       # dy must have 64 columns
    with pytest.raises(ValueError):
        z.linear_grouped(x, o, codes, scales, 4, 32, 64, out=torch.zeros(4, 63, dtype=BF))
