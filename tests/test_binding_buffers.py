"""The binding's checks of the buffers that a caller hands to the helpers (no GPU call is made)."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def z():
    import block_quantization_codec_amd as z

    return z


@pytest.mark.parametrize("view", [lambda t: t[::2], lambda t: t[:1].expand(1 << 20), lambda t: t.view(-1, 64)[:, :32]],
                         ids=["every other byte", "one byte expanded", "half rows"])
def test_a_workspace_with_gaps_or_repeats_is_refused(z, view, monkeypatch):
    """Its elements are fewer, or further apart, than the bytes the kernels would take."""
    monkeypatch.setattr(z, "_call", lambda *args: pytest.fail("the call was made"))
    ws = view(torch.zeros(1 << 20, dtype=torch.uint8))
    codes, scales = torch.zeros(64 * 16, dtype=torch.uint8), torch.ones(64)
    x, dy, stats = torch.zeros(40, 32), torch.zeros(40, 64), torch.ones(40)
    with pytest.raises(ValueError):
        z.linear(x, codes, scales, 4, 32, 64, workspace=ws)
    with pytest.raises(ValueError):
        z.linear_grad(dy, codes, scales, 4, 32, 32, workspace=ws)
    with pytest.raises(ValueError):
        z.layer_norm_grad(x, x, None, stats, stats, workspace=ws)


def test_norm_results_go_where_they_are_asked_for(z, monkeypatch):
    calls = []
    monkeypatch.setattr(z, "_call", lambda name, *args: calls.append(args))
    monkeypatch.setattr(z, "_stream", lambda stream: 0)
    x, w, mean, rstd = torch.zeros(5, 8, 32), torch.ones(32, dtype=torch.bfloat16), torch.empty(5, 8), torch.empty(5, 8)
    _, m, r = z.layer_norm(x, w, w, mean=mean, rstd=rstd)
    assert m is mean and r is rstd and calls[-1][-3:-1] == (mean.data_ptr(), rstd.data_ptr())
    dw, db = torch.empty_like(w), torch.empty_like(w)
    _, a, b = z.layer_norm_grad(x, x, w, mean, rstd, dweight=dw, dbias=db)
    assert a is dw and b is db and calls[-1][-5:-3] == (dw.data_ptr(), db.data_ptr())
    n = len(calls)
    for bad in (torch.empty(5, 7), torch.empty(40), torch.empty(5, 8, dtype=torch.float64), torch.empty(8, 5).t()):
        with pytest.raises(ValueError):
            z.layer_norm(x, w, w, mean=bad)
        with pytest.raises(ValueError):
            z.layer_norm(x, w, w, rstd=bad)
    for bad in (torch.empty(32), dw[:31], torch.empty(64, dtype=dw.dtype)[::2]):
        with pytest.raises(ValueError):
            z.layer_norm_grad(x, x, w, mean, rstd, dweight=bad)
        with pytest.raises(ValueError):
            z.layer_norm_grad(x, x, w, mean, rstd, dbias=bad)
    assert len(calls) == n


def test_workspace_of_far_rows(z):
    """Rows more than 2^22 elements apart are packed: a query with another stride is no answer for them."""
    w = z.zpp_linear_blocks_workspace
    near, edge, far = (w(0, z.ZPP_BF16, s, z.ZPP_BF16, 4096, 8192, 1024) for s in (1024, 1 << 22, (1 << 22) + 8))
    assert near == edge == 0 and far == 4096 * 1024 * 2
    # and a query for many rows is none for few: 8 rows have a split contraction, 4096 none
    assert w(0, z.ZPP_BF16, 8192, z.ZPP_BF16, 8, 1024, 8192) > w(0, z.ZPP_BF16, 8192, z.ZPP_BF16, 4096, 8192, 8192) == 0
    f = z.library().zpp_linear_blocks
    a, g = 1 << 40, 1 << 36  # fake addresses: refused before any GPU call is made
    assert f(a, z.ZPP_BF16, (1 << 22) + 8, 4096, a + g, a + 2 * g, 4, 8192, 1024, 128, a + 3 * g, z.ZPP_BF16, 8192,
             a + 4 * g, far - 1, None) == z.ZPP_ERR_ARG
