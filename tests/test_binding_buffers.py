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
