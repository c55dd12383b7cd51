"""Layer norm where every unit of threads walks over several rows, and a row that is not finite among them."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402
from test_gpu_layer_norm import BF, EPS, F32, check_backward, check_forward, inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    need_gpu()
    import block_quantization_codec_amd as z

    return z


# rows held in registers, of whole 16-byte pieces and not; bf16 rows whose weights are read again for each;
# rows that are read again for every sum (all more than 512 rows), and backward by columns in 128 shares
SHAPES = [(9001, 100), (9001, 512), (5000, 2048), (2500, 4096), (2500, 4099), (1300, 8192), (1300, 8190), (1100, 16384),
          (1100, 16383), (1100, 20000), (1100, 20001), (1100, 32768), (2100, 16388), (1100, 32769), (600, 40004)]


@pytest.mark.parametrize("types", [(BF, BF), (F32, F32), (F32, BF)], ids=["bb", "ff", "fb"])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_units_of_many_rows(z, rows, width, types):
    x, dy, w, b = inputs(rows + width, rows, width, *types)
    # rows of sizes of their own, so that a row's mean or rstd taken for another's shows
    x = (x.float() * torch.linspace(0.5, 2.0, rows, device="cuda")[:, None] +
         torch.linspace(-1.0, 1.0, rows, device="cuda")[:, None]).to(types[0])
    _, mean, rstd = check_forward(z, x, w, b)
    check_backward(z, dy, x, w, mean, rstd)


@pytest.mark.parametrize("types", [(BF, BF), (F32, F32)], ids=["bb", "ff"])
@pytest.mark.parametrize("rows,width", [(1100, 96), (700, 3000), (1100, 16384), (1100, 20001)])
def test_a_non_finite_row_of_the_gradient_stays_its_own(z, rows, width, types):
    x, dy, w, b = inputs(3, rows, width, *types)
    _, mean, rstd = z.layer_norm(x, w, b, EPS)
    dx0, dw0, db0 = z.layer_norm_grad(dy, x, w, mean, rstd)
    row, col = rows - 3, 7
    for value in (float("inf"), float("nan")):
        bad = dy.clone()
        bad[row, col] = value
        dx, dw, db = z.layer_norm_grad(bad, x, w, mean, rstd)
        keep = torch.arange(rows, device="cuda") != row
        assert torch.equal(dx[keep], dx0[keep]) and not bool(torch.isfinite(dx[row, col]))
        cols = torch.arange(width, device="cuda") != col
        assert torch.equal(dw[cols], dw0[cols]) and torch.equal(db[cols], db0[cols])
        assert not bool(torch.isfinite(dw[col])) and not bool(torch.isfinite(db[col]))
    bad_mean, bad_rstd = mean.clone(), rstd.clone()  # what a row with NaN in x leaves
    bad_mean[row] = bad_rstd[row] = float("nan")
    dx, _, db = z.layer_norm_grad(dy, x, w, bad_mean, bad_rstd)
    assert torch.equal(dx[keep], dx0[keep]) and torch.equal(db, db0) and bool(torch.isnan(dx[row]).all())
