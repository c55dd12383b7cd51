"""Linear products with low-rank adapters, forward and backward, on the GPU against 64 bits.

With small whole numbers and bf16 everywhere every sum is exact, so results equal
the 64-bit ones, rounded once; real numbers are held to the roundings that the
formulas make.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402
from test_gpu_linear import gen, weights  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def z():
    need_gpu()
    import block_quantization_codec_amd as z

    return z


def make_ids(kind, rows, adapters, g):
    """None, one adapter for all, neighbouring runs, or any at all: with some rows that have none."""
    if kind == "null":
        return None
    if kind == "one":
        return torch.full((rows,), adapters - 1, dtype=I32, device="cuda")
    if kind == "none":
        return torch.full((rows,), -1, dtype=I32, device="cuda")
    if kind == "runs":
        r = torch.arange(rows, device="cuda") * 5 // max(rows, 1)
        return ((r * 7) % (adapters + 1) - 1).to(I32)
    ids = torch.randint(-1, adapters, (rows,), generator=g, device="cuda").to(I32)
    ids[::7] = adapters          # numbers of no adapter
    ids[3::11] = -(1 << 31)
    ids[5::13] = (1 << 31) - 1
    return ids


def dense(z, ids, rows, adapters):
    """[rows] adapter numbers as int64, -1 for none."""
    if ids is None:
        return torch.zeros(rows, dtype=torch.int64, device="cuda")
    i = ids.long()
    return torch.where((i >= 0) & (i < adapters), i, -1)


def select(t, at, adapters):
    """[rows, adapters, n] -> [rows, n], zeros where there is no adapter (a select, not a product)."""
    own = t.gather(1, at.clamp(min=0)[:, None, None].expand(-1, 1, t.shape[2]))[:, 0]
    return torch.where(at[:, None] >= 0, own, 0.0)


class Case:
    def __init__(self, seed, rows, n, k, bits, block, adapters, rank, kind, xt, wt, whole, z, scaled=True, pad=0):
        g = gen(seed)
        self.z, self.at, self.bits, self.block = z, None, bits, block
        self.rows, self.n, self.k, self.adapters, self.rank = rows, n, k, adapters, rank

        def small(top, *shape):
            return torch.randint(-top, top + 1, shape, generator=g, device="cuda")

        def normal(*shape, std=1.0):
            return torch.randn(*shape, generator=g, device="cuda") * std

        self.codes, self.scales, self.w = weights(g, n, k, bits, block, lambda m: torch.pow(
            2.0, torch.randint(-1, 2, (m,), generator=g, device="cuda").float()) if whole else
            0.01 + 0.01 * torch.rand(m, generator=g, device="cuda"))
        if whole:
            x, dy, a, b = small(4, rows, k + pad), small(4, rows, n + pad), small(1, adapters, rank, k), \
                small(1, adapters, n, rank)
            s = torch.pow(2.0, torch.randint(-1, 2, (adapters,), generator=g, device="cuda").float())
        else:
            x, dy, a, b = normal(rows, k + pad), normal(rows, n + pad), normal(adapters, rank, k, std=k ** -0.5), \
                normal(adapters, n, rank, std=0.1)
            s = 0.5 + torch.rand(adapters, generator=g, device="cuda")
        self.x, self.dy = x.to(xt)[:, :k], dy.to(xt)[:, :n]
        self.a, self.b = a.to(wt), b.to(wt)
        self.s = s if scaled else None
        self.ids = make_ids(kind, rows, adapters, g)
        self.at = dense(z, self.ids, rows, adapters)

    def scale(self):
        s = torch.ones(self.adapters, device="cuda") if self.s is None else self.s
        return torch.where(self.at >= 0, s.double()[self.at.clamp(min=0)], 0.0)[:, None]

    def low(self, x, m):
        """s_g x m_g^T of each row, m [adapters, rank, len]: (value, magnitudes' sum)."""
        x = x.double()
        t = (x @ m.double().reshape(-1, x.shape[1]).t()).view(-1, self.adapters, self.rank)
        u = (x.abs() @ m.double().abs().reshape(-1, x.shape[1]).t()).view(-1, self.adapters, self.rank)
        return select(t, self.at, self.adapters) * self.scale(), select(u, self.at, self.adapters) * self.scale()

    def up(self, t, m):
        """Each row of t by its adapter's m [adapters, rank, len]."""
        out = torch.zeros(t.shape[0], m.shape[2], dtype=torch.float64, device="cuda")
        for g in range(self.adapters):
            r = (self.at == g).nonzero().flatten()
            out[r] = t[r].double() @ m[g].double()
        return out

    def sums(self, t, x):
        """For each adapter, over its rows, t^T x."""
        return torch.stack([t[self.at == g].double().t() @ x[self.at == g].double() for g in range(self.adapters)])

    def forward(self, dtype, **kw):
        return self.z.linear_adapters(self.x, self.codes, self.scales, self.bits, self.block, self.n, self.a, self.b,
                                      self.ids, self.s, dtype=dtype, **kw)

    def backward(self, reduced, dtype, **kw):
        return self.z.linear_adapters_grad(self.dy, self.x, reduced, self.codes, self.scales, self.bits, self.block,
                                           self.a, self.b, self.ids, self.s, dtype=dtype, **kw)

    def check_whole(self, dtype):
        y, t = self.forward(dtype)
        at, bt = self.a, self.b.transpose(1, 2)
        want, _ = self.low(self.x, at)
        assert torch.equal(t.double(), want)
        assert torch.equal(y, (self.x.double() @ self.w.t() + self.up(want, bt)).to(dtype))
        dx, da, db = self.backward(t, dtype)
        u, _ = self.low(self.dy, bt)
        assert torch.equal(dx, (self.dy.double() @ self.w + self.up(u, at)).to(dtype))
        assert torch.equal(da, self.sums(u, self.x).to(da.dtype))
        assert torch.equal(db, self.sums(want, self.dy).transpose(1, 2).to(db.dtype))

    def check_real(self, dtype):
        all_bf = self.x.dtype == dtype == self.a.dtype == BF
        # low enters the second product as two bf16 parts, the second rounded: off by 2^-9 of at most 2^-7
        cut = 2.0 ** -16 if all_bf else 0.0
        w_cut = 2.0 ** -8 if self.x.dtype == dtype == BF else 0.0   # weights as bf16
        half = torch.finfo(dtype).eps / 2
        at, bt = self.a, self.b.transpose(1, 2)

        def close(got, want, tol):
            off = (got.double() - want).abs()
            assert bool((off <= tol * (1 + 2.0 ** -7) + 1e-37).all()), (off / (tol + 1e-37)).max().item()

        def product(x, w, t, mags_t, off_t, m):
            """(value, bound) of x w + t m: each sum's additions and dropped small parts, 2^-24 of the magnitudes
            each; low's own error; the result's rounding."""
            c = w.shape[0]
            more = self.up(t, m)
            want = x.double() @ w + more
            mags = x.double().abs() @ w.abs()
            mags_m = self.up(t.abs(), m.abs())
            tol = mags * ((c + 16) * U + w_cut) + mags_m * ((self.rank + c // 64 + 16) * U + cut) + \
                self.up(off_t, m.abs()) + want.abs() * half + (mags + mags_m) * 4 * U
            return want, tol

        y, t = self.forward(dtype)
        want, mags = self.low(self.x, at)
        off = mags * (self.k + 16) * U
        close(t, want, off)
        close(y, *product(self.x, self.w.t(), want, mags, off, bt))
        dx, da, db = self.backward(t, dtype)
        u, mags_u = self.low(self.dy, bt)
        off_u = mags_u * (self.n + 16) * U
        close(dx, *product(self.dy, self.w, u, mags_u, off_u, at))
        cut = 2.0 ** -16 if self.x.dtype == self.a.dtype == BF else 0.0
        for got, low, off, x in ((da, u, off_u, self.x), (db, t.double(), torch.zeros_like(want), self.dy)):
            want_g = self.sums(low, x)
            tol = self.sums(low.abs(), x.abs()) * ((self.rows + 16) * U + cut) + self.sums(off, x.abs()) + \
                want_g.abs() * torch.finfo(got.dtype).eps / 2
            if got is db:
                want_g, tol = want_g.transpose(1, 2), tol.transpose(1, 2)
            close(got, want_g, tol)


# every kernel's rows, the kinds of ids, ranks on either side of 32 and 64
WHOLE = [
    (1, 64, 64, 32, 1, 8, "null"), (1, 100, 256, 128, 3, 64, "one"), (2, 257, 224, 32, 2, 16, "runs"),
    (3, 300, 1056, 32, 4, 72, "any"), (4, 64, 160, 32, 1, 128, "none"), (5, 129, 384, 128, 33, 24, "any"),
    (16, 64, 160, 32, 2, 8, "runs"), (17, 300, 1056, 32, 5, 64, "any"), (33, 259, 128, 64, 3, 40, "runs"),
    (64, 8, 1024, 1024, 40, 16, "any"), (65, 257, 224, 32, 2, 256, "runs"), (129, 129, 384, 128, 1, 64, "null"),
    (200, 96, 160, 32, 7, 8, "any"), (257, 300, 256, 256, 3, 88, "runs"), (300, 1000, 512, 64, 2, 64, "one"),
    (300, 520, 1056, 32, 100, 16, "any"), (700, 100, 256, 64, 1, 32, "null"), (64, 1, 32, 32, 2, 8, "any"),
    (1100, 515, 320, 64, 3, 64, "runs"), (130, 1000, 128, 64, 2, 16, "none"),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["to_bf16", "to_f32"])
@pytest.mark.parametrize("case", WHOLE, ids=["-".join(map(str, c)) for c in WHOLE])
def test_whole_numbers(z, case, dtype, bits):
    rows, n, k, block, adapters, rank, kind = case
    Case(rows, rows, n, k, bits, block, adapters, rank, kind, BF, BF, True, z).check_whole(dtype)


@pytest.mark.parametrize("types", [(BF, BF, BF), (BF, F32, BF), (BF, BF, F32), (BF, F32, F32), (F32, F32, F32),
                                   (F32, BF, F32), (F32, F32, BF)], ids=["bbb", "bfb", "bbf", "bff", "fff", "fbf", "ffb"])
@pytest.mark.parametrize("rows,kind", [(1, "null"), (3, "any"), (20, "runs"), (60, "any"), (100, "one"), (300, "runs"),
                                       (520, "null"), (300, "any")])
def test_real_numbers(z, rows, kind, types):
    xt, wt, dtype = types
    for n, k, rank, adapters in ((200, 416, 16, 3), (515, 1056, 72, 2)):
        Case(rows, rows, n, k, 4, 32, adapters, rank, kind, xt, wt, False, z).check_real(dtype)


@pytest.mark.parametrize("types", [(BF, BF, BF), (BF, F32, BF), (F32, F32, F32)], ids=["bbb", "bfb", "fff"])
@pytest.mark.parametrize("rows,n,k,kind", [(2100, 2560, 320, "runs"), (2100, 320, 2560, "one"), (70, 4160, 192, "any"),
                                           (70, 192, 4160, "runs"), (13, 8200, 96, "any"), (600, 1001, 1024, "null")])
def test_many_tiles_and_split_sums(z, rows, n, k, kind, types):
    xt, wt, dtype = types
    Case(9, rows, n, k, 4, 32, 3, 64, kind, xt, wt, False, z).check_real(dtype)


@pytest.mark.parametrize("rows,n,k,adapters,rank,kind", [(2100, 24640, 8224, 1, 256, "null"), (192, 4128, 4096, 4, 64, "any"),
                                                         (150, 4096, 4128, 4, 16, "runs"), (192, 1000, 512, 4, 64, "any"),
                                                         (1600, 2080, 2080, 32, 16, "any")])
def test_gradients_of_adapters_by_waves_and_by_workgroups(z, rows, n, k, adapters, rank, kind):
    """Sizes on either side of the estimate that shares the adapters' gradients out: many sums and many rows, few
    sums and few rows."""
    Case(rows, rows, n, k, 4, 32, adapters, rank, kind, BF, BF, True, z).check_whole(F32)


def test_without_scaling_and_in_more_dimensions(z):
    c = Case(2, 12, 96, 128, 4, 32, 3, 16, "any", BF, BF, True, z, scaled=False)
    c.check_whole(BF)
    y, t = c.forward(None)
    y3, t3 = z.linear_adapters(c.x.view(3, 4, 128), c.codes, c.scales, 4, 32, 96, c.a, c.b, c.ids.view(3, 4))
    assert y3.shape == (3, 4, 96) and t3.shape == (3, 4, 16)
    assert torch.equal(y3.view(12, 96), y) and torch.equal(t3.view(12, 16), t)
    dx, da, db = c.backward(t, None)
    dx3, da3, db3 = z.linear_adapters_grad(c.dy.view(3, 4, 96), c.x.view(3, 4, 128), t3, c.codes, c.scales, 4, 32, c.a,
                                           c.b, c.ids.view(3, 4))
    assert torch.equal(dx3.view(12, 128), dx) and torch.equal(da3, da) and torch.equal(db3, db)
    only, none, nothing = c.backward(None, None, want_adapters=False)
    assert torch.equal(only, dx) and none is None and nothing is None


@pytest.mark.parametrize("rows", [1, 4, 40, 100, 300])
def test_row_strides_leave_gaps_alone(z, rows):
    for xt in (BF, F32):
        c = Case(3, rows, 75, 128, 4, 32, 2, 24, "any", xt, xt, True, z, pad=8)
        y = torch.full((rows, 78), 77.0, dtype=xt, device="cuda")
        dx = torch.full((rows, 136), 77.0, dtype=xt, device="cuda")
        _, t = c.forward(None, out=y[:, :75])
        _, da, db = c.backward(t, None, out=dx[:, :128])
        assert bool((y[:, 75:] == 77).all()) and bool((dx[:, 128:] == 77).all())
        c.x, c.dy = c.x.contiguous(), c.dy.contiguous()
        y2, t2 = c.forward(None)
        dx2, da2, db2 = c.backward(t2, None)
        assert torch.equal(t, t2) and torch.equal(da, da2) and torch.equal(db, db2)
        # a dy whose rows stand on no 16-byte piece goes another way through the first product: whole numbers,
        # so the same
        assert torch.equal(y[:, :75], y2) and torch.equal(dx[:, :128], dx2)


@pytest.mark.parametrize("rows", [2, 4, 40, 100, 300, 600])
@pytest.mark.parametrize("wt", [BF, F32], ids=["bf16", "f32"])
def test_non_finite_adapters_and_rows_stay_their_own(z, rows, wt):
    c = Case(4, rows, 96, 160, 4, 32, 3, 16, "runs" if rows == 600 else "any", BF, wt, True, z)
    c.ids[0], c.ids[1] = 1, 2
    c.at = dense(z, c.ids, rows, 3)
    y, t = c.forward(None)
    dx, da, db = c.backward(t, None)
    # adapter 1 holds infinities and NaNs
    a, b = c.a.clone(), c.b.clone()
    a[1, 3, 5], a[1, 0, 0], b[1, 7, 2], b[1, 0, 0] = float("inf"), float("nan"), float("nan"), float("-inf")
    c.a, c.b, (a, b) = a, b, (c.a, c.b)
    y2, t2 = c.forward(None)
    dx2, da2, db2 = c.backward(t, None)
    ok = c.at != 1
    for got, want in ((y2, y), (t2, t), (dx2, dx)):
        assert torch.equal(got[ok], want[ok]) and not bool(torch.isfinite(got[~ok].float()).all())
    assert torch.equal(da2[[0, 2]], da[[0, 2]]) and torch.equal(db2[[0, 2]], db[[0, 2]])
    # a row of x and dy that is infinite or NaN
    c.a, c.b = a, b
    c.x[0, 5], c.dy[0, 7] = float("inf"), float("nan")
    y2, t2 = c.forward(None)
    dx2, da2, db2 = c.backward(t, None)
    for got, want in ((y2, y), (t2, t), (dx2, dx)):
        assert torch.equal(got[1:], want[1:]) and not bool(torch.isfinite(got[0].float()).all())
    assert torch.equal(da2[[0, 2]], da[[0, 2]]) and torch.equal(db2[[0, 2]], db[[0, 2]])


@pytest.mark.parametrize("rows", [2, 4, 40, 100, 300, 600])
@pytest.mark.parametrize("wt", [BF, F32], ids=["bf16", "f32"])
def test_what_is_not_finite_reaches_all_that_it_enters(z, rows, wt):
    """And nothing else: every element that the formulas make of an infinity or a NaN (a factor of zero makes a
    NaN), in the adapter's rows and gradients, and in a row of x or dy that holds one."""
    c = Case(17, rows, 96, 160, 4, 32, 3, 16, "runs" if rows == 600 else "any", BF, wt, True, z)
    c.ids[0], c.ids[1] = 1, 2
    c.at = dense(z, c.ids, rows, 3)
    _, t = c.forward(None)
    own = (c.at == 1)[:, None]

    def lost(got, want):
        assert torch.equal(~torch.isfinite(got.float()), want.expand(got.shape))

    a, b = c.a.clone(), c.b.clone()
    c.a[1, 3, 5], c.b[1, 7, 2] = float("inf"), float("nan")
    y2, t2 = c.forward(None)
    dx2, da2, db2 = c.backward(t, None)
    lost(y2, own)
    lost(t2, own & (torch.arange(16, device="cuda") == 3))
    lost(dx2, own)
    # u is lost at rank 2, so that rank of the adapter's gradient is; dB has finite factors alone
    lost(da2, (torch.arange(3, device="cuda") == 1)[:, None, None] & (torch.arange(16, device="cuda") == 2)[:, None])
    lost(db2, torch.zeros(1, dtype=torch.bool, device="cuda"))
    c.a, c.b = a, b
    first, of_its = (torch.arange(rows, device="cuda") == 0)[:, None], (torch.arange(3, device="cuda") == 1)[:, None, None]
    c.x[0, 5], c.dy[0, 7] = float("inf"), float("nan")
    y2, t2 = c.forward(None)
    dx2, da2, db2 = c.backward(t, None)
    for got in (y2, t2, dx2):
        lost(got, first)
    lost(da2, of_its)  # u of row 0 is
    lost(db2, of_its & (torch.arange(96, device="cuda") == 7)[:, None])


def test_no_rows_and_adapters_without_rows(z):
    c = Case(5, 40, 96, 128, 4, 32, 5, 16, "one", BF, BF, True, z)
    _, t = c.forward(None)
    _, da, db = c.backward(t, None, da=torch.full_like(c.a, 7), db=torch.full_like(c.b, 7))
    assert bool((da[:4] == 0).all()) and bool((db[:4] == 0).all()) and bool((da[4] != 0).any())
    c.x, c.dy, c.ids = c.x[:0], c.dy[:0], c.ids[:0]
    y, t = c.forward(None)
    dx, da, db = c.backward(t, None, da=torch.full_like(c.a, 7), db=torch.full_like(c.b, 7))
    assert y.shape == (0, 96) and t.shape == (0, 16) and dx.shape == (0, 128)
    assert bool((da == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("wt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 5, 16, 40, 64])
def test_few_rows_have_the_results_own_rounding_alone(z, rows, wt, bits):
    """From bf16 to bf16: up to 64 rows, weights enter with 16 bits or more, not as bf16, forward and back."""
    for n, k, adapters, rank, kind in ((200, 416, 3, 16, "any"), (2752, 1152, 2, 24, "runs"), (67, 1056, 1, 8, "null")):
        c = Case(19, rows, n, k, bits, 32, adapters, rank, kind, BF, wt, False, z)
        y, t = c.forward(None)
        dx, _, _ = c.backward(t, None)
        for got, x, w, m, m2 in ((y, c.x, c.w.t(), c.a, c.b.transpose(1, 2)), (dx, c.dy, c.w, c.b.transpose(1, 2), c.a)):
            low, mags_l = c.low(x, m)
            want = x.double() @ w + c.up(low, m2)
            # as in check_real, with a weight's second part off by half a step of 2^-8 of what the first leaves, 2^-8
            # in its binade: 2^-16, and low's likewise
            mags, mags_m = x.double().abs() @ w.abs(), c.up(low.abs(), m2.abs())
            tol = mags * ((w.shape[0] + 16) * U + 2.0 ** -16) + mags_m * ((rank + w.shape[0] // 64 + 16) * U + 2.0 ** -16) + \
                c.up(mags_l * (w.shape[0] + 16) * U, m2.abs()) + want.abs() * 2.0 ** -8
            off = (got.double() - want).abs()
            assert bool((off <= tol * (1 + 2.0 ** -7)).all()), (n, k, (off / tol).max().item())


def test_gradients_against_differences(z):
    """The gradients' products with directions, against differences of the forward formula in 64 bits: it is
    bilinear in A and B and linear in x, so central differences are exact there but for rounding."""
    c = Case(6, 30, 100, 128, 8, 32, 2, 8, "runs", F32, F32, False, z)
    _, t = c.forward(None)
    dx, da, db = c.backward(t, None)
    g = gen(7)
    ex, ea, eb = (torch.randn(v.shape, generator=g, device="cuda").double() for v in (c.x, c.a, c.b))

    def loss(x, a, b):
        low = select((x @ a.reshape(-1, 128).t()).view(-1, 2, 8), c.at, 2) * c.scale()
        y = x @ c.w.t()
        for i in range(2):
            r = (c.at == i).nonzero().flatten()
            y[r] += low[r] @ b[i].t()
        return (y * c.dy.double()).sum().item()

    x, a, b = c.x.double(), c.a.double(), c.b.double()
    for got, e, step in ((dx, ex, (1, 0, 0)), (da, ea, (0, 1, 0)), (db, eb, (0, 0, 1))):
        s = 2.0 ** -4
        up = loss(x + s * step[0] * ex, a + s * step[1] * ea, b + s * step[2] * eb)
        down = loss(x - s * step[0] * ex, a - s * step[1] * ea, b - s * step[2] * eb)
        mags = (got.double() * e).abs().sum().item()
        # binary32 sums of at most 128 + 8 + 30 terms; terms of a gradient exceed it 2^6-fold at most here
        assert abs((up - down) / (2 * s) - (got.double() * e).sum().item()) <= 166 * U * 64 * mags


def test_far_rows(z):
    stride, rows = (1 << 30) + 8, 5
    c = Case(8, rows, 96, 128, 4, 32, 2, 16, "any", BF, BF, True, z)

    def apart(t):
        return torch.empty(rows * stride, dtype=t.dtype, device="cuda").view(rows, stride)[:, :t.shape[1]].copy_(t)

    y, t = c.forward(None)
    dx, da, db = c.backward(t, None)
    c.x, c.dy = apart(c.x), apart(c.dy)
    y2, t2 = c.forward(None)
    dx2, da2, db2 = c.backward(t2, None)
    for a, b in ((y, y2), (t, t2), (dx, dx2), (da, da2), (db, db2)):
        assert torch.equal(a, b)


def test_adapters_past_32_bits(z):
    """The last adapter lies beyond 4 GB of them."""
    n, k, rank, adapters = 2048, 8192, 256, 1100
    g = gen(9)
    codes, scales, w = weights(g, n, k, 4, 128, lambda m: torch.ones(m, device="cuda"))
    a, b = torch.zeros(adapters, rank, k, dtype=BF, device="cuda"), torch.zeros(adapters, n, rank, dtype=BF, device="cuda")
    a[-1, 255], b[-1, :, 255] = 1, 2
    for rows in (2, 40, 300):
        x = torch.randint(-2, 3, (rows, k), generator=g, device="cuda").to(BF)
        ids = torch.full((rows,), adapters - 1, dtype=I32, device="cuda")
        ids[0] = 0
        y, t = z.linear_adapters(x, codes, scales, 4, 128, n, a, b, ids, dtype=F32)
        s = x.double().sum(1)
        s[0] = 0
        assert torch.equal(t[:, 255].double(), s) and int(torch.count_nonzero(t[:, :255])) == 0
        assert torch.equal(y.double(), x.double() @ w.t() + 2 * s[:, None])
        dy = torch.randint(-2, 3, (rows, n), generator=g, device="cuda").to(BF)
        dx, da, db = z.linear_adapters_grad(dy, x, t, codes, scales, 4, 128, a, b, ids, dtype=F32)
        u = 2 * dy.double().sum(1)
        u[0] = 0
        assert torch.equal(dx.double(), dy.double() @ w + u[:, None])
        assert torch.equal(da[-1, 255].double(), (u[:, None] * x.double()).sum(0).to(BF).double())
        assert torch.equal(db[-1, :, 255].double(), (s[:, None] * dy.double()).sum(0).to(BF).double())
        assert int(torch.count_nonzero(da[:-1])) == 0 and int(torch.count_nonzero(db[:-1])) == 0
        del da, db


def test_a_captured_pass_replays_with_new_adapters(z):
    c = Case(10, 300, 1000, 512, 4, 64, 4, 16, "runs", BF, BF, True, z)
    few = torch.zeros(3, 512, dtype=BF, device="cuda")
    few_ids = torch.zeros(3, dtype=I32, device="cuda")

    def step():
        y, t = c.forward(None)
        one = z.linear_adapters(few, c.codes, c.scales, 4, 64, 1000, c.a, c.b, few_ids, c.s)
        return y, t, *c.backward(t, None), *one

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    g = gen(11)
    for i in range(4):
        for t in (c.x, c.dy, few):
            t.copy_(torch.randint(-4, 5, t.shape, generator=g, device="cuda"))
        c.ids.copy_(make_ids(["any", "one", "none", "runs"][i], 300, 4, g))
        few_ids.copy_(torch.randint(-1, 4, (3,), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for a, b in zip(kept, step()):
            assert torch.equal(a, b)


def test_on_a_stream_that_is_behind(z):
    c = Case(12, 300, 1000, 512, 4, 64, 4, 16, "runs", F32, F32, True, z)
    want = c.forward(None)
    dwant = c.backward(want[1], None)
    side = torch.cuda.Stream()
    kept = c.x, c.dy, c.ids, c.a, c.b, c.s
    c.x, c.dy, c.ids, c.a, c.b, c.s = (t.clone() for t in kept)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = c.forward(None, stream=side)
    dgot = c.backward(got[1], None, stream=side)
    sizes = {t.numel() * t.element_size() for t in (*kept, *want, *dwant)}
    sizes |= {z.zpp_linear_adapters_workspace(d, 2, 1000 if d else 512, 2, 300, 1000, 512, 4, 16) for d in (0, 1)}
    c.x = c.dy = c.ids = c.a = c.b = c.s = None
    taken = [torch.full((s,), 255, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((*got, *dgot), (*want, *dwant)):
        assert torch.equal(a, b)
    assert taken
