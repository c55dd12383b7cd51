"""Linear products with adapters or groups of rows whose sizes take several launches.

Rows past 2^20 (what the adapters make of x or dy), sums past 2^22 workgroups (the
adapters' gradients), groups and rows past 2^23 workgroups (grouped products): a wrong base
in a launch after the first would show in these alone. Small whole numbers, for which every
sum is exact. What no row uses is filled with other codes, or NaN.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402
from test_gpu_linear import gen, weights  # noqa: E402
from test_gpu_linear_adapters import Case  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def z():
    need_gpu()
    import block_quantization_codec_amd as z

    return z


def ones(m):
    return torch.ones(m, device="cuda")


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_adapters_over_rows_of_two_launches(z, t):
    Case(1, (1 << 20) + 70, 64, 64, 4, 32, 3, 8, "any", t, t, True, z).check_whole(F32)


def test_adapter_gradients_of_two_launches(z):
    adapters, n, k, rank, rows = 4096, 262400, 32, 8, 70
    g = gen(2)
    codes, scales, w = weights(g, n, k, 4, 4096, ones)
    used = [0, 5, 4087, 4088, 4095]  # 4088 adapters to a launch
    a = torch.full((adapters, rank, k), float("nan"), dtype=BF, device="cuda")
    b = torch.full((adapters, n, rank), float("nan"), dtype=BF, device="cuda")
    for e in used:
        a[e] = torch.randint(-1, 2, (rank, k), generator=g, device="cuda").to(BF)
        b[e] = torch.randint(-1, 2, (n, rank), generator=g, device="cuda").to(BF)
    ids = torch.tensor([(used + [-1])[m % 6] for m in range(rows)], dtype=I32, device="cuda")
    x = torch.randint(-4, 5, (rows, k), generator=g, device="cuda").to(BF)
    dy = torch.randint(-4, 5, (rows, n), generator=g, device="cuda").to(BF)
    y, t = z.linear_adapters(x, codes, scales, 4, 4096, n, a, b, ids, dtype=F32)
    dx, da, db = z.linear_adapters_grad(dy, x, t, codes, scales, 4, 4096, a, b, ids, dtype=F32)
    base, back = x.double() @ w.t(), dy.double() @ w
    for e in used:
        r = (ids == e).nonzero().flatten()
        low, u = x[r].double() @ a[e].double().t(), dy[r].double() @ b[e].double()
        assert torch.equal(t[r].double(), low)
        assert torch.equal(y[r].double(), base[r] + low @ b[e].double().t())
        assert torch.equal(dx[r].double(), back[r] + u @ a[e].double())
        assert torch.equal(da[e], (u.t() @ x[r].double()).to(BF)), e
        assert torch.equal(db[e], (dy[r].double().t() @ low).to(BF)), e
    none = (ids < 0).nonzero().flatten()
    assert torch.equal(y[none].double(), base[none]) and torch.equal(dx[none].double(), back[none])
    for e0 in range(0, adapters, 256):
        for e in used:
            if e0 <= e < e0 + 256:
                da[e], db[e] = 0, 0
        assert int(torch.count_nonzero(da[e0:e0 + 256])) == 0 and int(torch.count_nonzero(db[e0:e0 + 256])) == 0


def grouped_codes(g, groups, n, k, block, used):
    """(codes, scales, {group: W}): 0x77 where no row looks."""
    each = n * k // 2
    codes = torch.full((groups * each,), 0x77, dtype=torch.uint8, device="cuda")
    scales = torch.full((groups * (n * k // block),), 3.0, device="cuda")
    w = {}
    for e in used:
        c, s, m = weights(g, n, k, 4, block, ones)
        codes[e * each:(e + 1) * each] = c
        scales[e * s.numel():(e + 1) * s.numel()] = s
        w[e] = m.float()
    return codes, scales, w


def offsets_of(groups, counts):
    each = torch.zeros(groups, dtype=torch.int64)
    for e, c in counts.items():
        each[e] = c
    return torch.cat((torch.zeros(1, dtype=torch.int64), each.cumsum(0))).to(I32).cuda()


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_groups_of_two_launches(z, grad):
    groups, counts = 4096, {0: 3, 64: 1, 4090: 2, 4091: 5, 4094: 1, 4095: 4}  # 4091 groups to a launch
    n, k = (16, 262400) if grad else (131200, 32)
    g = gen(3)
    codes, scales, w = grouped_codes(g, groups, n, k, 4096, counts)
    rows = sum(counts.values())
    a = torch.randint(-4, 5, (rows, n if grad else k), generator=g, device="cuda").to(BF)
    f = z.linear_grouped_grad if grad else z.linear_grouped
    got = f(a, offsets_of(groups, counts), codes, scales, 4, 4096, k if grad else n, dtype=F32)
    at = 0
    for e, c in counts.items():
        assert torch.equal(got[at:at + c], a[at:at + c].float() @ (w[e] if grad else w[e].t())), e
        at += c


def test_groups_and_rows_of_two_launches(z):
    """2048 rows and 128 groups to a launch; the row where the second begins is inside of a group of the second."""
    groups, counts = 132, {0: 1, 60: 2030, 127: 9, 128: 31, 131: 29}
    n, k = 1 << 22, 32
    g = gen(4)
    codes, scales, w = grouped_codes(g, groups, n, k, 4096, counts)
    rows = sum(counts.values())
    x = torch.randint(-1, 2, (rows, k), generator=g, device="cuda").to(BF)  # results of up to 256: exact in bf16
    y = z.linear_grouped(x, offsets_of(groups, counts), codes, scales, 4, 4096, n)
    at = 0
    for e, c in counts.items():
        for r in range(at, at + c, 64):
            here = slice(r, min(r + 64, at + c))
            assert torch.equal(y[here], (x[here].float() @ w[e].t()).to(BF)), (e, r)
        at += c
