"""Linear products of rows in groups, and their input gradient, on the GPU.

As for one weight: small whole numbers and power-of-two scales, for which every
order of every sum is exact, so the result equals the 64-bit one, rounded once.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402
from test_gpu_linear import gen, weights  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def z():
    need_gpu()
    import block_quantization_codec_amd as z

    return z


def ascending(counts, first=0):
    return torch.tensor([first, *counts], dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def case(z, seed, grad, counts, n, k, bits, block, it, ot, first=0, tail=0, pad_in=0, pad_out=0, scale=None):
    """(result, the exact one, what lies around the rows in groups)."""
    g = gen(seed)
    e, rows = len(counts), first + sum(counts) + tail
    codes, scales, w = weights(g, e * n, k, bits, block, scale or (lambda m: torch.pow(
        2.0, torch.randint(-1, 2, (m,), generator=g, device="cuda").float())))
    w = w.view(e, n, k)
    al, ol = (n, k) if grad else (k, n)
    top = 300 if it == F32 else 4
    a = torch.randint(-top, top + 1, (rows, al + pad_in), generator=g, device="cuda").to(it)
    out = torch.full((rows, ol + pad_out), 77.0, dtype=ot, device="cuda")
    f = z.linear_grouped_grad if grad else z.linear_grouped
    f(a[:, :al], ascending(counts, first), codes, scales, bits, block, ol, out=out[:, :ol])
    want = torch.full((rows, ol), 77.0, dtype=ot, device="cuda")
    at = first
    for i, c in enumerate(counts):
        want[at:at + c] = (a[at:at + c, :al].double() @ (w[i] if grad else w[i].t())).to(ot)
        at += c
    return out[:, :ol], want, out[:, ol:]


COUNTS = [[1], [0, 1], [3, 0, 1, 0], [16, 17, 15], [0, 0, 64, 1, 65, 0], [5] * 70, [129, 2, 300, 0, 63], [1] * 130,
          [700], [257, 256, 255]]
SHAPES = [(1, 32, 32), (64, 160, 32), (100, 256, 256), (257, 224, 32), (300, 1056, 32), (8, 1024, 1024)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=["bb", "bf", "ff", "fb"])
@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_whole_numbers(z, grad, types, bits):
    for i, counts in enumerate(COUNTS):
        for n, k, block in SHAPES:
            got, want, _ = case(z, i, grad, counts, n, k, bits, block, *types, first=i % 3, tail=(i + 1) % 4)
            assert torch.equal(got, want), (counts, n, k, block, (got != want).sum().item())


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_many_tiles_and_split_sums(z, grad):
    for types in ((BF, BF), (BF, F32), (F32, F32)):
        for counts, n, k, block in [([1100, 0, 900, 333], 2560, 320, 64), ([600, 1200], 320, 2560, 256),
                                    ([70, 3], 4160, 192, 64), ([9, 61], 192, 4160, 64), ([13, 1], 8200, 96, 32),
                                    ([300, 301, 299], 1001, 1024, 128)]:
            got, want, _ = case(z, 9, grad, counts, n, k, 4, block, *types, first=2, tail=3)
            assert torch.equal(got, want), (counts, n, k, block)


@pytest.mark.parametrize("counts", [[300, 0, 70, 129], [1, 2, 3], [900, 257], [65] * 9, [2000], [1290, 800, 1]],
                         ids=lambda c: "-".join(map(str, c[:4])))
@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_whole_rounds_of_tiles_and_what_is_left(z, grad, counts):
    """Tiles past whole rounds of the GPU take the contraction in parts, whose number follows from the offsets."""
    for long, (across, block) in [(1024, (16384, 128)), (1087 if grad else 1088, (7904 if grad else 7903, 32))]:
        n, k = (long, across) if grad else (across, long)
        for types in ((BF, BF), (F32, F32), (BF, F32)) if grad else ((BF, BF), (F32, F32)):
            if types[0] == F32 and sum(counts) > 1500:
                continue
            got, want, gap = case(z, 4, grad, counts, n, k, 8, block, *types, first=1, tail=2, pad_out=8)
            assert torch.equal(got, want) and bool((gap == 77).all()), (long, across, types)


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_row_strides_leave_gaps_alone(z, grad):
    for it, ot in [(BF, BF), (F32, F32)]:
        for pad_in, pad_out in ([(1, 8), (5, 16), (8, 8)] if grad else [(8, 1), (16, 3), (8, 8)]):
            for counts in ([1, 2], [20, 0, 33], [200, 70]):
                for n in (72, 75):
                    got, want, gap = case(z, 3, grad, counts, n, 128, 4, 32, it, ot, 1, 2, pad_in, pad_out)
                    assert torch.equal(got, want) and bool((gap == 77).all()), (it, pad_in, pad_out, n)


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_one_group_gives_what_one_weight_gives_within_its_roundings(z, grad):
    """Real-valued: the same bounds as the single product's, against 64 bits."""
    g = gen(1)
    n, k, block = 1000, 1056, 32
    for counts in ([3, 40], [70, 500]):
        for it, ot in ((BF, BF), (BF, F32), (F32, F32)):
            w = torch.randn(2 * n, k, generator=g, device="cuda") * 0.02
            codes, scales = z.quantize(w, block, 4)
            w = z.dequantize(codes, scales, 4, 2 * n * k, block, dtype=F32).double().view(2, n, k)
            a = torch.randn(sum(counts), n if grad else k, generator=g, device="cuda").to(it)
            f = z.linear_grouped_grad if grad else z.linear_grouped
            got = f(a, ascending(counts), codes, scales, 4, block, k if grad else n, dtype=ot).double()
            at = 0
            for i, c in enumerate(counts):
                m = w[i] if grad else w[i].t()
                x = a[at:at + c].double()
                want, mags = x @ m, x.abs() @ m.abs()
                # binary32 sums of at most 1056 + 2 products and parts, each addition off by at most 2^-24 of the
                # magnitudes; the product (code times scale) 2^-24; from bf16 to bf16 the weights 2^-8; the result
                # half a step of its type
                tol = mags * (1060 * 2.0 ** -24 + (2.0 ** -8 if it == ot == BF else 0)) + \
                    want.abs() * torch.finfo(ot).eps / 2
                assert bool(((got[at:at + c] - want).abs() <= tol * (1 + 2.0 ** -7)).all())
                at += c


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_few_rows_have_the_results_own_rounding_alone(z, grad, bits):
    """From bf16 to bf16: weights enter with 16 bits or more, not as bf16, up to 64 rows a group, back up to 64 rows
    a call."""
    g = gen(18)
    for counts in ([1], [0, 1, 2], [5, 0, 3, 9], [16] * 4, [64]) if grad else ([1], [5, 0, 3, 9], [60, 100, 2, 30], [64] * 3):
        for n, k, block in ((632, 448, 128), (1000, 224, 32), (4992, 96, 32), (67, 1056, 32)):
            w = torch.randn(len(counts) * n, k, generator=g, device="cuda") * 0.02
            codes, scales = z.quantize(w, block, bits)
            w = z.dequantize(codes, scales, bits, len(counts) * n * k, block, dtype=F32).double().view(-1, n, k)
            a = torch.randn(sum(counts), n if grad else k, generator=g, device="cuda").to(BF)
            f = z.linear_grouped_grad if grad else z.linear_grouped
            got = f(a, ascending(counts), codes, scales, bits, block, k if grad else n).double()
            at = 0
            for i, c in enumerate(counts):
                m = w[i] if grad else w[i].t()
                x = a[at:at + c].double()
                want, mags = x @ m, x.abs() @ m.abs()
                # each of the binary32 sums' additions 2^-24 of the magnitudes, and as much for code times scale; a
                # weight's second part half a step of 2^-8 of what the first leaves, 2^-8 in its binade: 2^-16; the
                # result half a step of bf16
                tol = mags * ((m.shape[0] + 8) * 2.0 ** -24 + 2.0 ** -16) + want.abs() * 2.0 ** -8
                off = (got[at:at + c] - want).abs()
                assert bool((off <= tol * (1 + 2.0 ** -7)).all()), (counts, n, k, (off / tol).max().item())
                at += c


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_non_finite_rows_stay_their_own(z, grad):
    g = gen(2)
    codes, scales, w = weights(g, 3 * 96, 160, 4, 32, lambda m: torch.ones(m, device="cuda"))
    w = w.view(3, 96, 160)
    f = z.linear_grouped_grad if grad else z.linear_grouped
    for counts in ([2, 3, 1], [30, 70, 100], [300, 10, 90]):
        rows, o = sum(counts), ascending(counts)
        a = torch.randint(-4, 5, (rows, 96 if grad else 160), generator=g, device="cuda").to(BF)
        want = f(a, o, codes, scales, 4, 32, 160 if grad else 96)
        bad = a.clone()
        bad[1, 3], bad[rows - 1, 7] = float("inf"), float("nan")
        got = f(bad, o, codes, scales, 4, 32, 160 if grad else 96)
        ok = [r for r in range(rows) if r not in (1, rows - 1)]
        assert torch.equal(got[ok], want[ok])
        assert not bool(torch.isfinite(got[1].float()).any() and torch.isfinite(got[rows - 1].float()).any())
    # a group's weights, infinite or NaN, reach no other group's rows
    scales = scales.clone()
    scales[:96 * 160 // 32] = float("nan")
    for counts in ([2, 3, 1], [30, 70, 100], [300, 10, 90]):
        rows, o = sum(counts), ascending(counts)
        a = torch.randint(-4, 5, (rows, 96 if grad else 160), generator=g, device="cuda").to(BF)
        got = f(a, o, codes, scales, 4, 32, 160 if grad else 96)
        m = w[1] if grad else w[1].t()
        assert torch.equal(got[counts[0]:counts[0] + counts[1]],
                           (a[counts[0]:counts[0] + counts[1]].double() @ m).to(BF))


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_offsets_that_do_not_ascend_stay_in_bounds(z, grad):
    """Results are unspecified; what lies around the rows is not."""
    g = gen(4)
    n, k = 96, 128
    codes, scales, _ = weights(g, 4 * n, k, 4, 32, lambda m: torch.ones(m, device="cuda"))
    f = z.linear_grouped_grad if grad else z.linear_grouped
    for rows in (5, 100, 600):
        a = torch.randint(-4, 5, (rows, n if grad else k), generator=g, device="cuda").to(BF)
        big = torch.full((rows + 64, k if grad else n), 77.0, dtype=BF, device="cuda")
        for o in ([0, rows, 0, rows, rows], [-5, 3, 1 << 30, -(1 << 31), (1 << 31) - 1], [rows, 0, 0, 0, 0],
                  [rows + 9, rows + 90, rows + 900, rows + 901, rows + 902]):
            f(a, torch.tensor(o, dtype=torch.int32).cuda(), codes, scales, 4, 32, k if grad else n, out=big[32:-32])
            torch.cuda.synchronize()
            assert bool((big[:32] == 77).all()) and bool((big[-32:] == 77).all())
        f(a, torch.tensor([0, 1, 2, 3, rows], dtype=torch.int32).cuda(), codes, scales, 4, 32, k if grad else n,
          out=big[32:-32])
        assert not bool((big[32:-32] == 77).all())


@pytest.mark.parametrize("types", [(BF, BF), (BF, F32), (F32, F32)], ids=["bb", "bf", "ff"])
@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_no_element_of_a_non_finite_row_is_finite(z, grad, types):
    """Each of the rows by itself, and every element: a code of zero makes a NaN of an infinity."""
    g = gen(15)
    n, k = 96, 160
    codes, scales, _ = weights(g, 3 * n, k, 4, 32, lambda m: torch.ones(m, device="cuda"))
    f = z.linear_grouped_grad if grad else z.linear_grouped
    for counts in ([2, 3, 1], [30, 70, 100], [300, 10, 90]):
        rows, o = sum(counts), ascending(counts)
        a = torch.randint(-4, 5, (rows, n if grad else k), generator=g, device="cuda").to(types[0])
        for row, value in ((1, float("inf")), (counts[0], float("-inf")), (rows - 1, float("nan"))):
            bad = a.clone()
            bad[row, 7] = value
            got = f(bad, o, codes, scales, 4, 32, k if grad else n, dtype=types[1])
            finite = torch.isfinite(got.float())
            assert not bool(finite[row].any()), (counts, row)
            assert bool(finite[:row].all()) and bool(finite[row + 1:].all()), (counts, row)


@pytest.mark.parametrize("grad", [False, True], ids=["y", "dx"])
def test_results_after_offsets_that_do_not_ascend(z, grad):
    """A call with such offsets leaves nothing behind: the next one's results are its own, in a buffer filled anew."""
    g = gen(16)
    n, k = 96, 128
    codes, scales, w = weights(g, 4 * n, k, 4, 32, lambda m: torch.ones(m, device="cuda"))
    w = w.view(4, n, k)
    f = z.linear_grouped_grad if grad else z.linear_grouped
    need = max(z.zpp_linear_grouped_workspace(int(grad), z.ZPP_BF16, n if grad else k, z.ZPP_BF16, r, 4, n, k)
               for r in (5, 100, 600))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    for rows in (5, 100, 600):
        a = torch.randint(-4, 5, (rows, n if grad else k), generator=g, device="cuda").to(BF)
        big = torch.empty(rows + 64, k if grad else n, dtype=BF, device="cuda")
        for bad in ([0, rows, 0, rows, rows], [-5, 3, 1 << 30, -(1 << 31), (1 << 31) - 1], [rows, 0, 0, 0, 0]):
            big.fill_(77)
            f(a, torch.tensor(bad, dtype=torch.int32).cuda(), codes, scales, 4, 32, k if grad else n, out=big[32:-32],
              workspace=ws)
            big.fill_(77)
            o = [0, 1, 2, 3, rows - 1]
            f(a, torch.tensor(o, dtype=torch.int32).cuda(), codes, scales, 4, 32, k if grad else n, out=big[32:-32],
              workspace=ws)
            want = torch.full_like(big, 77)
            for i in range(4):
                m = w[i] if grad else w[i].t()
                want[32 + o[i]:32 + o[i + 1]] = (a[o[i]:o[i + 1]].double() @ m).to(BF)
            assert torch.equal(big, want), (rows, bad)


def test_many_groups(z):
    """4096 weights: the offsets are read in many runs of 64."""
    g = gen(5)
    e, n, k = 4096, 8, 32
    counts = torch.randint(0, 3, (e,), generator=torch.Generator().manual_seed(1)).tolist()
    for grad in (False, True):
        got, want, _ = case(z, 6, grad, counts, n, k, 4, 32, BF, F32, 1, 1)
        assert torch.equal(got, want)
    assert e == len(counts) and g is not None


def test_codes_past_32_bits(z):
    """The last of many weights lies beyond 4 GB of codes."""
    e, n, k, block = 70, 8192, 8192, 4096
    codes = torch.zeros(e * n * k, dtype=torch.uint8, device="cuda")
    scales = torch.ones(e * n * k // block, device="cuda")
    codes.view(e, n, k)[e - 1, :, ::2] = 3
    for rows in (3, 200):
        o = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
        o[e] = rows
        y = z.linear_grouped(torch.ones(rows, k, dtype=BF, device="cuda"), o, codes, scales, 8, block, n)
        assert bool((y == 3 * (k // 2)).all())
        dx = z.linear_grouped_grad(torch.ones(rows, n, dtype=BF, device="cuda"), o, codes, scales, 8, block, k)
        assert bool((dx[:, ::2] == 3 * n).all()) and bool((dx[:, 1::2] == 0).all())


def test_a_captured_pass_replays_with_new_groups(z):
    """Offsets are read on the device: a graph takes those of its replay."""
    g = gen(7)
    e, n, k, rows = 6, 1000, 512, 300
    codes, scales, w = weights(g, e * n, k, 4, 64, lambda m: torch.ones(m, device="cuda"))
    w = w.view(e, n, k)
    x, dy = torch.zeros(rows, k, dtype=BF, device="cuda"), torch.zeros(rows, n, dtype=BF, device="cuda")
    o = ascending([50] * e)

    def step():
        return (z.linear_grouped(x, o, codes, scales, 4, 64, n), z.linear_grouped(x[:40], o, codes, scales, 4, 64, n),
                z.linear_grouped_grad(dy, o, codes, scales, 4, 64, k))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, few, dx = step()
    for counts in ([50] * e, [300, 0, 0, 0, 0, 0], [0, 1, 99, 100, 0, 100], [60, 40, 50, 50, 70, 30]):
        x.copy_(torch.randint(-4, 5, x.shape, generator=g, device="cuda"))
        dy.copy_(torch.randint(-4, 5, dy.shape, generator=g, device="cuda"))
        o.copy_(ascending(counts))
        for t in (y, few, dx):
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for i, c in enumerate(counts):
            here = slice(at, at + c)
            assert torch.equal(y[here], (x[here].double() @ w[i].t()).to(BF))
            assert torch.equal(dx[here], (dy[here].double() @ w[i]).to(BF))
            here = slice(at, min(at + c, 40))
            assert torch.equal(few[here], (x[here].double() @ w[i].t()).to(BF))
            at = min(at + c, rows)


def test_a_replay_takes_the_parts_that_its_groups_leave(z):
    """One captured pass, whose groups leave from no tile to nearly a round of them for parts; bad offsets too."""
    g = gen(14)
    e, n, k, rows = 4, 1024, 16384, 900
    codes, scales, w = weights(g, e * n, k, 4, 128, lambda m: torch.ones(m, device="cuda"))
    w = w.view(e, n, k)
    dy, o = torch.zeros(rows, n, dtype=BF, device="cuda"), ascending([225] * e)
    dx = torch.empty(rows, k, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        z.linear_grouped_grad(dy, o, codes, scales, 4, 128, k, out=dx)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.linear_grouped_grad(dy, o, codes, scales, 4, 128, k, out=dx)
    for counts in ([225] * e, [900, 0, 0, 0], [0, 0, 0, 1], [256, 256, 256, 132], [1, 0, 300, 2], [0] * e, [64] * e):
        dy.copy_(torch.randint(-4, 5, dy.shape, generator=g, device="cuda"))
        o.copy_(ascending(counts))
        dx.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        at = 0
        for i, c in enumerate(counts):
            assert torch.equal(dx[at:at + c], (dy[at:at + c].double() @ w[i]).to(BF)), (counts, i)
            at += c
        assert bool((dx[at:] == 9).all()), counts
    o.copy_(torch.tensor([700, -5, 2_000_000_000, 30, 890], dtype=torch.int32))
    graph.replay()  # rows of no group or of two hold what they hold; nothing outside is touched
    torch.cuda.synchronize()
    o.copy_(ascending([225] * e))
    graph.replay()
    torch.cuda.synchronize()
    for i in range(e):
        here = slice(225 * i, 225 * i + 225)
        assert torch.equal(dx[here], (dy[here].double() @ w[i]).to(BF))


def test_on_a_stream_that_is_behind(z):
    g = gen(8)
    n, k = 4160, 256
    codes, scales, _ = weights(g, 3 * n, k, 4, 64, lambda m: torch.ones(m, device="cuda"))
    x = torch.randint(-4, 5, (300, k), generator=g, device="cuda").to(F32)
    dy = torch.randint(-4, 5, (70, n), generator=g, device="cuda").to(BF)
    ox, od = ascending([100, 150, 50]), ascending([30, 0, 40])
    want = z.linear_grouped(x, ox, codes, scales, 4, 64, n), z.linear_grouped_grad(dy, od, codes, scales, 4, 64, k)
    side = torch.cuda.Stream()
    mine = [t.clone() for t in (x, ox, dy, od)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = (z.linear_grouped(mine[0], mine[1], codes, scales, 4, 64, n, stream=side),
           z.linear_grouped_grad(mine[2], mine[3], codes, scales, 4, 64, k, stream=side))
    sizes = {t.numel() * t.element_size() for t in (*mine, *want)} | {1 << 16, 1 << 20, 1 << 22}
    del mine
    taken = [torch.full((s,), 255, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert taken
