"""What the short helpers allocate belongs to the stream that they are told to use.

Memory from torch's current stream's pool would be handed out again, for work on
that stream, while the other one still reads or writes it. Seen here on the CPU:
allocations are recorded, the entry points and the streams replaced.
"""
from __future__ import annotations

import contextlib

import pytest

torch = pytest.importorskip("torch")
from torch.utils._python_dispatch import TorchDispatchMode  # noqa: E402

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
HANDLE = 77

# 64 x 32 weights of 4 bits in blocks of 32
CODES, SCALES = torch.zeros(64 * 16, dtype=U8), torch.ones(64)
X, DY, W = torch.zeros(40, 32, dtype=BF), torch.zeros(40, 64, dtype=BF), torch.ones(32)
STATS = torch.ones(40)
CALLS = {  # helper, arguments, and how many tensors it allocates
    "quantize": ((X, 32, 4), 2),
    "quantize_reordered": ((X, 2, 2, 32, 4), 2),
    "dequantize": ((CODES, SCALES, 4, 2048, 32), 1),
    "reorder": ((X, 2, 2), 1),
    "dequant_reduce_requant": ((CODES, SCALES, 2, 4, 1024, 32, 4), 3),
    "dequant_reduce_requant_split": ((CODES, SCALES, 2, 4, 1024, 32, 0, 512, 4), 4),
    "dequant_reduce_average": ((CODES, SCALES, 2, 4, 1024, 32, 2), 1),
    "linear": ((X, CODES, SCALES, 4, 32, 64), 1),
    "linear_grad": ((DY.float(), CODES, SCALES, 4, 32, 32), 2),
    "layer_norm": ((X, W, W), 3),
    "layer_norm_grad": ((X, X, W, STATS, STATS), 4),
}


class Allocations(TorchDispatchMode):
    """The stream that is current at each allocation."""

    def __init__(self, current):
        super().__init__()
        self.current, self.seen = current, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if "empty" in str(func):
            self.seen.append(self.current[-1])
        return func(*args, **(kwargs or {}))


class FakeStream:
    cuda_stream = HANDLE
    device = None


@pytest.fixture
def fake(monkeypatch):
    """(the package, the stack of current streams, the streams that entry points were called with)"""
    import block_quantization_codec_amd as z

    current, launched = [0], []

    @contextlib.contextmanager
    def under(stream):
        current.append(stream)
        yield
        current.pop()

    def stream_of(stream):
        return current[-1] if stream is None else stream if isinstance(stream, int) else stream.cuda_stream

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: type("S", (int,), {"device": None})(handle))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(z, "_stream", stream_of)
    monkeypatch.setattr(z, "_call", lambda name, *args: launched.append(args[-1]))
    return z, current, launched


@pytest.mark.parametrize("stream", [HANDLE, FakeStream()], ids=["handle", "object"])
@pytest.mark.parametrize("name", CALLS)
def test_allocations_belong_to_the_stream_in_use(fake, name, stream):
    z, current, launched = fake
    args, count = CALLS[name]
    with Allocations(current) as mode:
        getattr(z, name)(*args, stream=stream)
    assert launched == [HANDLE]
    assert mode.seen == [HANDLE] * count
    assert current == [0]


@pytest.mark.parametrize("name", CALLS)
def test_without_a_stream_the_current_one_is_used(fake, name):
    z, current, launched = fake
    args, count = CALLS[name]
    with Allocations(current) as mode:
        getattr(z, name)(*args)
    assert launched == [0] and mode.seen == [0] * count


def test_results_are_the_same_as_without_a_stream(fake, monkeypatch):
    """Every argument reaches the entry point, in its place."""
    z, _, _ = fake
    calls = []
    monkeypatch.setattr(z, "_call", lambda name, *args: calls.append((name, [
        a for a in args[:-1] if a is None or abs(a) < 1 << 32])))
    out, ws = torch.empty(40, 64), torch.empty(1 << 20, dtype=U8)
    for name, args, kw in [
        ("quantize_reordered", (X, 2, 2, 32, 4), dict(first_slice=1, n_slices=2)),
        ("dequantize", (CODES, SCALES, 4, 2048, 32), dict(dtype=F32)),
        ("dequant_reduce_requant", (CODES, SCALES, 2, 4, 512, 32),
         dict(bits_out=8, want_sum=False, codes_stride_bytes=512, scales_stride=32)),
        ("dequant_reduce_requant_split", (CODES, SCALES, 2, 4, 512, 32, 0, 512, 4),
         dict(codes_stride_bytes=512, scales_stride=32)),
        ("dequant_reduce_average", (CODES, SCALES, 2, 4, 512, 32, 3), dict(codes_stride_bytes=512, scales_stride=32)),
        ("linear", (X, CODES, SCALES, 4, 32, 64), dict(dtype=F32, out=out, workspace=ws)),
        ("linear_grad", (DY, CODES, SCALES, 4, 32, 32), dict(dtype=F32, workspace=ws)),
        ("layer_norm", (X, W, W), dict(eps=0.25, out=X.clone())),
        ("layer_norm_grad", (X, X, None, STATS, STATS), dict(workspace=ws, w_dtype=F32)),
    ]:
        got = getattr(z, name)(*args, **kw)
        again = getattr(z, name)(*args, **kw, stream=HANDLE)
        assert calls[-1] == calls[-2]
        for a, b in zip(*(o if isinstance(o, tuple) else (o,) for o in (got, again))):
            assert (a is None) == (b is None) and (a is None or (a.shape, a.dtype) == (b.shape, b.dtype))
