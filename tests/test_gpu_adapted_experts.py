"""The norm, the projection with adapters and the experts in a run, forward and back: the
example's errors are those of the types' roundings."""
from __future__ import annotations

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapted_experts.py")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,experts", [(40, 4), (333, 5)])
def test_adapted_experts(rows, experts, bits, dtype):
    need_gpu()
    spec = importlib.util.spec_from_file_location("adapted_experts", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    # A step's result has its own rounding, half an eps of values of its size, and that of the weights it
    # multiplies by (bf16: another half); each of the at most five steps before it leaves as much in what it
    # starts from, and a product or a norm carries a relative error of its input's norm on as one of its
    # result's (for the random values here; the norm's gradient subtracts a projection, which cannot
    # lengthen it): six steps of one eps. Binary32 sums of up to 544 terms add at most 544 * 2^-24 of their
    # terms' norm, and by sqrt(544) of it in practice, in each of the six: 6 * 24 * 2^-24 = 72 eps, which
    # leads there.
    eps = torch.finfo(dtype).eps
    bound = 6 * eps if dtype == torch.bfloat16 else (6 + 72) * eps
    errors = mod.run(rows=rows, width=288, out=544, experts=experts, bits=bits, block=32, dtype=dtype)
    # codes of 8 bits: half a step of 1/127 of a block's largest value at most, which is at most sqrt(32)
    # times the block's root mean square
    sent = errors.pop("sent")
    assert sent <= 0.5 / 127 * 32 ** 0.5 + bound
    for name, err in errors.items():
        assert err <= bound, (name, err)
