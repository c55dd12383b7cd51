"""The example runs, and its errors are those of the types' roundings."""
from __future__ import annotations

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
from gpu_util import need_gpu  # noqa: E402

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "quantized_layer.py")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_quantized_layer(bits, dtype):
    need_gpu()
    spec = importlib.util.spec_from_file_location("quantized_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    # Every result goes through at most four roundings to the type (activations, weights, the
    # result before, the result), each relative to values of its own size and at most eps / 2, which
    # the norms of whole results add up to at most: 2 eps. Binary32 sums of up to 512 terms in any
    # order add at most 512 * 2^-24 of the terms' norm, and by sqrt(512) of it in practice: 64 eps.
    bound = 2 * torch.finfo(dtype).eps if dtype == torch.bfloat16 else 64 * torch.finfo(dtype).eps
    for name, err in mod.run(rows=130, width=288, out=512, bits=bits, block=32, dtype=dtype).items():
        assert err <= bound, (name, err)
