"""Wait states around the matrix instructions that are written out, in the tiled
products with adapters (see test_matrix_operands.py and test_matrix_results.py).

There the compiler has matrix instructions of its own too, into registers of either
kind, and keeps their distances itself. The assembly marks what comes from the source:
only that is held to the source's explicit waits.
"""
from __future__ import annotations

import os
import subprocess

import pytest

import test_matrix_operands as operands
import test_matrix_results as results

BUILD = results.BUILD
UNITS = [u for u in BUILD.LINEAR_UNITS if u.startswith("linear_adapt_")]


def only_written_out(asm: str) -> str:
    """The compiler's own matrix instructions renamed: ordinary instructions to the checks."""
    out, inside = [], False
    for line in asm.splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            inside = "#ASMSTART" in line
        out.append(line if inside else line.replace("v_mfma", "v_own_mfma"))
    return "\n".join(out)


def test_the_compilers_own_are_told_apart():
    asm = "\n".join(["_Zk:", ";;#ASMSTART", results.MFMA, ";;#ASMEND", results.MFMA.replace("a[", "a["), "s_endpgm"])
    lines = results.kernels(only_written_out(asm))["_Zk"]
    assert [line.split()[0] for line in lines] == ["v_mfma_f32_16x16x32_bf16", "v_own_mfma_f32_16x16x32_bf16", "s_endpgm"]
    assert len(results.too_close(lines)) == 1  # an ordinary use of the first's sums, at once


def test_there_are_units():
    assert len(UNITS) == 4


@pytest.mark.parametrize("unit", UNITS)
def test_waits_of_the_products_written_out(unit):
    r = subprocess.run([BUILD.hipcc(), *BUILD.HIPCC_FLAGS, "-S", "--cuda-device-only", "-o", "-",
                        os.path.join(BUILD.CSRC, unit)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    asm = only_written_out(r.stdout)
    count, bad = operands.too_close(asm)
    assert count > 1000 and not bad, bad[:5]
    pinned = 0
    for name, lines in results.kernels(asm).items():
        pinned += any(line.startswith("v_mfma") and " a[" in line for line in lines)
        bad = results.too_close(lines)
        assert not bad, (name, len(bad), bad[:3])
    assert pinned >= 5
