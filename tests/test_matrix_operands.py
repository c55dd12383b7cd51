"""Wait states before the tiled products' matrix instructions, in the compiled code.

Some of those instructions are written out in the source, so the compiler does
not keep the distance that they need from an ordinary instruction that writes
one of their operands: two wait states. The device code is compiled to assembly
here (no GPU needed) and every matrix instruction is checked.
"""
from __future__ import annotations

import os
import re
import subprocess

import pytest

import __graft_entry__ as entry

BUILD = entry._build_module()
UNITS = [u for u in BUILD.LINEAR_UNITS if u.startswith("linear_big")]


def registers(operand: str) -> set[str]:
    """{"v4", "v5"} of "v[4:5]", {"v7"} of "v7", nothing of the rest."""
    m = re.fullmatch(r"([va])\[(\d+):(\d+)\]", operand)
    if m:
        return {f"{m[1]}{i}" for i in range(int(m[2]), int(m[3]) + 1)}
    return {operand} if re.fullmatch(r"[va]\d+", operand) else set()


def too_close(asm: str) -> tuple[int, list[str]]:
    """How many matrix instructions there are, and those that read what an ordinary vector
    instruction wrote less than two wait states before."""
    count, bad, recent = 0, [], []  # recent: (registers written, wait states) newest last
    for line in asm.splitlines():
        line = line.split(";")[0].strip()
        if not line or line.startswith(".") or line.endswith(":"):
            continue
        op, _, rest = line.partition(" ")
        args = [a.strip() for a in rest.split(",")]
        if op.startswith("v_mfma"):
            count += 1
            reads = registers(args[1]) | registers(args[2])
            states = 0
            for written, n in reversed(recent):
                if states >= 2:
                    break
                if written & reads:
                    bad.append(line)
                states += n
            recent.append((set(), 1))
        elif op == "s_nop":
            recent.append((set(), int(rest, 0) + 1))
        else:
            written = registers(args[0]) if op.startswith("v_") else set()
            if "_swap" in op:
                written |= registers(args[1])
            recent.append((written, 1))
        del recent[:-3]
    return count, bad


def test_the_check_sees_a_close_write():
    mfma = "v_mfma_f32_16x16x32_bf16 a[0:3], v[8:11], v[12:15], a[0:3]"
    assert too_close(f"v_perm_b32 v9, v1, v2, s0\ns_mov_b32 s1, 0\n{mfma}")[1] == [mfma]
    assert too_close(f"v_perm_b32 v9, v1, v2, s0\ns_nop 1\n{mfma}") == (1, [])
    assert too_close(f"v_perm_b32 v7, v1, v2, s0\n{mfma}") == (1, [])


@pytest.mark.parametrize("unit", UNITS)
def test_operands_are_two_wait_states_old(unit):
    r = subprocess.run([BUILD.hipcc(), *BUILD.HIPCC_FLAGS, "-S", "--cuda-device-only", "-o", "-",
                        os.path.join(BUILD.CSRC, unit)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    count, bad = too_close(r.stdout)
    assert count > 1000 and not bad, bad[:5]
