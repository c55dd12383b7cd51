"""Wait states behind the tiled products' matrix instructions, in the compiled code.

The sums of the matrix instructions that are written out in the source must not
be read or written by anything but another of them for eight wait states, and
the compiler, which does not know what those instructions are, keeps no such
distance: neither for the code that uses the sums nor for copies of them that it
makes where control flow meets. The source puts explicit waits there. The device
code is compiled to assembly here (no GPU needed) and followed along every path;
between the last product of a sum and its first other use the explicit waits
alone must suffice, so that nothing rests on what happens to stand in between.
"""
from __future__ import annotations

import functools
import os
import re
import subprocess

import pytest

import __graft_entry__ as entry

BUILD = entry._build_module()
UNITS = [u for u in BUILD.LINEAR_UNITS if u.startswith("linear_big")]
STATES = 8   # after v_mfma_f32_16x16x32_bf16, what the compiler itself puts behind the builtin
BEFORE = 2   # from an ordinary vector instruction to a product that reads what it wrote


@functools.lru_cache(maxsize=None)
def registers(operand: str) -> tuple[str, ...]:
    """("a4", "a5") of "a[4:5]", ("v7",) of "v7" or "-v7", nothing of the rest."""
    operand = operand.strip("-|")
    m = re.fullmatch(r"([va])\[(\d+):(\d+)\]", operand)
    if m:
        return tuple(f"{m[1]}{i}" for i in range(int(m[2]), int(m[3]) + 1))
    return (operand,) if re.fullmatch(r"[va]\d+", operand) else ()


def kernels(asm: str) -> dict[str, list[str]]:
    """Instructions and block labels of each kernel."""
    out: dict[str, list[str]] = {}
    here = None
    for line in asm.splitlines():
        line = line.split(";")[0].strip()
        m = re.fullmatch(r"(_Z\w+):", line)
        if m:
            here = out.setdefault(m[1], [])
        elif line.startswith(".Lfunc_end"):
            here = None
        elif here is not None and line and (line.startswith(".LBB") or not line.startswith(".")):
            here.append(line)
    return out


def blocks(lines: list[str]):
    """Basic blocks, as (operation, operands) pairs, and the blocks that may follow each."""
    parts, names = [[]], {}
    for line in lines:
        if line.endswith(":"):
            names[line[:-1]] = len(parts)
            parts.append([])
            continue
        op, _, rest = line.partition(" ")
        parts[-1].append((op, [a.strip().split(" ")[0] for a in rest.split(",")]))
        if op.startswith(("s_cbranch", "s_branch", "s_endpgm")):
            parts.append([])
    after = []
    for i, b in enumerate(parts):
        op, args = b[-1] if b else ("", [])
        to = set()
        if op.startswith(("s_cbranch", "s_branch")):
            to.add(names[args[0]])
        if op not in ("s_branch", "s_endpgm") and i + 1 < len(parts):
            to.add(i + 1)
        after.append(to)
    return parts, after


def walk(block, sums: dict, written: dict, bad: list | None = None):
    """Through a block: `sums` holds the explicit wait states since a written-out product wrote a
    register (those into accumulation registers are the written-out ones), `written` all wait
    states since an ordinary instruction did."""
    sums, written = dict(sums), dict(written)
    for op, args in block:
        wait = int(args[0], 0) + 1 if op == "s_nop" else 0
        if op.startswith("v_mfma"):
            out, acc = registers(args[0]), registers(args[3])
            close = [r for a in args[1:4] for r in registers(a) if r in written]
            if acc != out:  # a product may follow at once on a sum that it continues
                close += [r for r in out + acc if r in sums]
            close += [r for a in args[1:3] for r in registers(a) if r in sums]
        else:
            close = [r for a in args for r in registers(a) if r in sums]
        if close and bad is not None:
            bad.append((op, *args))
        sums = {r: s + wait for r, s in sums.items() if s + wait < STATES}
        written = {r: s + max(wait, 1) for r, s in written.items() if s + max(wait, 1) < BEFORE}
        if op.startswith("v_mfma"):
            for r in out:
                written.pop(r, None)
                if r[0] == "a":
                    sums[r] = 0
        elif op.startswith("v_") and not op.startswith("v_cmp"):
            for r in registers(args[0]) + (registers(args[1]) if "_swap" in op else ()):
                written[r] = 0
    return sums, written


def too_close(lines: list[str]) -> list[tuple]:
    parts, after = blocks(lines)
    into = [None] * len(parts)
    into[0] = ({}, {})
    todo = {0}
    while todo:
        i = min(todo)
        todo.remove(i)
        left = walk(parts[i], *into[i])
        for j in after[i]:
            if into[j] is None:
                into[j] = tuple(dict(d) for d in left)
                todo.add(j)
                continue
            grew = False
            for have, come in zip(into[j], left):
                for r, s in come.items():
                    if have.get(r, STATES) > s:
                        have[r], grew = s, True
            if grew:
                todo.add(j)
    bad: list[tuple] = []
    for b, at in zip(parts, into):
        if at is not None:
            walk(b, *at, bad)
    return bad


MFMA = "v_mfma_f32_16x16x32_bf16 a[0:3], v[8:11], v[12:15], a[0:3]"


@pytest.mark.parametrize("lines,want", [
    ([MFMA, "v_accvgpr_read_b32 v1, a3"], 1),
    ([MFMA, "s_nop 7", "v_accvgpr_read_b32 v1, a3"], 0),
    ([MFMA, "s_nop 6", "v_accvgpr_read_b32 v1, a3"], 1),
    ([MFMA, *["s_mov_b32 s1, 0"] * 12, "v_accvgpr_read_b32 v1, a3"], 1),    # instructions that happen to stand there
    ([MFMA, "s_nop 0", "v_accvgpr_mov_b32 a2, a9"], 1),                     # an overwritten sum
    ([MFMA, "scratch_store_dwordx4 off, a[0:3], off"], 1),
    ([MFMA, MFMA, "v_accvgpr_read_b32 v1, a4"], 0),
    ([".LBB0_1:", "s_nop 7", "v_accvgpr_read_b32 v1, a0", MFMA, "s_cbranch_scc1 .LBB0_1", "s_nop 7",
      "v_accvgpr_read_b32 v1, a0"], 0),
    ([".LBB0_1:", "v_accvgpr_read_b32 v1, a0", MFMA, "s_cbranch_scc1 .LBB0_1", "s_nop 7"], 1),  # round the loop
    ([MFMA, "s_cbranch_scc1 .LBB0_1", "s_nop 7", ".LBB0_1:", "v_accvgpr_read_b32 v1, a0"], 1),  # past the wait
    (["v_accvgpr_write_b32 a0, 0", "s_mov_b32 s1, 0", MFMA], 1),
    (["v_accvgpr_write_b32 a0, 0", "s_nop 1", MFMA], 0),
    (["v_perm_b32 v9, v1, v2, s0", "s_branch .LBB0_1", ".LBB0_1:", MFMA], 1),
])
def test_the_check_sees_close_uses(lines, want):
    assert len(too_close([*lines, "s_endpgm"])) == want


@pytest.mark.parametrize("unit", UNITS)
def test_sums_are_left_alone_until_they_are_ready(unit):
    r = subprocess.run([BUILD.hipcc(), *BUILD.HIPCC_FLAGS, "-S", "--cuda-device-only", "-o", "-",
                        os.path.join(BUILD.CSRC, unit)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    pinned = 0
    for name, lines in kernels(r.stdout).items():
        pinned += any(line.startswith("v_mfma") and " a[" in line for line in lines)
        bad = too_close(lines)
        assert not bad, (name, len(bad), bad[:3])
    assert pinned >= 5
