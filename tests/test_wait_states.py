"""Wait states behind matrix instructions, on every path of every kernel in the built library.

The result of a matrix instruction may be used by another instruction (as anything but the accumulator
of the next matrix instruction) only after a number of wait states that depends on the form: the
hardware does not wait by itself.  The compiler has been seen to count them along one of two paths
around a block that may be jumped over.  The kernels put such waits themselves (settle() in
csrc/ss_device.h); this walks the listing of what was built.  No GPU needed.
"""
import os
import re
import shutil
import subprocess

import pytest

import selective_state_space_34_amd as ss
from selective_state_space_34_amd import _build

OBJDUMP = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.HIPCC))),
                       "llvm", "bin", "llvm-objdump")
# states that the compiler keeps in straight-line code on gfx950, by form
NEED = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10, "v_mfma_f32_32x32x16_bf16": 12}


def registers(operand):
    m = re.match(r"^[-|]*([va])\[(\d+):(\d+)\]", operand)
    if m:
        return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.match(r"^[-|]*([va])(\d+)\b", operand)
    return {(m.group(1), int(m.group(2)))} if m else set()


def functions(text):
    """name -> list of (opcode, operands, index a branch goes to or None)."""
    out = {}
    for block in re.split(r"\n(?=[0-9a-f]{16} <)", text):
        head = re.match(r"^([0-9a-f]{16}) <([^>]+)>:", block)
        if not head:
            continue
        start, code, where = int(head.group(1), 16), [], {}
        for line in block.split("\n")[1:]:
            m = re.match(r"^\s+([a-z]\w*)\s*(.*?)\s*// ([0-9A-F]+):[^<]*(?:<[^>+]*(?:\+0x([0-9a-f]+))?>)?", line)
            if not m:
                continue
            where[int(m.group(3), 16)] = len(code)
            to = start + int(m.group(4) or "0", 16) if "branch" in m.group(1) else None
            code.append((m.group(1), [t.strip() for t in m.group(2).split(",")], to))
        out[head.group(2)] = [(o, a, None if t is None else where[t]) for o, a, t in code]
    return out


def shortest(code, i):
    """Fewest states on any path from matrix instruction i to a use of its result; None if all
    paths are longer than is ever needed."""
    result = registers(code[i][1][0])
    best, seen, paths = None, {}, [(i + 1, 0)]
    while paths:
        j, n = paths.pop()
        if j >= len(code) or n >= max(NEED.values()) or seen.get(j, 99) <= n:
            continue
        seen[j] = n
        op, args, to = code[j]
        if op == "s_endpgm":
            continue
        if op.startswith("v_mfma"):
            used = any(registers(a) & result for a in args[1:3])
            ends = bool(registers(args[0]) & result)     # that one's result is looked at for itself
        else:
            used = ends = any(registers(a) & result for a in args)
        if used and (best is None or n < best):
            best = n
        if ends or used:
            continue
        step = 1 + (int(args[0], 0) if op == "s_nop" else 0)
        if to is not None:
            paths.append((to, n + step))
        if op != "s_branch":
            paths.append((j + 1, n + step))
    return best


def short_ones(text):
    found, count = [], 0
    for name, code in functions(text).items():
        for i, (op, _, _) in enumerate(code):
            if op.startswith("v_mfma") or op.startswith("v_smfma"):
                count += 1
                n = shortest(code, i)
                if n is not None and n < NEED[op]:
                    found.append((name, i, op, n))
    return found, count


def test_every_path_of_the_library(tmp_path):
    if _build.stale():
        _build.build()
    shutil.copy(ss.LIB, tmp_path / "libss.so")
    subprocess.run([OBJDUMP, "--offloading", "libss.so"], cwd=tmp_path, check=True, capture_output=True)
    total = 0
    for f in sorted(tmp_path.iterdir()):
        if not f.name.endswith("gfx950"):
            continue
        text = subprocess.run([OBJDUMP, "-d", str(f)], check=True, capture_output=True, text=True).stdout
        found, count = short_ones(text)
        assert not found, found[:5]
        total += count
    assert total > 1000


LISTING = """
0000000000001000 <kernel>:
	v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0      // 000000001000: D3B50000 00000000
	s_cbranch_scc1 9                                           // 000000001008: BF850009 <kernel+0x{to:x}>
	{body}                                                     // 00000000100C: BF800000
	v_add_f32_e32 v5, v5, v6                                   // 000000001010: 020A0D05
	v_add_f32_e32 v0, v0, v6                                   // 000000001014: 02000D00
	s_endpgm                                                   // 000000001018: BF810000
"""


@pytest.mark.parametrize("body,to,states", [
    ("s_nop 7", 0x10, 2),        # the jump leaves the wait out: itself and one addition
    ("s_nop 7", 0xC, None),      # both ways wait
    ("s_nop 4", 0x14, 1),        # the jump goes to the use
    ("s_nop 4", 0xC, 7),
], ids=str)
def test_the_walk_finds_short_paths(body, to, states):
    found, count = short_ones(LISTING.format(body=body, to=to))
    assert count == 1
    assert [n for *_, n in found] == ([] if states is None else [states])
