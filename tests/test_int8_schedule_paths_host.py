"""The waits around the matrix instructions that csrc/int8.hip issues as assembly, along every path of the built code: through loops' back
edges and past branches, and with the instructions that write two registers. For each place in the code the least number of wait states
since a register was written by a vector instruction, and since a matrix instruction that writes it was issued, over all ways of getting
there, is found by going round until nothing changes."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import test_int8_schedule_host as straight
from conftest import ROOT

AFTER, BEFORE = straight.AFTER, straight.BEFORE
LONG = 64                                                                 # wait states beyond which nothing matters


def _parse(line):
    """(address, mnemonic, operands, branch target's address or None) of a line of the listing."""
    text, _, note = line.partition("//")
    op, _, rest = text.strip().partition(" ")
    operands = [o.strip() for o in re.split(r",(?![^\[]*\])", rest.strip())] if rest.strip() else []
    return int(note.split(":")[0], 16), op, operands, note


def _listing():
    tools = [os.path.join(straight.LLVM, t) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-objdump")]
    if not all(os.path.exists(t) for t in tools) or not os.path.exists(straight.OBJ):
        pytest.skip("the build's intermediate files or the tools are not here")
    return tools


def _kernels(tmp):
    objcopy, bundler, objdump = _listing()
    run = lambda *a: subprocess.run(a, check=True, capture_output=True, text=True).stdout  # noqa: E731
    obj, fat, co = (os.path.join(tmp, n) for n in ("int8.o", "fat", "co"))
    shutil.copy(straight.OBJ, obj)
    run(objcopy, f"--dump-section=.hip_fatbin={fat}", obj)
    target = [t for t in run(bundler, "--list", "--type=o", f"--input={fat}").split() if "gfx950" in t][0]
    run(bundler, "--unbundle", "--type=o", f"--targets={target}", f"--input={fat}", f"--output={co}")
    name, start, code = None, 0, {}
    for line in run(objdump, "-d", "--no-show-raw-insn", co).splitlines():
        m = re.match(r"^([0-9a-f]+) <(\w+)>:", line)
        if m:
            start, name = int(m.group(1), 16), m.group(2)
            code[name] = []
        elif name and "//" in line:                                       # not the padding behind a kernel
            at, op, operands, note = _parse(line)
            t = re.search(r"<\w+\+0x([0-9a-f]+)>", note)
            to = None if "branch" not in op else start + (int(t.group(1), 16) if t else 0)
            code[name].append((at, op, operands, to))
    return code


def _index(operand):
    return [n + (512 if kind == "a" else 0) for kind, n in straight._registers(operand)]


def hazards(insns):
    """Places where a matrix instruction reads what was written within BEFORE wait states, or something else touches a matrix
    instruction's result within AFTER, on any path. insns: (address, mnemonic, operands, branch target or None)."""
    place = {at: i for i, (at, *_) in enumerate(insns)}
    heads = sorted({0} | {place[to] for *_, to in insns if to is not None} |
                   {i + 1 for i, (_, op, _, to) in enumerate(insns) if (to is not None or op == "s_endpgm") and i + 1 < len(insns)})
    ends = dict(zip(heads, heads[1:] + [len(insns)]))
    steps = []
    for _, op, operands, _ in insns:
        matrix = op.startswith("v_mfma")
        vector = op.startswith("v_") and not matrix
        touches = matrix or op.startswith(("v_", "ds_", "global_", "buffer_", "flat_", "scratch_"))
        reads = _index(operands[1]) + _index(operands[2]) + _index(operands[0]) + _index(operands[3]) if matrix else []
        used = sorted({r for o in operands for r in _index(o)}) if touches else []
        wrote = operands[:2] if "swap" in op else operands[:1] if vector else []
        steps.append((matrix, reads, used, [r for o in wrote for r in _index(o)],
                      _index(operands[0]) if matrix else [],
                      int(operands[0], 0) + 1 if op == "s_nop" else 1))
    entry = {h: None for h in heads}
    entry[0] = np.full((2, 1024), LONG, np.int64)
    work, found = [0], {}
    while work:
        h = work.pop()
        written, issued = entry[h].copy()
        for i in range(h, ends[h]):
            matrix, reads, used, wrote, sums, states = steps[i]
            if matrix and (written[reads] <= BEFORE).any():
                found[i] = "an operand was just written"
            if used and (issued[used] <= AFTER).any():
                found[i] = "a matrix instruction's result is touched too early"
            written[wrote] = issued[sums] = 0
            written, issued = np.minimum(written + states, LONG), np.minimum(issued + states, LONG)
        _, op, _, to = insns[ends[h] - 1]
        follow = [] if op in ("s_endpgm", "s_branch") else [ends[h]]
        for n in follow + ([place[to]] if to is not None else []):
            now = np.stack([written, issued])
            if n in entry and (entry[n] is None or (now < entry[n]).any()):
                entry[n] = now if entry[n] is None else np.minimum(now, entry[n])
                work.append(n)
    assert all(entry[h] is not None for h in heads if any(s[0] for s in steps[h:ends[h]]))         # every matrix instruction is reached
    return [(hex(insns[i][0]), insns[i][1], insns[i][2], found[i]) for i in sorted(found)]


def test_large_tile_kernels(tmp_path):
    code = {n: c for n, c in _kernels(str(tmp_path)).items() if "int8_gemm_large_kernel" in n}
    assert len(code) == 8
    for name, insns in code.items():
        at = {a: i for i, (a, *_) in enumerate(insns)}
        assert sum(to is not None and at[to] <= i for i, (*_, to) in enumerate(insns)) >= 2, name       # its loops are seen
        assert not hazards(insns), (name, hazards(insns))


def _code(*lines):
    """Lines 'mnemonic operands' or 'label: mnemonic operands', branches to a label."""
    labels, out = {}, []
    for i, line in enumerate(lines):
        m = re.match(r"(\w+): (.*)", line)
        if m:
            labels[m.group(1)] = 4 * i
            line = m.group(2)
        op, _, rest = line.partition(" ")
        out.append((4 * i, op, [o.strip() for o in rest.split(", ")] if rest else []))
    return [(a, op, [] if "branch" in op else o, labels[o[0]] if "branch" in op else None) for a, op, o in out]


MFMA = "v_mfma_i32_16x16x64_i8 a[0:3], v[0:3], v[4:7], a[0:3]"


def test_the_check_itself():
    """Mistakes that a straight scan of the code passes over, and the same code without them."""
    gap = ["s_nop 15", "s_nop 15"]
    # a write at a loop's tail, read by the matrix instruction at its head
    assert hazards(_code("s_nop 0", "head: " + MFMA, *gap, "v_mov_b32_e32 v3, v9", "s_cbranch_scc1 head", "s_endpgm"))
    assert not hazards(_code("s_nop 0", "head: " + MFMA, *gap, "v_mov_b32_e32 v3, v9", "s_nop 4", "s_cbranch_scc1 head", "s_endpgm"))
    # a result read at a loop's head, issued at its tail
    assert hazards(_code("head: v_accvgpr_read_b32 v9, a2", "s_nop 4", MFMA, "s_cbranch_scc1 head", *gap, "s_endpgm"))
    assert not hazards(_code("head: v_accvgpr_read_b32 v9, a2", "s_nop 4", MFMA, *gap, "s_cbranch_scc1 head", "s_endpgm"))
    # a branch over the waits
    assert hazards(_code(MFMA, "s_cbranch_vccz past", *gap, "past: v_accvgpr_read_b32 v9, a0", "s_endpgm"))
    # the second register of a swap
    assert hazards(_code("v_permlane16_swap_b32_e32 v20, v5", MFMA, *gap, "s_endpgm"))
    assert not hazards(_code("v_permlane16_swap_b32_e32 v20, v21", MFMA, *gap, "s_endpgm"))
    # two uses of a sum in a row, and a store of an operand that nothing writes
    assert hazards(_code(MFMA, MFMA, *gap, "s_endpgm"))
    assert not hazards(_code(MFMA, "global_store_dword v[10:11], v4, off", *gap, "s_endpgm"))
