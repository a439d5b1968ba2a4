"""Machine-code checks of the tree's kernels on the CPU, from the assembly that hipcc writes for gfx950:

- no register spills;
- no read of a matrix instruction's result before it is written, on any path.  The hardware does not
  wait there; the compiler states the waits, but it has left them out where a branch lies between the
  instruction and the read (an accumulator copied at the start of the block behind).  Followed here over every
  path: an instruction is one wait state, s_nop n is n + 1."""
import os
import re
import shutil
import subprocess

import pytest

from ssd_chunked_scan_03_amd import build

# wait states from the instruction to a read of its result: what the compiler itself keeps within a block
NEED = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10}
READERS = ("ds_write", "ds_add", "ds_or", "ds_and", "ds_min", "global_store", "buffer_store", "flat_store", "scratch_store")


def regs(text):
    out = set()
    for m in re.finditer(r"\b([va])(\d+)\b|\b([va])\[(\d+):(\d+)\]", text):
        if m.group(1):
            out.add((m.group(1), int(m.group(2))))
        else:
            out |= {(m.group(3), i) for i in range(int(m.group(4)), int(m.group(5)) + 1)}
    return out


def operands(line):
    op, _, rest = line.partition(" ")
    return op, [p.strip() for p in re.split(r",(?![^\[]*\])", rest)]


def uses(line):
    """(registers read, registers written) of one instruction."""
    op, p = operands(line)
    if op.startswith("s_"):
        return set(), set()
    if op.startswith(READERS) or op.startswith("v_cmp"):
        return regs(",".join(p)), set()
    if op.startswith(("v_readlane", "v_readfirstlane")):
        return regs(",".join(p[1:])), set()
    r, w = regs(",".join(p[1:])), regs(p[0])
    if op.startswith(("v_fmac", "v_mac", "v_writelane", "v_permlane", "v_swap")) or "dpp" in line or "sdwa" in line:
        r |= w
    if op.startswith(("v_permlane", "v_swap")):
        w |= regs(p[1])
    return r, w


def functions(asm):
    for part in re.split(r"\n\t\.globl\t", asm)[1:]:
        name, ins, labels = part.split()[0], [], {}
        for line in part.split(".section")[0].splitlines():
            line = line.split(";")[0].strip()
            m = re.match(r"^(\.LBB\w+):", line)
            if m:
                labels[m.group(1)] = len(ins)
            elif line and not line.startswith(".") and not line.endswith(":"):
                ins.append(line)
        if any(i.startswith("v_mfma") for i in ins):
            yield name, ins, labels


def early_reads(ins, labels):
    """(matrix instruction, the instruction that reads its result, wait states between them), too few."""
    found = []
    for at, line in enumerate(ins):
        if not line.startswith("v_mfma"):
            continue
        op, p = operands(line)
        todo, seen = [(at + 1, 0, frozenset(regs(p[0])))], {}
        while todo:
            j, gone, live = todo.pop()
            if gone >= NEED[op] or j >= len(ins) or not live or seen.get((j, live), 99) <= gone:
                continue
            seen[j, live] = gone
            nxt, q = operands(ins[j])
            if nxt == "s_endpgm":
                continue
            if nxt.startswith("v_mfma"):  # (accumulating on the same registers is ordered by the hardware)
                read, wrote = regs(",".join(q[1:3])), regs(q[0])
            else:
                read, wrote = uses(ins[j])
            if read & live:
                found.append((line, ins[j], gone))
                continue
            live = frozenset(live - wrote)
            if nxt == "s_branch" or nxt.startswith("s_cbranch"):
                todo.append((labels[q[0]], gone + 1, live))
            if nxt != "s_branch":
                m = re.match(r"s_nop\s+(\d+)", ins[j])
                todo.append((j + 1, gone + (int(m.group(1)) + 1 if m else 1), live))
    return found


def test_scanner_sees_a_read_behind_a_branch():
    text = """
	.globl	f
f:
	v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]
	s_cbranch_vccnz .LBB0_2
	s_nop 7
	s_endpgm
.LBB0_2:
	%s
	v_accvgpr_read_b32 v9, a1
	s_endpgm
	.section x
"""
    for fill, bad in (("s_nop 0", 1), ("s_nop 5", 1), ("s_nop 6", 0), ("v_mov_b32 v8, v7", 1), ("v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]", 1)):
        [(_, ins, labels)] = functions(text % fill)
        assert len(early_reads(ins, labels)) == bad, fill


@pytest.mark.parametrize("unit", ["tree_bf16.hip", "tree_f32.hip"])
def test_tree_kernels(tmp_path, unit):
    if not (os.path.exists(build.HIPCC) or shutil.which(build.HIPCC)):
        pytest.skip("hipcc not available")
    out = tmp_path / (unit + ".s")
    r = subprocess.run([build.HIPCC, *build.CFLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, unit), "-o", str(out)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    asm = out.read_text()
    kernels = list(functions(asm))
    assert len(kernels) >= 50
    for name, ins, labels in kernels:
        assert early_reads(ins, labels) == [], name
    spills = re.findall(r"\.vgpr_spill_count:\s+(\d+)", asm)
    assert len(spills) >= 50 and not any(int(n) for n in spills), spills
