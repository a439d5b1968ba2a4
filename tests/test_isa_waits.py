"""The built library's machine code, on the CPU: no kernel reads a matrix instruction's result before it is
written, on any path.  The rule and the walk over the paths are test_isa_tree's, here over every kernel of
libssd.so as llvm-objdump shows it."""
import concurrent.futures
import os
import re
import struct
import subprocess

import pytest

import ssd_chunked_scan_03_amd as ssd
import test_isa_tree as tree
from ssd_chunked_scan_03_amd import build

OBJDUMP = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.HIPCC))), "llvm", "bin", "llvm-objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(path):
    """The gfx950 code objects in the bundles that hipcc leaves in a library."""
    data = open(path, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        p = at + len(MAGIC) + 8
        for _ in range(struct.unpack_from("<Q", data, at + len(MAGIC))[0]):
            off, size, n = struct.unpack_from("<QQQ", data, p)
            if size and data[p + 24:p + 24 + n].endswith(build.ARCH.encode()):
                yield data[at + off:at + off + size]
            p += 24 + n
        at = data.find(MAGIC, at + 1)


def functions(text):
    """(name, instructions, position of each branch target) of a disassembly's kernels with matrix instructions; a
    branch names its target's address."""
    for part in re.split(r"\n(?=[0-9a-f]+ <)", text)[1:]:
        start, name = re.match(r"([0-9a-f]+) <([^>]+)>:", part).groups()
        ins, labels = [], {}
        for line in part.splitlines()[1:]:
            m = re.match(r"\s+(\S.*?)\s*// ([0-9A-F]+): [0-9A-F ]+(?:<[^>+]+(?:\+0x([0-9a-f]+))?>)?", line)
            if not m:
                continue
            code = re.sub(r"\s+", " ", m.group(1))
            if code.startswith(("s_branch", "s_cbranch")):
                code = f"{code.split()[0]} {int(start, 16) + int(m.group(3) or '0', 16)}"
            here = int(m.group(2), 16)
            if code.startswith("s_getpc_b64"):
                far = here + 4
            elif code.startswith("s_setpc_b64"):  # a branch too far for its offset: getpc, add, addc, setpc
                add = re.fullmatch(r"s_add_u32 s\d+, s\d+, (-?\w+)", ins[-2])
                assert ins[-3].startswith("s_getpc_b64") and add, ins[-3:]
                step = int(add.group(1), 0)
                code = f"s_branch {far + step - (step >> 31 << 32)}"
            labels[str(here)] = len(ins)
            ins.append(code)
        if any(i.startswith("v_mfma") for i in ins):
            yield name, ins, labels


def test_disassembly_is_followed():
    text = "\n0000000000001000 <f>:\n" + "\n".join(f"\t{c:40} // {0x1000 + 4 * i:012X}: BF800000{t}" for i, (c, t) in enumerate([
        ("v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]", ""), ("s_cbranch_scc1 2", " <f+0x10>"), ("s_nop 7", ""),
        ("s_endpgm", ""), ("v_accvgpr_read_b32 v9, a1", ""), ("s_endpgm", "")])) + "\n"
    [(name, ins, labels)] = functions(text)
    assert name == "f" and len(ins) == 6 and labels[ins[1].split()[1]] == 4
    assert [(r, n) for _, r, n in tree.early_reads(ins, labels)] == [(ins[4], 1)]


def early(job):
    """(kernels, {kernel: its first early read}) of one code object."""
    code, path = job
    with open(path, "wb") as f:
        f.write(code)
    text = subprocess.run([OBJDUMP, "-d", path], capture_output=True, text=True, check=True).stdout
    found = {}
    for name, ins, labels in functions(text):
        assert not any(c.startswith("s_swappc") for c in ins), name  # (calls are not followed)
        found[name] = tree.early_reads(ins, labels)[:1]
    return len(found), {k: v for k, v in found.items() if v}


def test_no_kernel_reads_a_product_too_early(tmp_path):
    lib = ssd.library_path()
    if not os.path.exists(lib) or not os.path.exists(OBJDUMP):
        pytest.skip("needs the built library and llvm-objdump")
    jobs = [(code, str(tmp_path / f"{i}.elf")) for i, code in enumerate(code_objects(lib))]
    with concurrent.futures.ProcessPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        found = list(pool.map(early, jobs))
    bad = {k: v for _, b in found for k, v in b.items()}
    assert sum(n for n, _ in found) > 500 and not bad, (len(bad), bad)
