"""What the compiler made of the kernels, read from the built library.

A branch over a region that no lane enters (s_cbranch_execz) ends where exec is restored. The compiler (ROCm 7.2) may put the
copy of a spilled register at that end, before exec is restored: lanes that skipped the region then keep what the register held
before, and results depend on what ran earlier. A variant of the kernel behind dq of window attention (fp32, heads of 96) met
this: two of four waves never entered the region, and wrote dq and delta by a stale register. No source line shows it, so the
library is read for it; a kernel named here needs fewer live registers.
"""
import os
import re
import shutil
import subprocess

import pytest

_LLVM = "/opt/rocm/llvm/bin/llvm-objdump"
_LINE = re.compile(r"^\t(\S+)(.*?)\s*// ([0-9A-F]{12}):")
_COPY = re.compile(r"v_accvgpr_|scratch_|buffer_(load|store)")


def spills_before_exec(text):
    """(kernel, instruction) for each copy of a spilled register between the end of a skipped region and exec's restore."""
    found = []
    for part in re.split(r"\n(?=[0-9a-f]{16} <)", text):
        head = re.match(r"([0-9a-f]{16}) <([^>]+)>:", part)
        if not head:
            continue
        start, name, at, code = int(head.group(1), 16), head.group(2), {}, []
        ends = set()
        for line in part.split("\n"):
            m = _LINE.match(line)
            if not m:
                continue
            at[int(m.group(3), 16)] = len(code)
            code.append(m.group(1) + m.group(2))
            if m.group(1) == "s_cbranch_execz":
                to = re.search(r"<[^>]*?\+0x([0-9a-fA-F]+)>\s*$", line)
                assert to, line
                ends.add(start + int(to.group(1), 16))
        for end in ends:
            copies = []
            for ins in code[at[end]:]:
                if re.match(r"s_or_b64 exec, exec,", ins):
                    found += [(name, c) for c in copies]
                    break
                if re.match(r"s_c?branch|s_endpgm|s_\S*saveexec|s_\S+ exec", ins):
                    break
                if _COPY.match(ins):
                    copies.append(ins)
    return found


def _block(*lines):
    return "0000000000001000 <k>:\n" + "\n".join(f"\t{i} // {0x1000 + 4 * n:012X}: 00000000{to}"
                                                 for n, (i, to) in enumerate(lines))


def test_the_check_finds_what_it_is_for():
    skip = ("s_cbranch_execz 1", " <k+0x8>")
    copy, restore = ("v_accvgpr_write_b32 a57, v35", ""), ("s_or_b64 exec, exec, s[20:21]", "")
    inside = ("global_load_dwordx4 v[26:29], v[26:27], off", "")
    assert spills_before_exec(_block(skip, inside, copy, restore)) == [("k", "v_accvgpr_write_b32 a57, v35")]
    assert spills_before_exec(_block(skip, inside, restore, copy)) == []
    assert spills_before_exec(_block(skip, copy, restore, inside)) == []


def test_no_spill_is_copied_where_lanes_are_off(tmp_path):
    import sparse_convolution_amd
    library = os.path.join(os.path.dirname(sparse_convolution_amd.__file__), "libigconv.so")
    if not (os.path.exists(_LLVM) and os.path.exists(library)):
        pytest.skip("no disassembler or no built library")
    shutil.copy(library, tmp_path)
    subprocess.run([_LLVM, "--offloading", "libigconv.so"], cwd=tmp_path, check=True, capture_output=True)
    objects = sorted(p for p in tmp_path.iterdir() if "gfx950" in p.name)
    assert objects
    kernels = 0
    for p in objects:
        text = subprocess.run([_LLVM, "-d", str(p)], check=True, capture_output=True, text=True).stdout
        kernels += text.count("s_endpgm")
        found = spills_before_exec(text)
        assert not found, found[:3]
    assert kernels
