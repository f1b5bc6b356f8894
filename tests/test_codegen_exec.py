"""The rest of what tests/test_codegen.py looks for: a spilled register copied where a skipped region ends, before lanes are on again,
whatever turns them on (or a branch away first).

A region that lanes skip starts with an instruction that takes lanes out of exec (s_and_saveexec_b64 and others) and a branch over it if none is left;
a branch of this kind without such an instruction before it in its block is taken or not by all lanes, and ends nothing.
"""
import os
import re
import shutil
import subprocess

import pytest

from tests.test_codegen import _COPY, _LINE, _LLVM

_NARROWS = re.compile(r"s_(and|andn2|xor|nand|andn1)\w*_saveexec_b64|s_(and|andn2|xor)_b64 exec,")
_WRITES = re.compile(r"s_\w+ exec,|s_\w+_saveexec_b64")
_LEAVES = re.compile(r"s_c?branch|s_endpgm|s_setpc|s_swappc")


def copies_in_the_dark(text):
    """(kernel, instruction) for each copy of a spilled register between the end of a region that lanes skip and the next write of exec."""
    found = []
    for part in re.split(r"\n(?=[0-9a-f]{16} <)", text):
        head = re.match(r"([0-9a-f]{16}) <([^>]+)>:", part)
        if not head:
            continue
        start, name, at, code, to = int(head.group(1), 16), head.group(2), {}, [], {}
        for line in part.split("\n"):
            m = _LINE.match(line)
            if not m:
                continue
            at[int(m.group(3), 16)] = len(code)
            if re.match(r"s_c?branch", m.group(1)):
                target = re.search(r"<[^>+]*(?:\+0x([0-9a-fA-F]+))?>\s*$", line)
                assert target, line
                to[len(code)] = start + int(target.group(1) or "0", 16)
            code.append(m.group(1) + m.group(2))
        labels = {at[t] for t in to.values() if t in at}
        for i, target in to.items():
            if not code[i].startswith("s_cbranch_execz"):
                continue
            narrowed, k = False, i
            while k > 0 and k not in labels and not _LEAVES.match(code[k - 1]):
                k -= 1
                if _NARROWS.match(code[k]) or _WRITES.match(code[k]):
                    narrowed = bool(_NARROWS.match(code[k]))
                    break
            if not narrowed:
                continue
            for ins in code[at[target]:]:
                if _WRITES.match(ins) or _LEAVES.match(ins):
                    break
                if _COPY.match(ins):
                    found.append((name, ins))
    return found


def _block(*lines):
    return "0000000000001000 <k>:\n" + "\n".join(f"\t{i} // {0x1000 + 4 * n:012X}: 00000000{to}" for n, (i, to) in enumerate(lines))


@pytest.mark.parametrize("restore", ["s_or_b64 exec, exec, s[20:21]", "s_mov_b64 exec, s[20:21]", "s_or_saveexec_b64 s[2:3], s[20:21]", "s_branch 3"])
def test_the_check_finds_what_it_is_for(restore):
    skip, narrow = ("s_cbranch_execz 2", " <k+0xc>"), ("s_and_saveexec_b64 s[20:21], vcc", "")
    inside, copy = ("global_load_dwordx4 v[26:29], v[26:27], off", ""), ("v_accvgpr_write_b32 a57, v35", "")
    back = (restore, " <k+0x0>" if "branch" in restore else "")
    assert copies_in_the_dark(_block(narrow, skip, inside, copy, back)) == [("k", "v_accvgpr_write_b32 a57, v35")]
    if "branch" not in restore:
        assert copies_in_the_dark(_block(narrow, skip, inside, back, copy)) == []
    # A branch of all lanes.
    assert copies_in_the_dark(_block(("s_mov_b64 s[2:3], 0", ""), skip, inside, copy, back)) == []
    assert copies_in_the_dark(_block(("s_or_b64 exec, exec, s[4:5]", ""), skip, inside, copy, back)) == []


def test_no_spill_is_copied_in_the_dark(tmp_path):
    import sparse_convolution_amd
    library = os.path.join(os.path.dirname(sparse_convolution_amd.__file__), "libigconv.so")
    if not (os.path.exists(_LLVM) and os.path.exists(library)):
        pytest.skip("no disassembler or no built library")
    shutil.copy(library, tmp_path)
    subprocess.run([_LLVM, "--offloading", "libigconv.so"], cwd=tmp_path, check=True, capture_output=True)
    objects = sorted(p for p in tmp_path.iterdir() if "gfx950" in p.name)
    assert objects
    for p in objects:
        text = subprocess.run([_LLVM, "-d", str(p)], check=True, capture_output=True, text=True).stdout
        found = copies_in_the_dark(text)
        assert not found, found[:3]
