"""The direct global->LDS loads of the built library.

They are inline assembly, which the compiler's hazard recogniser does not see.
A load needs one wait state after an instruction that wrote m0 and five after a
vector instruction that wrote its scalar base (v_readlane of a spilled one);
a base or m0 that is still on its way sends the load to a stale address.  Each
load therefore carries its guard, whatever the compiler puts before it or jumps
from: s_nop 4, or a scalar move of its base to itself (a wait state for m0; the
hardware holds it until the base is written, and the load until it is done).
The test reads that from the device code."""

import glob
import re
import shutil
import subprocess

import pytest

import mxfp8_block_scaled_topk_amd as mx

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def disassembly(tmp_path):
    lib = tmp_path / "lib.so"
    shutil.copy(mx.lib_path(), lib)
    subprocess.run([OBJDUMP, "--offloading", lib.name], cwd=tmp_path, check=True, capture_output=True)
    codes = sorted(glob.glob(f"{lib}.*gfx950"))
    assert codes
    return [subprocess.run([OBJDUMP, "-d", c], check=True, capture_output=True, text=True).stdout for c in codes]


def unguarded(text):
    """(loads into LDS, kernels whose loads lack the wait states with their counts)."""
    loads, bad, kernel, before = 0, {}, "", ""
    for line in text.splitlines():
        name = re.match(r"^[0-9a-f]+ <(.*)>:$", line)
        if name:
            kernel, before = name[1], ""
            continue
        op = line.split("//")[0].strip()
        if not line.startswith("\t") or not op:
            continue
        if re.match(r"(global|buffer|scratch)_load_lds|buffer_load.* lds$", op):
            loads += 1
            nop = re.match(r"s_nop (\d+)$", before)
            move = re.match(r"s_mov_b64 (s\[\d+:\d+\]), \1$", before)
            if not (nop and int(nop[1]) >= 4) and not (move and op.endswith(", " + move[1])):
                bad[kernel] = bad.get(kernel, 0) + 1
        before = op
    return loads, bad


def test_loads_into_lds_carry_their_wait_states(tmp_path):
    if not shutil.which(OBJDUMP):
        pytest.skip("no llvm-objdump")
    total = 0
    for text in disassembly(tmp_path):
        loads, bad = unguarded(text)
        total += loads
        assert not bad, bad
    assert total > 1000   # the kernels were found


@pytest.mark.parametrize("code,want", [
    ("s_mov_b32 m0, s3\n\tglobal_load_lds_dwordx4 v1, s[2:3]", 1),
    ("v_readlane_b32 s3, v9, 0\n\ts_nop 0\n\tglobal_load_lds_dword v1, s[2:3]", 1),
    ("s_mov_b64 s[2:3], s[2:3]\n\tglobal_load_lds_dwordx4 v1, s[2:3]", 0),
    ("s_mov_b64 s[2:3], s[2:3]\n\tglobal_load_lds_dwordx4 v1, s[4:5]", 1),
    ("s_mov_b32 m0, s3\n\ts_nop 4\n\tglobal_load_lds_dword v[2:3], off", 0),
])
def test_the_reading_itself(code, want):
    loads, bad = unguarded("0000000000001000 <kernel>:\n\t" + code + "\n")
    assert loads == 1 and bad.get("kernel", 0) == want
