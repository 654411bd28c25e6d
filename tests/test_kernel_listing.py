"""Waits that the compiler does not insert, checked in the listing of the built kernels.

The tile form's direct loads to LDS stand in inline assembly, whose instructions the compiler's hazard pass does not
see.  A vector-memory instruction may read a scalar register (its descriptor, its offset) only five wait states after
a vector instruction (a lane read that brings a spilled descriptor back) wrote it.  So the five states before every
such load have to be the assembly's own.
"""
import os
import re
import shutil
import subprocess

import pytest

import int4_group_quantized_w4a16_amd as kaio

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
STATES = 5
LOAD = re.compile(r"buffer_load_dword(x4)? v\d+, s\[\d+:\d+\], \S+ offen lds$")
OWN = re.compile(r"(s_mul_i32|s_nop|s_mov_b32 m0,|s_add_u32 m0,|buffer_load_dword)")


def short_of_states(listing):
    """(direct loads, those with fewer than STATES wait states of the assembly's own before them)"""
    ins = [x for x in (line.split("//")[0].strip() for line in listing) if x]
    loads, short = 0, []
    for at, text in enumerate(ins):
        if not LOAD.match(text):
            continue
        loads += 1
        states, j = 0, at - 1
        while states < STATES and j >= 0 and OWN.match(ins[j]):
            nop = re.match(r"s_nop (\d+)", ins[j])
            states += 1 + (int(nop[1]) if nop else 0)
            j -= 1
        if states < STATES:
            short.append((at, states))
    return loads, short


def test_the_count_itself():
    load = "\tbuffer_load_dwordx4 v8, s[16:19], s7 offen lds      // 000000006740: E05D1000"
    lane = "v_readlane_b32 s16, v9, 3"
    assert short_of_states([lane, "s_mul_i32 s7, s5, s6", "s_mov_b32 m0, s4", "s_nop 0", load]) == (1, [(4, 3)])
    assert short_of_states([lane, "s_mul_i32 s7, s5, s6", "s_mov_b32 m0, s4", "s_nop 2", load]) == (1, [])
    assert short_of_states(["s_nop 3", lane, load]) == (1, [(2, 0)])


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump is needed")
def test_direct_loads_bring_their_own_wait_states(tmp_path):
    lib = shutil.copy(kaio.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    loads = 0
    for obj in sorted(tmp_path.glob("lib.so.*gfx950")):
        if b"attention_tile_kernel" not in obj.read_bytes():
            continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(obj)], check=True, capture_output=True, text=True)
        n, short = short_of_states(text.stdout.splitlines())
        assert not short, f"{len(short)} of {n} loads, first (instruction, states): {short[:3]}"
        loads += n
    assert loads > 0
