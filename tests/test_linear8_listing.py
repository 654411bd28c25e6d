"""The 8-bit product's direct loads to LDS bring their own wait states (why: tests/test_kernel_listing.py)."""
import os
import shutil
import subprocess

import pytest

import int4_group_quantized_w4a16_amd as kaio
from tests.test_kernel_listing import OBJDUMP, short_of_states


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="llvm-objdump is needed")
def test_direct_loads_bring_their_own_wait_states(tmp_path):
    lib = shutil.copy(kaio.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    loads = 0
    for obj in sorted(tmp_path.glob("lib.so.*gfx950")):
        if b"linear8_tile_kernel" not in obj.read_bytes():
            continue
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(obj)], check=True, capture_output=True, text=True)
        n, short = short_of_states(text.stdout.splitlines())
        assert not short, f"{len(short)} of {n} loads, first (instruction, states): {short[:3]}"
        loads += n
    assert loads > 0
