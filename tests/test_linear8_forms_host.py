"""The sizes of tests/linear8_forms.py run every form that the selection (csrc/launch.hpp, host code) can choose."""
import os
import shutil
import subprocess

import pytest

from tests.linear8_forms import SIZES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
PROGRAM = r"""
#include "launch.hpp"
#include <cstdio>
#include <cstdlib>
using namespace kaio;
// a form; whether k is ragged (tiles) or who rounds 16-bit tokens (strips); whether a workgroup takes several tiles
void tell(uint32_t m, uint32_t n, uint32_t k) {
  const Linear8Form f = linear8_form(m, n);
  bool several = false;
  for (const Linear8Cost& c : kLinear8Forms)
    if (c.f == f && c.channels >= 128) several = (uint64_t)((m + c.tokens - 1) / c.tokens) * ((n + c.channels - 1) / c.channels) > kComputeUnits;
  printf("%d %d %d\n", (int)f, m <= 16 ? linear8_rounds(m, n, k) : k % 128 != 0, several);
}
int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3) tell(atoi(argv[i]), atoi(argv[i + 1]), atoi(argv[i + 2]));
  if (argc > 1) return 0;
  for (uint32_t m = 1; m <= 8192; m += m < 130 ? 1 : 97)
    for (uint32_t n = 8; n <= 65544; n += 512)
      for (uint32_t k : {256u, 400u, 8192u}) tell(m, n, k);
}
"""


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is needed")
def test_every_form_has_a_size(tmp_path):
    (tmp_path / "forms.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "forms")
    subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "int4_group_quantized_w4a16_amd", "csrc"), str(tmp_path / "forms.cpp"), "-o", exe],
                   check=True, capture_output=True)
    run = lambda *a: subprocess.run([exe, *a], check=True, capture_output=True, text=True).stdout.splitlines()
    forms, tested = set(run()), set(run(*[str(x) for size in SIZES for x in size]))
    assert len({f.split()[0] for f in forms}) == 10
    assert tested == forms, sorted(forms ^ tested)
