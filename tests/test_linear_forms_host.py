"""The sizes of tests/linear_forms.py run every form that the selection (csrc/launch.hpp, host code) can choose."""
import os
import shutil
import subprocess

import pytest

from tests.linear_forms import SIZES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
PROGRAM = r"""
#include "launch.hpp"
#include <cstdio>
#include <cstdlib>
using namespace kaio;
int main(int argc, char** argv) {
  if (argc > 1) {
    for (int i = 1; i + 2 < argc; i += 3) {
      const uint32_t m = atoi(argv[i]), n = atoi(argv[i + 1]), k = atoi(argv[i + 2]);
      const LinearForm f = linear_form(m, n, k);
      printf("%u %d\n", f.code(), f.vec ? n % f.vec == 0 : n % 8 == 0);
    }
    return 0;
  }
  for (const LinearFormCost& c : kLinearForms) printf("%u 0\n%u 1\n", c.f.code(), c.f.code());
  for (uint32_t m = 1; m <= 4096; m += m < 130 ? 1 : 97)
    for (uint32_t n = 8; n <= 32776; n += 512)
      for (uint32_t odd = 0; odd < 4; ++odd)
        for (uint32_t k : {128u, 256u, 512u}) {
          const LinearForm f = linear_form(m, n + odd, k);
          printf("%u %d\n", f.code(), f.vec ? (n + odd) % f.vec == 0 : (n + odd) % 8 == 0);
        }
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
    assert len(forms) > 24
    assert tested == forms, sorted(forms - tested)
