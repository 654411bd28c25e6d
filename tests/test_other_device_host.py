"""Tensors on another device than the current one: the C library launches on the current device, so it is called with theirs
current, and kernels are allowed their LDS on each device once.  (No GPU: fakes stand for the library and the devices.)"""
import contextlib
import os
import shutil
import subprocess

import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


class FakeLibrary:
    """Every entry point returns OK and notes the device that is current; sizes of workspaces are zero."""

    def __init__(self, current):
        self.current, self.seen = current, []

    def __getattr__(self, name):
        def call(*args):
            if not name.endswith("workspace_size"):
                self.seen.append((name, self.current[-1]))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    current = [3]
    fake = FakeLibrary(current)

    @contextlib.contextmanager
    def device(d):
        current.append(d)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(kaio, "lib", lambda: fake)
    monkeypatch.setattr(kaio, "_fast", False)
    monkeypatch.setattr(kaio, "_quick", lambda: None)
    monkeypatch.setattr(kaio, "_tensor", lambda t, *a, **kw: t)
    monkeypatch.setattr(kaio, "_stream", lambda *a: None)
    return fake


def calls():
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8)
    x = f16(4, 128)
    paged = lambda: kaio.KaioPagedKV(f16(2, 16, 1, 64), f16(2, 16, 1, 64), i32(1, 2), i32(2), i32(1))
    experts = lambda: kaio.KaioExperts(f16(2, 128), i32(2, 16, 128), f16(2, 1, 128), i32(2, 16, 128), f16(2, 1, 128),
                                       i32(2, 16, 128), f16(2, 1, 128))
    w, s, w8 = i32(16, 64), f16(1, 64), i32(32, 64)
    return {
        "kaio_qkv_w4a16": lambda: kaio.kaio_qkv_w4a16(x, w, w, w, s, s, s),
        "kaio_qkv_w8a16": lambda: kaio.kaio_qkv_w8a16(x, w8, w8, w8, s, s, s),
        "kaio_gemm_f16f32": lambda: kaio.kaio_gemm_f16f32(x, f16(128, 8)),
        "kaio_gemm_f16f32_bwd": lambda: kaio.kaio_gemm_f16f32_bwd(x, f16(128, 8), torch.zeros(4, 8)),
        "kaio_dequant_group_bwd": lambda: kaio.kaio_dequant_group_bwd(x, f16(4, 2), 64),
        "kaio_linear_w4a16": lambda: kaio.kaio_linear_w4a16(x, w, s),
        "kaio_quantize_rows": lambda: kaio.kaio_quantize_rows(x),
        "kaio_linear_w8a8": lambda: kaio.kaio_linear_w8a8(x, i8(8, 128), torch.zeros(8)),
        "kaio_moe_w4a16": lambda: kaio.kaio_moe_w4a16(x, experts(), 1),
        "kaio_rope_append": lambda: kaio.kaio_rope_append(f16(1, 2, 64), f16(1, 1, 64), f16(1, 1, 64), i32(1, 1),
                                                          torch.zeros(32, dtype=torch.float64), [32], paged()),
        "kaio_paged_attention": lambda: kaio.kaio_paged_attention(f16(1, 2, 64), paged(), 1, 0.125),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_the_library_is_called_on_the_tensors_device(library, name):
    calls()[name]()
    assert library.seen == [(name, torch.device("cpu"))] and library.current == [3]


PROGRAM = r"""
#include <hip/hip_runtime.h>
static int device = 0, sets = 0;
static hipError_t next_result = hipSuccess;
static hipError_t fake_get(int* d) { *d = device; return hipSuccess; }
static hipError_t fake_set(const void*, hipFuncAttribute, int) { ++sets; return next_result; }
#define hipGetDevice fake_get
#define hipFuncSetAttribute fake_set
#include "launch.hpp"
#include <cstdio>
int main() {
  static kaio::LdsOf lds;
  int n = 0;
  for (int d : {0, 0, 1, 0, 1, 63, 63, 5}) {   // once on each
    device = d;
    if (lds.allow(nullptr, 100000) != hipSuccess) return 1;
  }
  n = sets;
  device = 7;
  next_result = hipErrorInvalidValue;          // an error is told, and not taken for done
  if (lds.allow(nullptr, 100000) != hipErrorInvalidValue) return 2;
  next_result = hipSuccess;
  if (lds.allow(nullptr, 100000) != hipSuccess) return 3;
  printf("%d %d\n", n, sets - n);
}
"""


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is needed")
def test_lds_is_allowed_on_each_device_once(tmp_path):
    (tmp_path / "lds.cpp").write_text(PROGRAM)
    exe = str(tmp_path / "lds")
    subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "int4_group_quantized_w4a16_amd", "csrc"), str(tmp_path / "lds.cpp"), "-o", exe],
                   check=True, capture_output=True)
    assert subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split() == ["4", "2"]
