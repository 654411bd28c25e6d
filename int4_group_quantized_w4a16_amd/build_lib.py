"""Build libkaio.so (the gfx950 HIP kernels plus the C ABI) in-tree with hipcc.

    python -m int4_group_quantized_w4a16_amd.build_lib
    python -m int4_group_quantized_w4a16_amd.build_lib --host-sanitizers

The second form builds _build/sanitize/libkaio.so: the same kernels, with the
host-side ABI layer (validation, device check, dispatch) instrumented by
AddressSanitizer and UndefinedBehaviorSanitizer (host code only; the GPU code
is built as usual).  Run the CPU boundary tests against it with

    LD_PRELOAD=$(/opt/rocm/llvm/bin/clang -print-file-name=libclang_rt.asan-x86_64.so) \
    ASAN_OPTIONS=detect_leaks=0 UBSAN_OPTIONS=halt_on_error=1 \
    KAIO_LIBRARY=$PWD/int4_group_quantized_w4a16_amd/_build/sanitize/libkaio.so \
    python -m pytest tests/test_abi_host.py
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkaio.so")
SOURCES = ["kaio_abi.cpp", "qkv_prefill.hip", "qkv_decode.hip", "gemm_f16f32.hip", "dequant_group_bwd.hip",
           "linear_w4a16.hip", "rope_append.hip", "attention_rows.hip", "attention_stream.hip", "attention_join.hip",
           "attention_tile.hip"]
# measurement aid for the benchmark (a plain streaming read), a library of its own
ROOF_LIB = os.path.join(PKG, "libkaio_roof.so")
ROOF_SOURCES = ["roof.hip"]

# the Python call path of the serving operators (host code, against torch's headers)
BINDING = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = "torch_binding.cpp"

ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # keep packed-FP32 VALU ops out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link(objs, lib):
    tmp = lib + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


# host-only sanitizer flags: each one behind -Xarch_host so that no GPU code is instrumented
HOST_SANITIZE = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                 "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer",
                 "-g"]


def build_host_sanitized(verbose: bool = False) -> str:
    """libkaio.so with the host ABI layer under ASan/UBSan, in _build/sanitize/ (CPU testing only)."""
    out = os.path.join(BUILD, "sanitize")
    os.makedirs(out, exist_ok=True)
    objs = []
    for src in SOURCES:
        stem = os.path.splitext(src)[0] + ".o"
        plain = os.path.join(BUILD, stem)
        if not src.endswith(".cpp") and os.path.exists(plain) and \
                os.path.getmtime(plain) >= os.path.getmtime(os.path.join(CSRC, src)):
            objs.append(plain)        # GPU sources: the regular build's object, unchanged
            continue
        obj = os.path.join(out, stem)
        extra = HOST_SANITIZE if src.endswith(".cpp") else []
        cmd = [hipcc(), *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        objs.append(obj)
    lib = os.path.join(out, "libkaio.so")
    _link(objs, lib)
    if verbose:
        print(f"built {lib}")
    return lib


def build_binding() -> str:
    """_binding.so: csrc/torch_binding.cpp by the host compiler, for the torch that is here (it says which)."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include")]
    libs = os.path.join(root, "lib")
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DKAIO_TORCH_VERSION="{torch.__version__}"', *[f"-I{i}" for i in inc],
           os.path.join(CSRC, BINDING_SOURCE), "-o", tmp, f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10",
           "-lc10_hip", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SOURCE}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


def _binding_if_possible() -> str:
    """build_binding(), or, where torch's headers, its libraries or a host compiler are missing, a warning and no
    binding (nor an older one): Python then calls the C library by ctypes, a few us slower per call."""
    try:
        return build_binding()
    except (ImportError, OSError, RuntimeError) as e:
        if os.path.exists(BINDING):
            os.remove(BINDING)
        warnings.warn(f"{os.path.basename(BINDING)} was not built, calls go through ctypes: {e}")
        return ""


def build(extra_flags=(), verbose: bool = False) -> str:
    """Compile every source for gfx950, link libkaio.so (and the benchmark's
    libkaio_roof.so) and, where that is possible, the Python binding; returns the
    path of libkaio.so."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = SOURCES + ROOF_SOURCES
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        binding = ex.submit(_binding_if_possible)
        objs = list(ex.map(lambda s: _compile(s, list(extra_flags)), srcs))
    _link(objs[:len(SOURCES)], LIB)
    _link(objs[len(SOURCES):], ROOF_LIB)
    built = [LIB, ROOF_LIB] + [b for b in (binding.result(),) if b]
    if verbose:
        print("built " + ", ".join(built))
    return LIB


if __name__ == "__main__":
    if sys.argv[1:] == ["--host-sanitizers"]:
        build_host_sanitized(verbose=True)
    else:
        build(extra_flags=sys.argv[1:], verbose=True)
