"""Tensors on another device than the current one: the C library launches on the current device, so it is called with theirs
current.  (No GPU: fakes stand for the library and the devices.)"""
import contextlib

import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio


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
