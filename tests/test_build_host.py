"""The C library is built and used also where its short Python call path cannot be."""
import os
import sys
import types

import pytest

import int4_group_quantized_w4a16_amd as kaio
from int4_group_quantized_w4a16_amd import build_lib


def test_the_library_is_built_without_the_binding(monkeypatch, tmp_path):
    # (nothing is compiled: only what happens when the binding's own compilation fails)
    old = tmp_path / "_binding.so"
    old.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build_lib, "_compile", lambda src, extra: src)
    monkeypatch.setattr(build_lib, "_link", lambda objs, lib: None)
    monkeypatch.setattr(build_lib, "BINDING", str(old))
    monkeypatch.setattr(build_lib, "BINDING_SOURCE", "no_such_file.cpp")
    with pytest.warns(UserWarning, match="ctypes"):
        assert build_lib.build() == build_lib.LIB
    assert not old.exists()


@pytest.fixture
def fresh(monkeypatch):
    """The package as before its first serving call, with a file where the binding would be."""
    monkeypatch.setattr(kaio, "_fast", None)
    monkeypatch.delattr(kaio, "_binding", raising=False)
    real = os.path.exists
    monkeypatch.setattr(os.path, "exists", lambda p: str(p).endswith("_binding.so") or real(p))
    return lambda module: monkeypatch.setitem(sys.modules, kaio.__name__ + "._binding", module)


def test_a_binding_that_does_not_load_is_left_alone(fresh):
    fresh(None)          # importing it raises ImportError
    with pytest.warns(UserWarning, match="does not load"):
        assert kaio._quick() is False
    assert kaio._quick() is False


def test_a_binding_of_another_torch_is_left_alone(fresh):
    def bind(*addresses):
        raise AssertionError("bound all the same")
    fresh(types.SimpleNamespace(torch_version="0.1", bind=bind))
    with pytest.warns(UserWarning, match="another torch"):
        assert kaio._quick() is False
    fresh(types.SimpleNamespace(bind=bind))
    kaio._fast = None
    with pytest.warns(UserWarning, match="another torch"):
        assert kaio._quick() is False


def test_the_binding_of_this_build_is_used():
    import torch
    if not os.path.exists(build_lib.BINDING):
        pytest.skip("not built")
    b = kaio._quick()
    assert b and b.torch_version == torch.__version__
