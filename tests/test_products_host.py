"""Refusals of the 8-bit product and of the mixture of experts on the host: every check runs before a device is touched
(fake pointers)."""
import ctypes

import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from tests.test_abi_host import A, ARG, DEVICE, OK, PROB, STEP, UNSUP, no_gpu_only

F32, BF16, F16 = 0, 1, 2


def last():
    return kaio.kaio_last_error()


def rows(dt=F16, x=A, q=A + STEP, scale=A + 2 * STEP, m=4, k=64):
    return kaio.lib().kaio_quantize_rows(dt, x, q, scale, m, k, None), last()


def linear(dt=F16, x=A, xs=A + STEP, w=A + 2 * STEP, ws=A + 3 * STEP, b=A + 4 * STEP, r=A + 5 * STEP, y=A + 6 * STEP,
           m=40, n=64, k=256, act=0, scratch=A + 7 * STEP, size=1 << 20):
    return kaio.lib().kaio_linear_w8a8(dt, x, xs, w, ws, b, r, y, m, n, k, act, scratch, size, None), last()


def experts(**kw):
    d = dict(router=A, w_gate=A + STEP, s_gate=A + 2 * STEP, w_up=A + 3 * STEP, s_up=A + 4 * STEP, w_down=A + 5 * STEP,
             s_down=A + 6 * STEP, experts=8, hidden=256, inner=128, group_size=128)
    d.update(kw)
    return kaio._Experts(**d)


def moe(e=None, x=A + 7 * STEP, r=A + 8 * STEP, y=A + 9 * STEP, tokens=3, top=2, act=4, ws=A + 10 * STEP, size=None, **kw):
    c = experts(**kw) if e is None else e
    ref = ctypes.byref(c) if c else None
    if size is None:
        size = kaio.lib().kaio_moe_w4a16_workspace_size(ref, tokens, top)
    return kaio.lib().kaio_moe_w4a16(ref, x, r, y, tokens, top, 1, act, ws, size, None), last()


def test_quantize_rows_refusals():
    for dt in (F32, 3, 7, -1):
        st, msg = rows(dt=dt)
        assert st == UNSUP and msg.startswith("kaio::quantize_rows:") and "dtype" in msg
    assert rows(k=72)[0] == PROB
    assert rows(m=0, x=0, q=0, scale=0)[0] == OK
    assert rows(m=1 << 24)[0] == PROB and rows(k=1 << 24)[0] == PROB
    for kw in (dict(x=0), dict(q=0), dict(scale=0)):
        st, msg = rows(**kw)
        assert st == ARG and "null" in msg
    for kw in (dict(x=A + 8), dict(q=A + STEP + 8), dict(scale=A + 2 * STEP + 4)):
        st, msg = rows(**kw)
        assert st == ARG and "16-byte aligned" in msg
    for kw, name in ((dict(q=A + 256), "x"), (dict(scale=A + 496), "x"), (dict(scale=A + STEP + 240), "scale")):
        st, msg = rows(**kw)
        assert st == ARG and msg.endswith("overlaps " + name)


def test_linear_w8a8_refusals():
    for dt in (F32, 3, 7, -1):
        st, msg = linear(dt=dt)
        assert st == UNSUP and msg.startswith("kaio::linear_w8a8:") and "dtype" in msg
    for act in (-1, 5, 2 ** 31 - 1):
        st, msg = linear(act=act)
        assert st == UNSUP and "activation" in msg
    assert linear(k=200)[0] == PROB and linear(k=131072)[0] == PROB
    assert linear(m=0, x=0, xs=0, y=0)[0] == OK and linear(n=0)[0] == OK
    assert linear(m=2 ** 32 - 1)[0] == PROB and linear(n=2 ** 26)[0] == PROB and linear(m=1 << 24)[0] == PROB
    for name, kw in (("x", dict(x=0)), ("input w", dict(w=0)), ("w_scale", dict(ws=0)), ("output y", dict(y=0)),
                     ("workspace", dict(xs=0, scratch=0))):
        st, msg = linear(**kw)
        assert st == ARG and name in msg and "null" in msg
    need = kaio.lib().kaio_linear_w8a8_workspace_size(40, 64, 256, 0)
    assert need >= 40 * 256 + 160 and kaio.lib().kaio_linear_w8a8_workspace_size(40, 64, 256, 1) == 0
    assert kaio.lib().kaio_linear_w8a8_workspace_size(40, 64, 200, 0) == 0
    assert kaio.lib().kaio_linear_w8a8_workspace_size(4, 64, 256, 0) == 0        # (rounded in the product's own workgroups)
    st, msg = linear(xs=0, size=need - 1)
    assert st == ARG and "workspace_bytes" in msg
    for kw in (dict(x=A + 8), dict(xs=A + STEP + 4), dict(w=A + 2 * STEP + 4), dict(ws=A + 3 * STEP + 4), dict(b=A + 4 * STEP + 2),
               dict(r=A + 5 * STEP + 2), dict(y=A + 6 * STEP + 2), dict(xs=0, scratch=A + 7 * STEP + 8)):
        st, msg = linear(**kw)
        assert st == ARG and "16-byte aligned" in msg
    for y, name in ((A + 16, "x"), (A + STEP, "x_scale"), (A + 2 * STEP, "w"), (A + 3 * STEP, "w_scale"), (A + 4 * STEP, "bias"),
                    (A + 5 * STEP + 16, "residual")):
        st, msg = linear(y=y)
        assert st == ARG and msg.endswith("overlaps " + name)
    assert linear(xs=0, scratch=A)[1].endswith("workspace overlaps x")
    assert linear(xs=0, scratch=A + 6 * STEP)[1].endswith("y overlaps workspace")


@no_gpu_only
def test_valid_calls_reach_the_device_check():
    for kw in ({}, dict(k=0, x=0, q=0), dict(dt=BF16), dict(m=1 << 20, k=16)):
        assert rows(**kw)[0] == DEVICE, kw
    for kw in ({}, dict(b=0, r=0), dict(r=A + 6 * STEP), dict(k=0, x=0, w=0), dict(act=4), dict(xs=0), dict(dt=BF16, xs=0),
               dict(scratch=0, size=0), dict(k=131056, m=1), dict(xs=0, x=A + 512)):
        assert linear(**kw)[0] == DEVICE, kw
    for kw in ({}, dict(r=0), dict(r=A + 9 * STEP), dict(top=8), dict(act=0), dict(tokens=200), dict(experts=512, top=16)):
        assert moe(**kw)[0] == DEVICE, kw


def test_moe_refusals():
    st, msg = moe(e=False, size=0)
    assert st == ARG and msg.startswith("kaio::moe_w4a16:") and "experts is null" in msg
    assert moe(group_size=64, size=0)[0] == UNSUP
    assert moe(act=5)[0] == UNSUP and moe(act=-1)[0] == UNSUP
    assert moe(experts=513)[0] == UNSUP and moe(experts=64, top=17)[0] == UNSUP
    for f in ("hidden", "inner"):
        for v in (0, 64, 200):
            assert moe(**{f: v})[0] == PROB
    for top in (0, 9):
        st, msg = moe(top=top)
        assert st == PROB and "top_k" in msg
    assert moe(experts=0)[0] == PROB
    assert moe(tokens=0, x=0, y=0, ws=0)[0] == OK
    assert moe(tokens=(1 << 17) + 1)[0] == PROB and moe(hidden=1 << 24)[0] == PROB and moe(inner=1 << 24)[0] == PROB
    for name in ("x", "y", "ws"):
        st, msg = moe(**{name: 0})
        assert st == ARG and "null" in msg
    for name in ("router", "w_gate", "s_gate", "w_up", "s_up", "w_down", "s_down"):
        st, msg = moe(**{name: 0})
        assert st == ARG and name in msg and "null" in msg
        st, msg = moe(**{name: A + 20 * STEP + 8})
        assert st == ARG and name in msg and "16-byte aligned" in msg
        st, msg = moe(**{name: A + 9 * STEP + 16})
        assert st == ARG and msg.endswith("y overlaps " + name)
    for kw in (dict(x=A + 7 * STEP + 2), dict(r=A + 8 * STEP + 2), dict(y=A + 9 * STEP + 2), dict(ws=A + 10 * STEP + 8)):
        st, msg = moe(**kw)
        assert st == ARG and "16-byte aligned" in msg
    need = kaio.lib().kaio_moe_w4a16_workspace_size(ctypes.byref(experts()), 3, 2)
    assert need > 0
    st, msg = moe(size=need - 1)
    assert st == ARG and "workspace_bytes" in msg
    assert moe(y=A + 7 * STEP + 16)[1].endswith("y overlaps x")
    assert moe(y=A + 8 * STEP + 16)[1].endswith("y overlaps residual")
    assert moe(ws=A + 5 * STEP)[1].endswith("workspace overlaps w_down")


def test_python_refusals():
    x = torch.zeros(2, 32, dtype=torch.float16)
    with pytest.raises(TypeError):
        kaio.kaio_quantize_rows([1])
    with pytest.raises(ValueError, match="HIP device"):
        kaio.kaio_quantize_rows(x)
    with pytest.raises(ValueError, match="HIP device"):
        kaio.kaio_linear_w8a8(x, torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(TypeError, match="int8"):
        kaio.kaio_linear_w8a8(x, torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4), x_scale=torch.zeros(2))
    with pytest.raises(ValueError, match="HIP device"):
        kaio.KaioExperts(*[torch.zeros(2, 128, dtype=torch.float16)] * 7)
    with pytest.raises(TypeError, match="KaioExperts"):
        kaio.kaio_moe_w4a16(x, None, 2)
