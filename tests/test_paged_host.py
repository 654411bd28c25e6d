"""Refusals of the serving operators on the host: every check runs before a device is touched (fake pointers)."""
import ctypes

import pytest

import int4_group_quantized_w4a16_amd as kaio
from tests.test_abi_host import A, ARG, DEVICE, OK, PROB, STEP, UNSUP, no_gpu_only

F16, BF16 = 2, 1


def last():
    return kaio.kaio_last_error()


def paged(**kw):
    d = dict(k_cache=A, v_cache=A + STEP, page_table=A + 2 * STEP, q_start=A + 3 * STEP, lens=A + 4 * STEP, dtype=F16,
             pages=10, page_size=16, kv_heads=2, head_dim=64, seqs=3, table_width=4)
    d.update(kw)
    return kaio._PagedKV(**d)


def rope(kv=None, q=A + 5 * STEP, k=A + 6 * STEP, v=A + 7 * STEP, pos=A + 8 * STEP, inv=A + 9 * STEP, sections=(32,),
         axes=None, q_out=A + 10 * STEP, tokens=3, hq=4, **kw):
    c = paged(**kw) if kv is None else kv
    sec = None if sections is None else (ctypes.c_uint32 * len(sections))(*sections)
    st = kaio.lib().kaio_rope_append(ctypes.byref(c) if c else None, q, k, v, pos, inv, sec,
                                     len(sections or ()) if axes is None else axes, 0, q_out, tokens, hq, None)
    return st, last()


def attn(kv=None, q=A + 5 * STEP, out=A + 6 * STEP, tokens=3, hq=4, max_new=1, scale=0.1, window=0, sinks=0,
         ws=A + 7 * STEP, ws_bytes=None, **kw):
    c = paged(**kw) if kv is None else kv
    ref = ctypes.byref(c) if c else None
    if ws_bytes is None:
        ws_bytes = kaio.lib().kaio_paged_attention_workspace_size(ref, tokens, hq, max_new)
    st = kaio.lib().kaio_paged_attention(ref, q, out, tokens, hq, max_new, scale, window, sinks, ws, ws_bytes, None)
    return st, last()


def linear(x=A, w=A + STEP, s=A + 2 * STEP, b=A + 3 * STEP, r=A + 4 * STEP, y=A + 5 * STEP, m=4, n=64, k=256, g=128, act=0):
    return kaio.lib().kaio_linear_w4a16(x, w, s, b, r, y, m, n, k, g, act, None), last()


def test_linear_refusals():
    st, msg = linear(g=64)
    assert st == UNSUP and msg.startswith("kaio::linear_w4a16:") and "group_size" in msg
    for act in (-1, 5, 2 ** 31 - 1):
        st, msg = linear(act=act)
        assert st == UNSUP and "activation" in msg
    assert linear(k=200)[0] == PROB
    assert linear(m=0, x=0, y=0)[0] == OK and linear(n=0)[0] == OK
    assert linear(m=2 ** 32 - 1, n=2 ** 26 - 1)[0] == PROB
    assert linear(n=2 ** 26)[0] == PROB and linear(k=2 ** 24)[0] == PROB
    for name, kw in (("x", dict(x=0)), ("w_packed", dict(w=0)), ("scales", dict(s=0)), ("output y", dict(y=0))):
        st, msg = linear(**kw)
        assert st == ARG and name in msg and "null" in msg
    for kw in (dict(x=A + 8), dict(w=A + STEP + 4), dict(s=A + 2 * STEP + 2), dict(b=A + 3 * STEP + 2), dict(r=A + 4 * STEP + 2), dict(y=A + 5 * STEP + 2)):
        st, msg = linear(**kw)
        assert st == ARG and "16-byte aligned" in msg
    for y, name in ((A + 16, "x"), (A + STEP, "w_packed"), (A + 2 * STEP, "scales"), (A + 3 * STEP, "bias"), (A + 4 * STEP + 16, "residual")):
        st, msg = linear(y=y)
        assert st == ARG and msg.endswith("overlaps " + name)


@no_gpu_only
def test_linear_valid_calls_reach_the_device_check():
    for kw in ({}, dict(b=0, r=0), dict(r=A + 5 * STEP), dict(k=0, x=0, w=0, s=0), dict(act=4)):
        assert linear(**kw)[0] == DEVICE, kw


def test_rope_append_refusals():
    st, msg = rope(kv=False)
    assert st == ARG and msg.startswith("kaio::rope_append:") and "kv is null" in msg
    for dt in (0, 3, 7, -1):
        assert rope(dtype=dt)[0] == UNSUP
    for f in ("page_size", "kv_heads", "head_dim"):
        assert rope(**{f: 0})[0] == PROB
    assert rope(sections=(), axes=0)[0] == UNSUP
    assert rope(sections=(4,) * 9)[0] == UNSUP
    assert rope(head_dim=1040)[0] == UNSUP
    assert rope(sections=None, axes=1)[0] == ARG
    assert rope(sections=(33,))[0] == PROB and rope(sections=(20, 13))[0] == PROB
    assert rope(sections=(2 ** 32 - 1, 2 ** 32 - 1, 2))[0] == PROB
    assert rope(tokens=0, q=0, k=0)[0] == OK
    assert rope(tokens=2 ** 24)[0] == PROB
    assert rope(pages=2 ** 27)[0] == PROB                       # 2^31 slots
    assert rope(hq=2 ** 26)[0] == PROB
    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(pos=0), dict(inv=0), dict(q_out=0), dict(k_cache=0), dict(v_cache=0),
               dict(page_table=0), dict(q_start=0), dict(lens=0)):
        st, msg = rope(**kw)
        assert st == ARG and "is null" in msg, kw
    for kw in (dict(q=A + 5 * STEP + 8), dict(pos=A + 8 * STEP + 2), dict(inv=A + 9 * STEP + 4), dict(k_cache=A + 8),
               dict(page_table=A + 2 * STEP + 1), dict(lens=A + 4 * STEP + 2)):
        st, msg = rope(**kw)
        assert st == ARG and "aligned" in msg, kw
    cache = 10 * 16 * 2 * 64 * 2
    assert "q_out overlaps q" in rope(q_out=A + 5 * STEP + 16)[1]
    assert "q_out overlaps k_cache" in rope(q_out=A + cache - 16)[1]
    assert "k_cache overlaps v_cache" in rope(v_cache=A + cache - 16)[1]
    assert "v_cache overlaps v" in rope(v=A + STEP)[1]
    assert "overlaps page_table" in rope(page_table=A + STEP + 16)[1]


@no_gpu_only
def test_rope_append_valid_calls_reach_the_device_check():
    for kw in ({}, dict(q_out=A + 5 * STEP), dict(sections=(0,), pos=0, inv=0), dict(hq=0, q=0, q_out=0),
               dict(seqs=0, page_table=0, q_start=0, lens=0), dict(dtype=BF16), dict(head_dim=72, sections=(5, 6)),
               dict(v_cache=A + 10 * 16 * 2 * 64 * 2)):
        assert rope(**kw)[0] == DEVICE, (kw, last())


def test_attention_refusals():
    st, msg = attn(kv=False, ws_bytes=0)
    assert st == ARG and msg.startswith("kaio::paged_attention:") and "kv is null" in msg
    for dt in (0, 3, -5):
        assert attn(dtype=dt)[0] == UNSUP
    for f in ("page_size", "kv_heads", "head_dim"):
        assert attn(**{f: 0})[0] == PROB
    assert attn(hq=5)[0] == PROB
    for scale in (float("nan"), float("inf")):
        assert attn(scale=scale)[0] == PROB
    assert attn(head_dim=264)[0] == UNSUP
    assert attn(tokens=0, q=0, out=0)[0] == OK and attn(hq=0, q=0, out=0)[0] == OK
    assert attn(max_new=0)[0] == PROB
    assert attn(tokens=2 ** 23, hq=4)[0] == PROB
    assert attn(pages=2 ** 27)[0] == PROB
    for kw in (dict(q=0), dict(out=0), dict(k_cache=0), dict(v_cache=0), dict(page_table=0), dict(q_start=0), dict(lens=0)):
        st, msg = attn(**kw)
        assert st == ARG and "null" in msg, kw
    for kw in (dict(q=A + 5 * STEP + 2), dict(out=A + 6 * STEP + 8), dict(v_cache=A + STEP + 4), dict(q_start=A + 3 * STEP + 2)):
        st, msg = attn(**kw)
        assert st == ARG and "aligned" in msg, kw
    assert "out overlaps q" in attn(out=A + 5 * STEP)[1]
    assert "out overlaps k_cache" in attn(out=A + 64)[1]
    assert "out overlaps lens" in attn(lens=A + 6 * STEP + 4)[1]
    L = kaio.lib()
    for kw in (dict(), dict(tokens=600, max_new=600)):
        c = paged()
        need = L.kaio_paged_attention_workspace_size(ctypes.byref(c), kw.get("tokens", 3), 4, kw.get("max_new", 1))
        if need:
            assert "workspace is null" in attn(ws=0, **kw)[1]
            assert "workspace_bytes" in attn(ws_bytes=need - 1, **kw)[1]
            assert "workspace is not 16-byte aligned" in attn(ws=A + 7 * STEP + 4, **kw)[1]
            assert "overlaps" in attn(ws=A + 5 * STEP + 16, **kw)[1]
    assert L.kaio_paged_attention_workspace_size(None, 3, 4, 1) == 0


@no_gpu_only
def test_attention_valid_calls_reach_the_device_check():
    for kw in ({}, dict(dtype=BF16), dict(seqs=0, page_table=0, q_start=0, lens=0), dict(pages=0, k_cache=0, v_cache=0),
               dict(table_width=0, page_table=0), dict(max_new=2 ** 31), dict(head_dim=40), dict(window=2 ** 32 - 1, sinks=2 ** 32 - 1),
               dict(tokens=600, max_new=600), dict(seqs=5000)):
        assert attn(**kw)[0] == DEVICE, (kw, last())


def test_binding_refusals():
    import torch
    h = torch.float16
    cpu = torch.zeros(2, 16, 2, 64, dtype=h)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError, match="no CPU fallback"):
        kaio.KaioPagedKV(cpu, cpu, i(1, 2), i(2), i(1))
    with pytest.raises(ValueError, match="no CPU fallback"):
        kaio.kaio_linear_w4a16(torch.zeros(2, 128, dtype=h), i(16, 8), torch.zeros(1, 8, dtype=h))
    with pytest.raises(TypeError, match="KaioPagedKV"):
        kaio.kaio_paged_attention(torch.zeros(1, 2, 64, dtype=h), None, 1, 1.0)
    with pytest.raises(TypeError, match="float32"):
        kaio.KaioPagedKV(cpu.float(), cpu, i(1, 2), i(2), i(1))


def test_caches_without_heads_columns_or_slots_per_page_are_refused(monkeypatch):
    # nothing may divide by such a size later; a cache of no pages is a cache
    import torch
    monkeypatch.setattr(kaio, "_tensor", lambda t, *a, **k: t)     # (the checks of device and type are not at issue)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for shape in ((2, 0, 2, 64), (2, 16, 0, 64), (2, 16, 2, 0)):
        cache = torch.zeros(shape, dtype=torch.float16)
        with pytest.raises(ValueError, match="at least 1"):
            kaio.KaioPagedKV(cache, cache.clone(), i(1, 2), i(2), i(1))
    cache = torch.zeros(0, 16, 2, 64, dtype=torch.float16)
    assert kaio.KaioPagedKV(cache, cache.clone(), i(1, 2), i(2), i(1)).pages == 0


@pytest.mark.parametrize("kw", [dict(), dict(tokens=600, max_new=600), dict(tokens=600, max_new=600, window=1000, sinks=4),
                                dict(head_dim=128, kv_heads=4, dtype=BF16)])
def test_workspace_refusals_of_calls_that_split_their_keys(kw):
    kw = dict(kw, table_width=300)                              # room for 4800 tokens: keys are split and joined
    need = kaio.lib().kaio_paged_attention_workspace_size(
        ctypes.byref(paged(**{k: v for k, v in kw.items() if k not in ("tokens", "max_new", "window", "sinks")})),
        kw.get("tokens", 3), 4, kw.get("max_new", 1))
    assert need > 0
    for change, msg in ((dict(ws=0, ws_bytes=need), "workspace is null"), (dict(ws=0, ws_bytes=0), "workspace is null"),
                        (dict(ws_bytes=need - 1), f"workspace_bytes ({need - 1}) < {need} needed"),
                        (dict(ws_bytes=0), "workspace_bytes (0)"),
                        (dict(ws=A + 7 * STEP + 4), "workspace is not 16-byte aligned"),
                        (dict(ws=A + 5 * STEP + 16), "workspace overlaps q"),
                        (dict(ws=A + 6 * STEP + 16), "out overlaps workspace"),
                        (dict(ws=A + 16), "workspace overlaps k_cache"), (dict(ws=A + STEP + 16), "workspace overlaps v_cache"),
                        (dict(ws=A + 2 * STEP + 16), "workspace overlaps page_table"),
                        (dict(ws=A + 3 * STEP), "workspace overlaps q_start"), (dict(ws=A + 4 * STEP), "workspace overlaps lens")):
        st, text = attn(**kw, **change)
        assert st == ARG and msg in text, (change, text)


@no_gpu_only
def test_workspace_of_calls_that_split_and_calls_that_do_not():
    c = paged(table_width=4)
    assert kaio.lib().kaio_paged_attention_workspace_size(ctypes.byref(c), 3, 4, 1) == 0
    assert attn(ws=0, ws_bytes=0)[0] == DEVICE                  # no workspace where none is needed
    assert attn(ws=A + 5 * STEP + 4, ws_bytes=0)[0] == DEVICE   # nor are one's address and size looked at
    assert attn(table_width=300)[0] == DEVICE                   # exactly what the query says is enough
    need = kaio.lib().kaio_paged_attention_workspace_size(ctypes.byref(paged(table_width=300)), 3, 4, 1)
    assert attn(table_width=300, ws_bytes=2 * need)[0] == DEVICE


def test_a_window_asks_for_no_more_workspace_than_the_query_says():
    # over many sizes: a call with a window that is refused for its null workspace is one whose query was not 0
    for seqs, tokens, max_new in ((1, 1, 1), (3, 3, 1), (64, 64, 1), (300, 300, 1), (1, 700, 700), (5, 2000, 900), (40, 400, 10)):
        for width in (1, 10, 100, 1000, 20000):
            for window, sinks in ((1, 0), (64, 4), (1000, 0), (5000, 70), (2 ** 31, 2 ** 31), (2 ** 32 - 1, 2 ** 32 - 1)):
                for d, hkv, hq in ((64, 1, 8), (128, 8, 8), (128, 2, 32)):
                    kw = dict(seqs=seqs, tokens=tokens, max_new=max_new, table_width=width, head_dim=d, kv_heads=hkv, hq=hq)
                    need = kaio.lib().kaio_paged_attention_workspace_size(
                        ctypes.byref(paged(seqs=seqs, table_width=width, head_dim=d, kv_heads=hkv)), tokens, hq, max_new)
                    # out = q: the next check after the workspace's size refuses it, on the host
                    st, text = attn(out=A + 5 * STEP, window=window, sinks=sinks, ws=A + 8 * STEP, ws_bytes=need, **kw)
                    assert st == ARG and "out overlaps q" in text, (kw, window, sinks, need, text)
