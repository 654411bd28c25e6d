"""Attention whose keys are split over workgroups and joined, against the float64 oracle.

What the host knows of a call decides whether it splits: the sizes, the page table's width and the window.  Every batch
here has a table with room for much longer sequences (or a long window), and every call is shown to be a split one.
(Tolerance: oracle.paged.attention_tolerance, as for calls that are not split.)
"""
import numpy as np
import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from oracle import paged
from tests.gpu_util import DEV
from tests.paged_util import EPS, Batch, f64

pytestmark = pytest.mark.gpu

WIDE = 8192      # tokens of room in a table: past the 64 blocks (of 64 keys) up to which a prompt's tile stays whole


def wide(page):
    return -(-WIDE // page)


def splits(b, max_new=None):
    """Whether the call that Batch.attention makes needs a workspace, which only a split call does."""
    q = b.dq
    st = kaio.lib().kaio_paged_attention(b.paged._ref, q.data_ptr(), torch.empty_like(q).data_ptr(), q.shape[0], q.shape[1],
                                         max_new or max(max(b.new, default=1), 1), b.scale, b.window, b.sinks, None, 0,
                                         torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return st == 1 and "workspace is null" in kaio.kaio_last_error()


def attention(b, **kw):
    b.on_gpu()
    assert splits(b)
    return b.attention(**kw)


@pytest.mark.parametrize("seqs", [2, 64, 65, 130, 255])
@pytest.mark.parametrize("dtype,hq,hkv,d,page", [("f16", 2, 1, 64, 8), ("bf16", 4, 2, 128, 16), ("f16", 3, 1, 128, 5)])
def test_decode_batches(seqs, dtype, hq, hkv, d, page):
    # lengths that differ much, sequences without new tokens, empty ones: the line of blocks in registers (up to 64
    # sequences) and in LDS, cut anywhere
    rng = np.random.default_rng(seqs)
    lens = [int(x) for x in rng.integers(0, 90, seqs)]
    lens[seqs // 2], lens[-1] = 1500, 700
    new = [1 if x and i % 11 != 5 else 0 for i, x in enumerate(lens)]
    b = Batch(new, lens, hq, hkv, d, page, dtype, seed=seqs, pad=3, extra_width=wide(page))
    b.check(attention(b))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 128), (8, 2, 128), (6, 2, 64), (8, 1, 64), (14, 2, 128), (40, 2, 128)])
def test_decode_lengths(dtype, hq, hkv, d):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300]
    b = Batch([1] * len(lens), lens, hq, hkv, d, 16, dtype, seed=d + hq, extra_width=wide(16))
    b.check(attention(b))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (4, 1, 64), (6, 2, 128), (7, 1, 64)])
@pytest.mark.parametrize("new,lens", [([130], [130]), ([1, 64, 17], [200, 64, 81]), ([65, 2], [65, 1259]),
                                      ([129, 31, 0, 1], [129, 420, 9, 1])])
def test_chunks(dtype, hq, hkv, d, new, lens):
    b = Batch(new, lens, hq, hkv, d, 16, dtype, seed=sum(new) + hq, extra_width=wide(16))
    b.check(attention(b))


def test_many_chunks():
    # more sequences than a wave has lanes, more tiles than sequences
    rng = np.random.default_rng(6)
    b = Batch([5] * 70 + [40, 90], [int(x) for x in rng.integers(5, 150, 70)] + [300, 90], 8, 2, 64, 16, "bf16", seed=5, pad=3,
              extra_width=wide(16))
    b.check(attention(b))


@pytest.mark.parametrize("page", [1, 2, 3, 5, 8, 12, 20, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_page_sizes(page, d):
    for new, lens in (([70, 1, 33], [240, 65, 533]), ([1, 1, 1], [700, 65, 3])):
        b = Batch(new, lens, 4, 2, d, page, "bf16", seed=page + d, extra_width=wide(page))
        b.check(attention(b))


@pytest.mark.parametrize("page", [3, 16])
@pytest.mark.parametrize("window,sinks", [(400, 0), (500, 4), (420, 70), (900, 300)])
@pytest.mark.parametrize("d", [64, 128])
def test_windows_of_decode(d, window, sinks, page):
    b = Batch([1] * 5, [2500, 64, 301, 450, 1200], 6, 2, d, page, "f16", seed=window + sinks, window=window, sinks=sinks,
              extra_width=wide(page))
    b.check(attention(b))


@pytest.mark.parametrize("page", [3, 16])
@pytest.mark.parametrize("d,window", [(64, 1200), (128, 900)])
@pytest.mark.parametrize("sinks", [0, 4, 70, 200])
@pytest.mark.parametrize("new,lens", [([70, 40], [2500, 1300]), ([33], [1500])])
def test_windows_of_chunks(new, lens, sinks, d, window, page):
    # sinks' blocks, then the window's, cut into pieces anywhere; pages between them are gone
    b = Batch(new, lens, 4, 2, d, page, "f16", seed=window + sinks, window=window, sinks=sinks, extra_width=wide(page))
    assert (b.table[0, :-(-lens[0] // page)] < 0).any()
    b.check(attention(b))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 30, 50]])
def test_rows_that_see_nothing_and_padding(new, d):
    b = Batch(new, [960, 700, 50], 4, 2, d, 16, "f16", seed=9, pad=5, extra_width=wide(16))
    b.table[1] = -1
    b.lens[2] = 0
    out = attention(b)
    b.check(out)
    assert not f64(out)[new[0]:].any()


@pytest.mark.parametrize("page", [3, 16])
@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("d", [64, 128])
def test_pages_gone_in_the_middle_and_bad_ids(d, new, page):
    # single pages, a whole block's, and from one block into the next
    b = Batch([new], [1333], 4, 2, d, page, "bf16", seed=2, extra_width=wide(page))
    b.table[0, 3] = -1
    b.table[0, 7] = b.pages
    b.table[0, 8] = -2 ** 31
    b.table[0, 128 // page:256 // page] = -1
    b.table[0, 600 // page:680 // page] = b.pages + 9
    b.check(attention(b))


@pytest.mark.parametrize("page", [3, 16])
@pytest.mark.parametrize("new", [1, 3, 90])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1200, 3)])
def test_what_invisible_slots_hold_does_not_matter(window, sinks, bad, d, new, page):
    b = Batch([new, new], [1703, 90], 4, 2, d, page, "f16", seed=4, window=window, sinks=sinks, extra_width=wide(page))
    ref = attention(b)
    b.check(ref)
    hide = ~b.used()
    assert hide.any()
    for c in (b.k_cache, b.v_cache):
        c.view(-1, *c.shape[2:])[hide] = bad
    assert torch.equal(ref, attention(b))


@pytest.mark.parametrize("d,window", [(64, 1200), (128, 900)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_masked_token_does_not_reach_the_rows_that_do_not_see_it(d, window, bad):
    # two tokens are not finite: one that the first rows see and the window then leaves behind, one among the new ones
    length, new = 1500, 100
    at = [length - new - window + 40, length - new + 57]      # rows 40 to 56 see neither
    b = Batch([new], [length], 4, 2, d, 16, "f16", seed=6, window=window, sinks=2, extra_width=wide(16))
    ref = f64(attention(b))
    for t in at:
        for c in (b.k_cache, b.v_cache):
            c[b.table[0, t // 16], t % 16] = bad
    out = f64(attention(b))
    pos = np.arange(length - new, length)
    hit = np.any([(pos >= t) & (t > pos - window) for t in at], axis=0)
    assert hit.any() and not hit.all()
    assert np.array_equal(out[~hit], ref[~hit])
    assert not np.isfinite(out[hit]).any()


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_growing_and_falling_scores(new, d):
    # pieces whose maxima differ by far: the first ones, or the last, weigh nothing in the end
    for sign in (1.0, -1.0):
        b = Batch([new, new], [1900, 700], 2, 1, d, 16, "f16", seed=13, extra_width=wide(16))
        b.q.fill_(1.0)
        for s in range(2):
            for c in range(b.lens[s]):
                b.k_cache[b.table[s, c // 16], c % 16] = sign * c / 16.0
        b.scale = 1.0 / 8
        b.check(attention(b))


@pytest.mark.parametrize("new", [1, 40])
def test_lowest_values(new):
    b = Batch([new, new], [1050, 77], 2, 1, 64, 16, "f16", seed=12, extra_width=wide(16))
    b.q[:, :, 0] = 1.0
    for s, t in ((0, 19), (0, 600), (1, 19)):
        b.k_cache[b.table[s, t // 16], t % 16, 0, 0] = -65504.0
    b.check(attention(b))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_large_equal_scores_weigh_alike(new, dtype, d):
    # (the bound of the same test of calls that are not split, with this one's number of keys)
    for size in (1e5, -2e7):
        b = Batch([new], [900], 2, 1, d, 16, dtype, seed=23, extra_width=wide(16))
        b.q.zero_()
        b.q[:, :, 0] = 1.0
        b.k_cache.zero_()
        b.k_cache[..., 0] = float(np.copysign(1000.0, size))
        b.scale = abs(size) / 1000.0
        y, terms = paged.attention(f64(b.q), f64(b.k_cache), f64(b.v_cache), b.table.numpy(), b.q_start.numpy(), b.lens,
                                   b.scale)
        eps, low = EPS[dtype]
        tol = eps / 2 * np.abs(y) + (eps / 2 + 2 * 908 * 2.0 ** -24) * terms[0] + eps * low / 2 * 901
        assert (np.abs(f64(attention(b)) - y) <= tol).all()


@pytest.mark.parametrize("d", [64, 128])
def test_negative_and_zero_scale(d):
    for scale in (-0.1, 0.0):
        for new in ([1, 1], [40, 3]):
            b = Batch(new, [1130, 77], 4, 2, d, 16, "f16", seed=11, extra_width=wide(16))
            b.scale = scale
            b.check(attention(b))


def test_max_new_is_only_a_hint():
    # tiles of few rows for a sequence of many, and the other way round
    b = Batch([1, 40, 3], [60, 70, 1200], 4, 2, 128, 16, "f16", seed=14, extra_width=wide(16))
    b.check(attention(b))
    for hint in (1, 2, 1000):
        assert splits(b, hint)
        out = torch.full_like(b.dq, float("nan"))
        kaio.kaio_paged_attention(b.dq, b.paged, hint, b.scale, out=out)
        torch.cuda.synchronize()
        b.check(out)


@pytest.mark.parametrize("new", [90, 200])
def test_large_offsets(new):
    # a cache of more than 2^32 bytes: a load per key, its slots at the far end
    page, hkv, d = 64, 8, 128
    pages = (2 ** 32 // (page * hkv * d * 2)) + 40
    small = Batch([new], [700], hkv, hkv, d, page, "f16", seed=new, extra_width=wide(page))
    small.check(attention(small))
    k = torch.zeros((pages, page, hkv, d), dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    far = pages - small.pages
    k[far:].copy_(small.dk)
    v[far:].copy_(small.dv)
    table = torch.where(small.table >= 0, small.table + far, small.table)
    small.paged = kaio.KaioPagedKV(k, v, table.to(DEV), small.q_start.to(DEV),
                                   torch.tensor([700], dtype=torch.int32, device=DEV))
    assert splits(small)
    out = kaio.kaio_paged_attention(small.dq, small.paged, new, small.scale)
    torch.cuda.synchronize()
    small.check(out)


@pytest.mark.parametrize("new,window,sinks", [([1] * 70, 0, 0), ([60, 1, 33], 0, 0), ([60, 1, 33], 1000, 4)])
def test_graph_replays_and_used_workspaces(new, window, sinks):
    # lengths change in place between replays, the workspace holds anything before each, eager calls run in between
    lens = [1400 if i == 1 else 20 + 7 * i % 100 + n for i, n in enumerate(new)]
    b = Batch(new, lens, 8, 2, 128, 16, "f16", seed=16, window=window, sinks=sinks, extra_width=wide(16), release=False)
    b.on_gpu()
    assert splits(b)
    need = kaio.lib().kaio_paged_attention_workspace_size(b.paged._ref, b.tokens, 8, max(new))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(b.dq)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kaio.kaio_paged_attention(b.dq, b.paged, max(new), b.scale, window=window, sinks=sinks, out=out, workspace=ws)
    for i in range(3):
        b.lens = [max(n, x - 150 * i) for n, x in zip(new, lens)]
        b.paged.lens.copy_(torch.tensor(b.lens, dtype=torch.int32))
        b.dq.normal_(generator=torch.Generator(device=DEV).manual_seed(i))
        b.q = b.dq.cpu()
        ws.fill_(0x7F if i else 0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.check(out)
        eager = kaio.kaio_paged_attention(b.dq, b.paged, max(new), b.scale, window=window, sinks=sinks)
        torch.cuda.synchronize()
        assert torch.equal(eager, out)


def test_as_many_sequences_as_the_schedule_holds():
    # 512 tiles, most of sequences without new tokens
    new = [1 if i in (0, 3, 64, 65, 300, 510, 511) else 0 for i in range(512)]
    lens = [1200 if i == 65 else 90 if n else i % 3 for i, n in enumerate(new)]
    b = Batch(new, lens, 2, 2, 64, 16, "f16", seed=30, pad=2, extra_width=wide(16))
    b.check(attention(b))


@pytest.mark.parametrize("extra", [1, wide(16)])
@pytest.mark.parametrize("d", [64, 128, 80])
@pytest.mark.parametrize("new", [[1, 1], [50, 3]])
def test_rows_before_the_first_sequence(new, d, extra):
    # q_start need not begin at 0: rows before it see nothing, whole tables or wide ones, whatever the form
    lead = 5
    b = Batch(new, [300, 77], 4, 2, d, 16, "f16", seed=31, pad=lead + 3, extra_width=extra)
    b.q_start += lead
    b.on_gpu()
    assert splits(b) == (extra > 1 and d != 80)
    out = b.attention()
    b.check(out)
    y = f64(out)
    assert not y[:lead].any() and not y[-3:].any() and y[lead:-3].any()
