"""Attention over the paged cache on the GPU against the float64 oracle (tolerance: oracle.paged.attention_tolerance)."""
import numpy as np
import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from oracle import paged
from tests.gpu_util import DEV
from tests.paged_util import Batch, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 128), (8, 2, 128), (6, 2, 64), (8, 1, 64), (14, 2, 128), (40, 2, 128)])
def test_decode(dtype, hq, hkv, d):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300]
    b = Batch([1] * len(lens), lens, hq, hkv, d, 16, dtype, seed=d + hq)
    b.check(b.attention())


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 128, 512])
def test_page_sizes(page):
    b = Batch([1, 1, 1], [700, 65, 3], 4, 2, 128, page, "f16", seed=page)
    b.check(b.attention())
    b = Batch([70, 1, 33], [140, 65, 33], 4, 2, 64, page, "bf16", seed=page + 1)
    b.check(b.attention())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (4, 1, 64), (6, 2, 128), (7, 1, 64)])
@pytest.mark.parametrize("new,lens", [([130], [130]), ([1, 64, 17], [200, 64, 81]), ([65, 2], [65, 259]),
                                      ([129, 31, 0, 1], [129, 420, 9, 1])])
def test_chunks(dtype, hq, hkv, d, new, lens):
    b = Batch(new, lens, hq, hkv, d, 16, dtype, seed=sum(new) + hq)
    b.check(b.attention())


def test_long_axis_few_rows():
    # one row over a long axis, and a few rows: the keys of a row are split over workgroups and joined
    for new, hq, hkv in ((1, 2, 1), (3, 4, 2)):
        b = Batch([new], [5003], hq, hkv, 128, 64, "f16", seed=new)
        b.check(b.attention())


def test_many_sequences():
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 60, 150)]
    new = [min(1, x) for x in lens]
    b = Batch(new, lens, 2, 1, 64, 8, "f16", seed=3)
    b.check(b.attention())


def test_many_sequences_unsplit():
    # so many tiles that each is one workgroup's: more sequences than the schedule holds, and many short chunks
    rng = np.random.default_rng(6)
    b = Batch([1] * 1100, [int(x) for x in rng.integers(1, 40, 1100)], 2, 1, 64, 8, "f16", seed=4)
    b.check(b.attention())
    b = Batch([5] * 140, [int(x) for x in rng.integers(5, 150, 140)], 64, 16, 64, 16, "bf16", seed=5, pad=3)
    b.check(b.attention())


@pytest.mark.parametrize("d", [64, 128])
def test_negative_and_zero_scale(d):
    for scale in (-0.1, 0.0):
        for new in ([1, 1], [40, 3]):
            b = Batch(new, [130, 77], 4, 2, d, 16, "f16", seed=11)
            b.scale = scale
            b.check(b.attention())


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (33, 4), (64, 70), (100, 1), (400, 4), (7, 1000)])
@pytest.mark.parametrize("new,lens", [([1, 1, 1, 1], [1, 64, 301, 450]), ([40, 3, 129], [300, 450, 129])])
def test_window_and_sinks(window, sinks, new, lens):
    for d, page in ((64, 16), (128, 8)):
        b = Batch(new, lens, 4, 2, d, page, "f16", seed=window + sinks, window=window, sinks=sinks)
        b.check(b.attention())


@pytest.mark.parametrize("d", [8, 40, 80, 96, 256])
def test_other_head_dims(d):
    b = Batch([1, 5], [70, 133], 4, 2, d, 16, "f16", seed=d)
    b.check(b.attention())


def test_rows_that_see_nothing_and_padding():
    # a sequence whose every page is gone, one with new tokens but length 0, rows past the last sequence
    for new in ([1, 1, 1], [40, 30, 50]):
        b = Batch(new, [60, 70, 50], 4, 2, 64, 16, "f16", seed=9, pad=5)
        b.table[1] = -1
        b.lens[2] = 0
        out = b.attention()
        b.check(out)
        y = f64(out)
        assert not y[new[0]:].any()


def test_pages_gone_in_the_middle_and_bad_ids():
    for new in ([1], [50]):
        b = Batch(new, [333], 4, 2, 128, 16, "bf16", seed=2)
        b.table[0, 3] = -1
        b.table[0, 7] = b.pages          # one past the last page: not there
        b.table[0, 8] = -2 ** 31
        b.check(b.attention())


@pytest.mark.parametrize("new", [1, 3, 90])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_invisible_slots_hold_does_not_matter(new, bad):
    # slots past the length, released pages and slots of no sequence hold NaN or infinities
    b = Batch([new, new], [203, 90], 4, 2, 64, 16, "f16", seed=4, window=50, sinks=3)
    ref = b.attention()
    b.check(ref)
    hide = ~b.used()
    for c in (b.k_cache, b.v_cache):
        c.view(-1, *c.shape[2:])[hide] = bad
    out = b.attention()
    assert torch.equal(ref, out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_masked_token_does_not_reach_the_rows_before_it(d, bad):
    # token 37's K and V are not finite: rows before it are as without it, and rows past its window too
    b = Batch([100], [100], 4, 2, d, 16, "f16", seed=6, window=20, sinks=2)
    ref = f64(b.attention())
    for c in (b.k_cache, b.v_cache):
        c[b.table[0, 37 // 16], 37 % 16] = bad
    out = f64(b.attention())
    ok = [t for t in range(100) if t < 37 or t >= 57]
    assert np.array_equal(out[ok], ref[ok])
    assert not np.isfinite(out[37:57]).any()


def test_visible_infinities_follow_the_formula():
    b = Batch([1], [40], 1, 1, 64, 16, "f16", seed=8)
    b.v_cache[b.table[0, 1], 2, 0, 5] = float("inf")
    b.v_cache[b.table[0, 0], 3, 0, 6] = float("nan")
    out = f64(b.attention())[0, 0]
    assert out[5] == np.inf and np.isnan(out[6]) and np.isfinite(np.delete(out, [5, 6])).all()
    # scores of minus infinity weigh nothing
    b = Batch([1], [40], 1, 1, 64, 16, "f16", seed=8)
    b.q[0, 0, 0] = 1.0
    b.k_cache[b.table[0, 2], 1, 0, 0] = -float("inf")
    b.check(b.attention())


def test_lowest_values():
    # the type's lowest value in K: scores far below the others, weights zero, nothing overflows to NaN
    b = Batch([1, 40], [50, 77], 2, 1, 64, 16, "f16", seed=12)
    b.q[:, :, 0] = 1.0
    b.k_cache[b.table[0, 1], 3, 0, 0] = -65504.0
    b.k_cache[b.table[1, 1], 3, 0, 0] = -65504.0
    b.check(b.attention())


def test_growing_scores():
    # scores that rise along the axis: the running maximum moves at every block
    b = Batch([1, 64], [900, 700], 2, 1, 64, 16, "f16", seed=13)
    b.q.fill_(1.0)
    for s in range(2):
        for c in range(b.lens[s]):
            b.k_cache[b.table[s, c // 16], c % 16] = c / 16.0
    b.scale = 1.0 / 8
    b.check(b.attention())


def test_max_new_is_only_a_hint():
    b = Batch([1, 40, 3], [60, 70, 200], 4, 2, 128, 16, "f16", seed=14)
    b.check(b.attention())
    for hint in (1, 2, 1000):
        out = torch.full_like(b.dq, float("nan"))
        kaio.kaio_paged_attention(b.dq, b.paged, hint, b.scale, out=out)
        torch.cuda.synchronize()
        b.check(out)


def test_empty_batches():
    b = Batch([], [], 4, 2, 64, 16, "f16", pad=3)
    out = b.attention()
    assert not out.any()
    assert kaio.kaio_paged_attention(b.dq[:0], b.paged, 1, 1.0).shape == (0, 4, 64)


def test_repeats_are_bit_equal_and_inputs_untouched():
    b = Batch([1, 1, 1, 90], [900, 31, 77, 400], 8, 2, 128, 16, "bf16", seed=15)
    a = b.attention()
    keep = [t.clone() for t in (b.dq, b.dk, b.dv)]
    for _ in range(3):
        out = torch.empty_like(a)
        kaio.kaio_paged_attention(b.dq, b.paged, 90, b.scale, out=out)
        torch.cuda.synchronize()
        assert torch.equal(a, out)
    assert all(torch.equal(x, y) for x, y in zip(keep, (b.dq, b.dk, b.dv)))


def test_side_stream_and_graph_replays():
    b = Batch([1] * 5, [400, 31, 77, 1, 900], 8, 2, 128, 16, "f16", seed=16)
    ref = b.attention()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = kaio.kaio_paged_attention(b.dq, b.paged, 1, b.scale)
    side.synchronize()
    assert torch.equal(ref, out)
    out = kaio.kaio_paged_attention(b.dq, b.paged, 1, b.scale, stream=side)   # allocated here, used there
    side.synchronize()
    assert torch.equal(ref, out)
    need = kaio.lib().kaio_paged_attention_workspace_size(b.paged._ref, 5, 8, 1)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kaio.kaio_paged_attention(b.dq, b.paged, 1, b.scale, out=out, workspace=ws)
    for i in range(3):          # lengths change between replays, in place
        b.lens = [400 - i, 31 + i, 60, 1, 900 - 100 * i]
        b.paged.lens.copy_(torch.tensor(b.lens, dtype=torch.int32))
        b.dq.normal_(generator=torch.Generator(device=DEV).manual_seed(i))
        b.q = b.dq.cpu()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.check(out)
        eager = kaio.kaio_paged_attention(b.dq, b.paged, 1, b.scale)
        torch.cuda.synchronize()
        assert torch.equal(eager, out)


def test_large_offsets():
    # a cache of more than 2^32 bytes: the sequence's pages at its far end
    page, hkv, d = 64, 8, 128
    pages = (2 ** 32 // (page * hkv * d * 2)) + 40
    small = Batch([1], [200], 8, hkv, d, page, "f16", seed=17)
    ref = small.attention()
    k = torch.empty((pages, page, hkv, d), dtype=torch.float16, device=DEV)
    v = torch.empty_like(k)
    far = pages - small.pages
    k[far:].copy_(small.dk)
    v[far:].copy_(small.dv)
    table = torch.where(small.table >= 0, small.table + far, small.table)
    paged = kaio.KaioPagedKV(k, v, table.to(DEV), small.q_start.to(DEV), torch.tensor([200], dtype=torch.int32, device=DEV))
    out = kaio.kaio_paged_attention(small.dq, paged, 1, small.scale)
    torch.cuda.synchronize()
    assert torch.equal(ref, out)
    del k, v


@pytest.mark.parametrize("new,heads", [(90, 8), (200, 8)])
def test_large_offsets_of_chunks(new, heads):
    # a cache of more than 2^32 bytes under tiles of many rows
    page, hkv, d = 64, 8, 128
    pages = (2 ** 32 // (page * hkv * d * 2)) + 40
    small = Batch([new], [300], heads, hkv, d, page, "f16", seed=new)
    small.check(small.attention())
    k = torch.zeros((pages, page, hkv, d), dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    far = pages - small.pages
    k[far:].copy_(small.dk)
    v[far:].copy_(small.dv)
    table = torch.where(small.table >= 0, small.table + far, small.table)
    paged = kaio.KaioPagedKV(k, v, table.to(DEV), small.q_start.to(DEV), torch.tensor([300], dtype=torch.int32, device=DEV))
    out = kaio.kaio_paged_attention(small.dq, paged, new, small.scale)
    torch.cuda.synchronize()
    small.check(out)
    del k, v


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 2, 3, 5, 12, 20])
def test_page_sizes_of_chunks(page, d):
    # pages that end anywhere in a tile, for tiles of many rows, with a window
    b = Batch([70, 1, 33], [240, 65, 33], 4, 2, d, page, "bf16", seed=page + d)
    b.check(b.attention())
    b = Batch([45, 140], [400, 333], 6, 2, d, page, "f16", seed=page, window=50, sinks=5)
    b.check(b.attention())


@pytest.mark.parametrize("page", [3, 16])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("bad", [float("nan"), -float("inf")])
def test_what_invisible_slots_hold_does_not_matter_at_128(page, new, bad):
    b = Batch([new, new], [203, 90], 4, 2, 128, page, "bf16", seed=4, window=50, sinks=3)
    ref = b.attention()
    b.check(ref)
    hide = ~b.used()
    for c in (b.k_cache, b.v_cache):
        c.view(-1, *c.shape[2:])[hide] = bad
    assert torch.equal(ref, b.attention())


def test_tensors_that_are_not_contiguous_and_the_checked_path():
    # an explicit stream takes the wrapper's checked path: the same bits; strided views of q are refused
    b = Batch([1, 9], [70, 40], 8, 2, 128, 16, "f16", seed=21)
    ref = b.attention()
    for out in (kaio.kaio_paged_attention(b.dq, b.paged, 9, b.scale),
                kaio.kaio_paged_attention(b.dq, b.paged, 9, b.scale, stream=torch.cuda.current_stream())):
        torch.cuda.synchronize()
        assert torch.equal(ref, out)
    wide = torch.cat([b.dq, b.dq], 1)
    with pytest.raises(ValueError, match="contiguous"):
        kaio.kaio_paged_attention(wide[:, ::2], b.paged, 9, b.scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_a_long_tail_of_small_weights_counts(new, dtype, d):
    # one key of weight 1 and V = 0, thousands of weight 2^-20.4 and V = 1: their mean is all of the result.  Weights
    # that small keep their bits: half a step for each weight and half a step for the output
    b = Batch([new], [3000], 2, 1, d, 64, dtype, seed=22)
    b.q.zero_()
    b.q[:, :, 0] = 1.0
    b.k_cache.zero_()
    b.k_cache[..., 0] = -20.4
    b.v_cache.fill_(1.0)
    first = b.table[0, 0]
    b.k_cache[first, 0, :, 0] = 0.0
    b.v_cache[first, 0] = 0.0
    b.scale = float(np.log(2.0))
    out = f64(b.attention())
    w = 2.0 ** f64(b.k_cache[first, 1, 0, :1])[0]
    seen = np.arange(3000 - new, 3000)                  # keys of small weight each row sees
    want = (seen * w / (1 + seen * w))[:, None, None]
    half = 2.0 ** -11 if dtype == "f16" else 2.0 ** -8
    assert (np.abs(out - want) <= 2 * half * 1.01 * want).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("size", [1e3, 1e5, 3e6, 2e7])
def test_large_equal_scores_weigh_alike(size, new, dtype, d):
    # every key has the same score, far from zero on either side: the result is the mean of V over what the row sees.
    # Equal scores give equal weights, whatever f32's steps at that size are: half a step of the output, half a step of
    # the mean (weights that do not round alike in value but alike for all), and the sums' 2 n roundings
    for sign in (1.0, -1.0):
        b = Batch([new], [300], 2, 1, d, 16, dtype, seed=23)
        b.q.zero_()
        b.q[:, :, 0] = 1.0
        b.k_cache.zero_()
        b.k_cache[..., 0] = sign * 1000.0
        b.scale = size / 1000.0
        y, terms = paged.attention(f64(b.q), f64(b.k_cache), f64(b.v_cache), b.table.numpy(), b.q_start.numpy(), b.lens,
                                   b.scale)
        eps, low = (2.0 ** -10, 2.0 ** -14) if dtype == "f16" else (2.0 ** -7, 2.0 ** -126)
        tol = eps / 2 * np.abs(y) + (eps / 2 + 2 * 308 * 2.0 ** -24) * terms[0] + eps * low / 2 * 301
        assert (np.abs(f64(b.attention()) - y) <= tol).all()


@pytest.mark.parametrize("extra", [1, 700])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (6, 2, 64), (8, 1, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
@pytest.mark.parametrize("new,lens", [([1, 1, 1], [300, 65, 1]), ([130], [333]), ([70, 1, 40, 0], [190, 64, 301, 20])])
def test_narrow_and_wide_tables(new, lens, hq, hkv, d, window, sinks, extra):
    # a table with room for much longer sequences splits the keys of a tile over workgroups, a narrow one does not
    b = Batch(new, lens, hq, hkv, d, 16, "f16", seed=extra + hq, window=window, sinks=sinks, pad=2, extra_width=extra)
    b.check(b.attention())


def test_a_window_needs_no_more_workspace():
    # the workspace is asked for without the window: a call with one takes it
    import ctypes
    from tests.test_paged_host import paged as cache
    size = kaio.lib().kaio_paged_attention_workspace_size
    b = Batch([1, 1], [900, 700], 8, 2, 128, 16, "f16", seed=24, window=64, sinks=2, extra_width=50)
    b.on_gpu()
    need = size(b.paged._ref, 2, 8, 1)
    assert need > 0 and size(ctypes.byref(cache(table_width=4)), 3, 4, 1) == 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    b.check(b.attention(workspace=ws))


def test_a_cache_without_heads_goes_to_the_checks():
    # the short call path must leave it to them (and not divide by its heads)
    import ctypes
    from tests.test_paged_host import paged as cache
    q = torch.zeros(3, 4, 64, dtype=torch.float16, device=DEV)
    c = cache(kv_heads=0)
    assert kaio._quick().attention(q, ctypes.addressof(c), q.device.index, 1, 1.0, 0, 0, None, None) is None
    st = kaio.lib().kaio_paged_attention(ctypes.byref(c), q.data_ptr(), q.data_ptr(), 3, 4, 1, 1.0, 0, 0, None, 0, None)
    assert st == 2 and "kv_heads" in kaio.kaio_last_error()      # INVALID_PROBLEM


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("new,lens,extra", [([100, 3], [100, 90], 1), ([70, 40], [330, 61], 700), ([1, 2], [90, 61], 1)])
def test_visible_non_finite_values_show_whatever_their_weight(new, lens, extra, bad, dtype, d):
    # token 37's score is 60 under the others', a weight that 16 bits may round to zero, and one column of its V is not
    # finite: every row that sees it must say so, no other row and no other column may
    b = Batch(new, lens, 4, 2, d, 16, dtype, seed=25, extra_width=extra)
    b.q.zero_()
    b.q[:, :, 0] = 1.0
    b.k_cache.zero_()
    b.scale = 1.0
    for s in range(2):
        at = b.table[s, 37 // 16], 37 % 16
        b.k_cache[at][:, 0] = -60.0
        b.v_cache[at][:, 5] = bad
    out = f64(b.attention())
    rows = paged.rows_of(b.q_start.numpy(), b.lens, b.tokens)
    sees = np.array([pos >= 37 for _, pos in rows])
    assert np.isfinite(out[~sees]).all() and np.isfinite(np.delete(out, 5, axis=2)).all()
    hit = out[sees][:, :, 5]
    assert np.isnan(hit).all() if np.isnan(bad) else not np.isfinite(hit).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("length,extra", [(64, 1), (1500, 700)])
def test_the_weights_used_add_up_to_one(length, extra, new, dtype, d):
    # weights a little under half a step of the 16-bit type above a power of two, all rounded the same way, and V = 1:
    # the weights that multiply V are those that are summed, so the result is 1 but for 2 n f32 roundings, which is 1
    # in 16 bits (2 * 1500 * 2^-24 is under 2^-12, half a step under 1 of f16)
    b = Batch([new], [length], 2, 1, d, 16, dtype, seed=26, extra_width=extra)
    b.q.zero_()
    b.q[:, :, :2] = 1.0
    b.k_cache.zero_()
    b.k_cache[..., 0] = -3.0
    b.k_cache[..., 1] = float(np.log2(1 + 0.9 * 2.0 ** (-11 if dtype == "f16" else -8)))
    for t in range(0, length, 32):                      # a key of weight 1 in whatever part of the keys has its own maximum
        b.k_cache[b.table[0, t // 16], t % 16, :, :2] = 0.0
    b.v_cache.fill_(1.0)
    b.scale = float(np.log(2.0))
    out = b.attention()
    assert torch.equal(out, torch.ones_like(out))
