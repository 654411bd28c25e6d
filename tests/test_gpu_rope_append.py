"""Rotary positions with the write to the paged cache on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from oracle import paged
from tests.gpu_util import DEV
from tests.paged_util import EPS, Batch, f64

pytestmark = pytest.mark.gpu


def run_case(b, sections, interleaved, positions, base=1e4, in_place=False):
    half = sum(sections)
    inv = torch.tensor([base ** (-j / max(half, 1)) for j in range(half)], dtype=torch.float64)
    b.on_gpu()
    k, v = b.k.to(DEV), b.v.to(DEV)
    out = b.dq if in_place else torch.full_like(b.dq, float("nan"))
    got = kaio.kaio_rope_append(b.dq, k, v, positions.to(DEV), inv.to(DEV), sections, b.paged, interleaved=interleaved,
                                q_out=out)
    torch.cuda.synchronize()
    assert got is out
    worst = 0.0
    for name, x, y in (("q", b.q, got), ("k", b.k, None)):
        turned = paged.rotate(f64(x), positions.numpy(), inv.numpy(), sections, interleaved)
        tol = paged.rotate_tolerance(f64(x), turned, sections, interleaved, *EPS[b.dtype])
        if name == "q":
            want, tol, have = turned, tol, f64(y)
        else:
            args = (b.table.numpy(), b.q_start.numpy(), b.lens)
            want = paged.append(f64(b.k_cache), turned, *args)
            tol, have = paged.append(np.zeros(b.k_cache.shape), tol, *args), f64(b.dk)
        err = np.abs(have - want)
        assert (err <= tol).all(), f"{name}: {(err > tol).sum()} of {err.size} outside tolerance"
        worst = max(worst, float((err / np.where(tol > 0, tol, 1)).max()))
    want = paged.append(b.v_cache.view(torch.int16).numpy(), b.v.view(torch.int16).numpy(), b.table.numpy(), b.q_start.numpy(), b.lens)
    assert np.array_equal(b.dv.view(torch.int16).cpu().numpy(), want), "v"
    return worst


def spread(b, axes, far=0):
    pos = torch.tensor([max(0, p) for _, p in paged.rows_of(b.q_start.numpy(), b.lens, b.tokens)])
    return torch.stack([pos + far, pos // 7, pos % 7][:axes]).int()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,sections", [(128, [64]), (64, [32]), (64, [8, 8, 8]), (128, [22, 21, 21]), (64, [16]),
                                        (80, [20]), (72, [5, 6]), (16, [8]), (40, [])])
def test_forms(dtype, interleaved, d, sections):
    b = Batch([1, 5, 0, 30], [40, 5, 3, 77], 6, 2, d, 16, dtype, seed=d)
    axes = max(1, len(sections))
    run_case(b, sections or [0], interleaved, spread(b, axes))


def test_decode_and_wide_heads():
    b = Batch([1] * 4, [900, 31, 16, 1], 32, 32, 128, 16, "f16", seed=1)
    run_case(b, [64], False, spread(b, 1))
    b = Batch([1] * 3, [31, 16, 1], 8, 1, 256, 16, "bf16", seed=2)
    run_case(b, [64, 64], True, spread(b, 2))


def test_many_sequences_and_page_sizes():
    for page in (1, 5, 128):
        lens = [1 + 3 * i % 50 for i in range(130)]
        b = Batch([1] * 130, lens, 2, 1, 64, page, "f16", seed=page)
        run_case(b, [32], False, spread(b, 1))


def test_far_positions():
    # angles of millions of radians keep a 64-bit fraction of a turn
    b = Batch([9], [30], 2, 1, 64, 16, "f16", seed=3)
    run_case(b, [32], False, spread(b, 1, far=2 ** 31 - 1 - 100))


def test_in_place_and_padding_and_missing_pages():
    b = Batch([3, 20], [10, 61], 4, 2, 64, 16, "bf16", seed=4, pad=6)
    b.table[1, 2] = -1            # writes to it are dropped
    b.table[1, 3] = b.pages + 3   # so are those to an id past the last page
    run_case(b, [32], False, spread(b, 1), in_place=True)
    b = Batch([3], [2], 4, 2, 64, 16, "f16", seed=5)      # more new tokens than the length: position -1 has no slot
    run_case(b, [32], True, spread(b, 1))


def test_graph_replays():
    b = Batch([1] * 5, [40, 31, 77, 1, 90], 8, 2, 128, 16, "f16", seed=6)
    b.on_gpu()
    k, v = b.k.to(DEV), b.v.to(DEV)
    inv = torch.tensor([1e4 ** (-j / 64) for j in range(64)], dtype=torch.float64, device=DEV)
    pos = spread(b, 1).to(DEV)
    out = torch.empty_like(b.dq)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kaio.kaio_rope_append(b.dq, k, v, pos, inv, [64], b.paged, q_out=out)
    for i in range(3):
        b.dk.zero_()
        b.paged.lens.copy_(torch.tensor([40 - i, 31, 70 + i, 1, 80 - i], dtype=torch.int32))
        pos.copy_((b.paged.lens - 1).view(1, -1))
        b.dq.mul_(0.5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got, got_k = out.clone(), b.dk.clone()
        b.dk.zero_()
        want = kaio.kaio_rope_append(b.dq, k, v, pos, inv, [64], b.paged)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_k, b.dk)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d,sections,tokens", [(4, 2, 64, [8, 8, 16], 2055), (4, 4, 64, [32], 1031), (2, 1, 16, [8], 2050),
                                                      (1, 1, 40, [8], 3001)])
def test_several_tokens_per_workgroup(hq, hkv, d, sections, tokens, interleaved):
    # more tokens than workgroups, a last workgroup that is not full, sequences that end inside one, slots that are missing
    new = [tokens - 13, 3, 0, 6]
    b = Batch(new, [tokens - 13 + 8, 40, 5, 6], hq, hkv, d, 16, "bf16", seed=tokens, pad=4)
    b.table[0, 5] = -1
    b.table[1, 2] = b.pages
    run_case(b, sections, interleaved, spread(b, len(sections)))


def test_large_offsets():
    # a cache of more than 2^32 bytes: the slots at its far end, with one token and several per workgroup
    page, hkv, d = 64, 8, 128
    pages = (2 ** 32 // (page * hkv * d * 2)) + 60
    k = torch.zeros((pages, page, hkv, d), dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    inv = torch.tensor([1e4 ** (-j / 64) for j in range(64)], dtype=torch.float64, device=DEV)
    for new, hq in ((9, 8), (2050, 8)):
        small = Batch([new], [new + 100], hq, hkv, d, page, "f16", seed=new)
        small.on_gpu()
        dk, dv, pos = small.k.to(DEV), small.v.to(DEV), spread(small, 1).to(DEV)
        far = pages - small.pages
        k[far:].copy_(small.dk)
        v[far:].copy_(small.dv)
        want = kaio.kaio_rope_append(small.dq, dk, dv, pos, inv, [64], small.paged)
        table = torch.where(small.table >= 0, small.table + far, small.table)
        there = kaio.KaioPagedKV(k, v, table.to(DEV), small.paged.q_start, small.paged.lens)
        got = kaio.kaio_rope_append(small.dq, dk, dv, pos, inv, [64], there)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(k[far:], small.dk) and torch.equal(v[far:], small.dv)
    del k, v
