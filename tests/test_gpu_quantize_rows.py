"""Rows rounded to 8 bits on the GPU against the oracle: whole numbers and scales are equal, bit for bit."""
import numpy as np
import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from oracle import linear8 as ol
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


def check(x):
    """x: a CPU tensor"""
    q = torch.full(x.shape, 77, dtype=torch.int8, device=DEV)
    s = torch.full(x.shape[:1], -1.0, device=DEV)
    got = kaio.kaio_quantize_rows(x.to(DEV), q=q, scale=s)
    torch.cuda.synchronize()
    assert got[0] is q and got[1] is s
    want_q, want_s = ol.quantize(x.double().numpy())
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,k", [(1, 16), (3, 32), (4, 1024), (5, 1008), (7, 1040), (2, 4096), (9, 4112), (3, 8192), (2, 8208), (3, 16384),
                                 (2, 16400), (2, 32768), (1, 32784), (1, 40000), (1000, 48), (257, 2064)])
def test_sizes(dtype, m, k):
    g = torch.Generator().manual_seed(m + k)
    check((torch.randn(m, k, generator=g) * torch.rand(m, 1, generator=g) * 4).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_every_number(dtype):
    # all finite numbers of the type, each below every kind of largest value: ties and steps near them, far exponents
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    finite = bits[torch.isfinite(bits.float())]
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        x = finite[torch.randperm(len(finite), generator=g)][:len(finite) // 4096 * 4096].view(-1, 64)
        check(x)
    order = finite[finite.float().abs().argsort()]
    check(order[:len(order) // 32 * 32].view(-1, 32))      # neighbours of like size


@pytest.mark.parametrize("dtype", TYPES)
def test_ties(dtype):
    # 127 x / a is n + 1/2 exactly for a = 127 * 2^e and x an odd multiple of 2^(e - 1)
    rows = []
    for e in (-3, 0, 1, 4):
        row = (torch.arange(64, dtype=torch.float64) - 32) * 2 + 1
        row = row[row.abs() < 127] / 2
        row = torch.cat([row, torch.tensor([127.0]), torch.zeros(127)])[:64] * 2.0 ** e
        row[-1] = 127 * 2.0 ** e
        rows.append(row)
    check(torch.stack(rows).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", [32, 4096, 20000])
def test_special_rows(dtype, k):
    g = torch.Generator().manual_seed(k)
    x = torch.randn(8, k, generator=g).to(dtype)
    x[1] = 0
    x[2, k // 2] = float("inf")
    x[3, k - 1] = float("nan")
    x[4] = -0.0
    x[5, 3] = -float("inf")
    x[6] = 0
    x[6, 5] = torch.finfo(dtype).smallest_normal
    x[7, 0] = -torch.finfo(dtype).max
    check(x)


def test_streams_graphs_offsets_and_empty():
    x = torch.randn(40, 512, device=DEV).half()
    ref = kaio.kaio_quantize_rows(x)
    part = kaio.kaio_quantize_rows(x[8:24])             # rows of a larger tensor
    torch.cuda.synchronize()
    assert torch.equal(part[0], ref[0][8:24]) and torch.equal(part[1], ref[1][8:24])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = kaio.kaio_quantize_rows(x, stream=side)
    side.synchronize()
    assert torch.equal(other[0], ref[0]) and torch.equal(other[1], ref[1])
    q, s = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kaio.kaio_quantize_rows(x, q=q, scale=s)
    for _ in range(3):
        x.mul_(0.7)
        g.replay()
        torch.cuda.synchronize()
        again = kaio.kaio_quantize_rows(x)
        assert torch.equal(again[0], q) and torch.equal(again[1], s)
    q, s = kaio.kaio_quantize_rows(x[:0])
    assert q.shape == (0, 512) and s.shape == (0,)
    q, s = kaio.kaio_quantize_rows(x[:, :0].contiguous())
    torch.cuda.synchronize()
    assert q.shape == (40, 0) and not s.any()


def test_refusals():
    x = torch.randn(4, 64, device=DEV).half()
    for bad in (x.float(), x.t(), x[:, :40], x[0], x[:, 8:40]):
        with pytest.raises((TypeError, ValueError)):
            kaio.kaio_quantize_rows(bad)
    with pytest.raises(ValueError):
        kaio.kaio_quantize_rows(x[:, :24].contiguous())
    with pytest.raises(ValueError):
        kaio.kaio_quantize_rows(x, q=torch.empty(4, 32, dtype=torch.int8, device=DEV))
    with pytest.raises(TypeError):
        kaio.kaio_quantize_rows(x, scale=torch.empty(4, dtype=torch.float16, device=DEV))
    with pytest.raises(kaio.KaioError):
        kaio.kaio_quantize_rows(x, q=x.view(torch.int8).view(-1)[:256].view(4, 64))
