"""Rows and channels of larger tensors in the 8-bit product: scales and biases that begin anywhere."""
import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def inputs(m, n, k, dtype=torch.float16):
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    x = torch.randn(m, k, generator=g, device=DEV).to(dtype)
    w = torch.randint(-127, 128, (n, k), generator=g, device=DEV, dtype=torch.int8)
    return x, w, torch.rand(n, generator=g, device=DEV) * 1e-3, torch.randn(n, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("first", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("m", [6, 40, 300])
def test_some_rows_of_a_rounded_batch(m, first):
    x, w, ws, b = inputs(m, 136, 272)
    q, s = kaio.kaio_quantize_rows(x)
    whole = kaio.kaio_linear_w8a8(q, w, ws, x_scale=s, bias=b, activation="silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    part = kaio.kaio_linear_w8a8(q[first:], w, ws, x_scale=s[first:], bias=b, activation="silu")
    other = kaio.kaio_linear_w8a8(q[first:], w, ws, x_scale=s[first:], bias=b, activation="silu", stream=side)
    torch.cuda.synchronize()
    assert torch.equal(whole[first:], part) and torch.equal(part, other)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("first", [1, 3, 8])
@pytest.mark.parametrize("m", [2, 20, 200])
def test_some_channels(m, first, dtype):
    x, w, ws, b = inputs(m, 145, 256, dtype)
    whole = kaio.kaio_linear_w8a8(x, w, ws, bias=b)
    part = kaio.kaio_linear_w8a8(x, w[first:], ws[first:], bias=b[first:])
    torch.cuda.synchronize()
    assert torch.equal(whole[:, first:], part)


@pytest.mark.parametrize("first", [1, 2, 7])
def test_scales_into_some_rows(first):
    x, *_ = inputs(30, 16, 512)
    want_q, want_s = kaio.kaio_quantize_rows(x)
    for stream in (None, torch.cuda.Stream()):
        q, s = torch.zeros_like(want_q), torch.full((31,), -1.0, device=DEV)
        torch.cuda.synchronize()
        out = kaio.kaio_quantize_rows(x[first:], q=q[first:], scale=s[first:30], stream=stream)
        torch.cuda.synchronize()
        assert out[1].data_ptr() == s[first:].data_ptr()
        assert torch.equal(q[first:], want_q[first:]) and torch.equal(s[first:30], want_s[first:])
        assert (s[:first] == -1).all() and s[30] == -1 and not q[:first].any()
    with pytest.raises(ValueError, match="overlaps"):
        kaio.kaio_quantize_rows(x, scale=x.view(torch.float32).view(-1)[1:31])


def test_in_a_graph():
    x, w, ws, b = inputs(21, 72, 256)
    q, s = kaio.kaio_quantize_rows(x)
    out = torch.empty(20, 72, dtype=torch.float16, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kaio.kaio_linear_w8a8(q[1:], w, ws, x_scale=s[1:], bias=b, y=out)
    for _ in range(3):
        s.mul_(0.5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kaio.kaio_linear_w8a8(q[1:], w, ws, x_scale=s[1:], bias=b))
        torch.cuda.synchronize()
