"""W4A16 product with its epilogue on the GPU against the float64 oracle (tolerance: oracle.linear.tolerance)."""
import numpy as np
import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from oracle import linear as ol
from tests.gpu_util import DEV, to_dev, to_host
from tests.linear_forms import SIZES

pytestmark = pytest.mark.gpu


def inputs(m, n, k, seed, bias=True, residual=True):
    r = np.random.default_rng(seed)
    x = r.standard_normal((m, k)).astype(np.float16)
    w = r.integers(0, 2 ** 32, (k // 8, n), dtype=np.uint64).astype(np.uint32)
    s = r.uniform(0.005, 0.02, (k // 128, n)).astype(np.float16)
    b = r.standard_normal(n).astype(np.float16) if bias else None
    res = r.standard_normal((m, n)).astype(np.float16) if residual else None
    return x, w, s, b, res


def run_case(m, n, k, act="none", bias=True, residual=True, seed=0, in_place=False):
    x, w, s, b, res = inputs(m, n, k, seed + m + n, bias, residual)
    dev = lambda a: None if a is None else to_dev(a)
    dres = dev(res)
    y = dres if in_place else torch.full((m, n), float("nan"), dtype=torch.float16, device=DEV)
    got = kaio.kaio_linear_w4a16(to_dev(x), to_dev(w), to_dev(s), bias=dev(b), activation=act, residual=dres, y=y)
    torch.cuda.synchronize()
    assert got is y
    want, z, t = ol.linear(x, w, s, b, act, res)
    tol = ol.tolerance(want, z, t, act, res)
    err = np.abs(to_host(got).astype(np.float64) - want)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} outside tolerance, max ratio {(err / tol).max():.3f}"
    return float((err / tol).max())


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m", [3, 40, 70, 200])
def test_activations(act, m):
    run_case(m, 264, 512, act)
    run_case(m, 132, 384, act, residual=False)


@pytest.mark.parametrize("m", [1, 2, 8, 9, 16, 17, 31, 32, 33, 48, 61, 64, 65, 96, 97, 128, 129, 193, 300])
@pytest.mark.parametrize("n,k", [(64, 512), (100, 384), (77, 640), (260, 1024), (513, 128)])
def test_sizes(m, n, k):
    run_case(m, n, k, "silu", bias=m % 2 == 0, residual=n % 2 == 0)


@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (5, 3, 256), (130, 7, 128), (8, 4096, 4096), (61, 1004, 4096),
                                   (260, 1000, 2688), (1030, 520, 256)])
def test_edges(m, n, k):
    run_case(m, n, k, "gelu_tanh")
    run_case(m, n, k, "none", bias=False, residual=False)


@pytest.mark.parametrize("m", [4, 50, 100, 300])
def test_in_place_residual_and_empty_k(m):
    run_case(m, 136, 256, "gelu", in_place=True)
    run_case(m, 133, 256, "relu", in_place=True)
    x, w, s, b, res = inputs(m, 72, 0, 1)
    y = kaio.kaio_linear_w4a16(to_dev(x), to_dev(w), to_dev(s), bias=to_dev(b), residual=to_dev(res), activation="relu")
    torch.cuda.synchronize()
    want = np.maximum(b.astype(np.float64), 0) + res.astype(np.float64)
    assert (np.abs(to_host(y) - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -23 * 8).all()


@pytest.mark.parametrize("m", [6, 60, 100, 260])
def test_equals_the_projection_without_an_epilogue(m):
    # the same weights through the QKV projection: the same exact products, so within both tolerances
    from oracle import compare
    x, w, s, _, _ = inputs(m, 256, 512, 5)
    q, _, _ = kaio.kaio_qkv_w4a16(*[to_dev(a) for a in (x, w, w, w, s, s, s)])
    y = kaio.kaio_linear_w4a16(to_dev(x), to_dev(w), to_dev(s))
    torch.cuda.synchronize()
    want, _, t = ol.linear(x, w, s)
    assert (np.abs(to_host(y).astype(np.float64) - to_host(q)) <= 2 * compare.qkv_tolerance(want, t)).all()


@pytest.mark.parametrize("m", [4, 40, 100, 300])
def test_special_values(m):
    # infinities and NaN go where the formula takes them, large arguments do not turn into NaN
    x, w, s, b, res = inputs(m, 72, 256, 3)
    x[:] = 0
    b[:8] = [np.inf, -np.inf, np.nan, 60000, -60000, 30, -30, 0]
    res[:] = 0
    res[0, 20], res[0, 21] = np.inf, np.nan
    with np.errstate(all="ignore"):
        for act in ("none", "relu", "gelu", "gelu_tanh", "silu"):
            y = to_host(kaio.kaio_linear_w4a16(to_dev(x), to_dev(w), to_dev(s), bias=to_dev(b), activation=act,
                                               residual=to_dev(res))).astype(np.float64)
            assert y[1, 0] == np.inf and np.isnan(y[1, 2])
            want = ol.ACT[act](b[3:8].astype(np.float64))
            assert (np.abs(y[1, 3:8] - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -24).all()
            assert np.isnan(y[0, 21])
            assert y[0, 20] == np.inf


def test_repeats_streams_and_graphs():
    for m in (5, 40, 100, 300):
        x, w, s, b, res = (to_dev(a) for a in inputs(m, 264, 512, 7))
        ref = kaio.kaio_linear_w4a16(x, w, s, bias=b, activation="silu", residual=res)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out = kaio.kaio_linear_w4a16(x, w, s, bias=b, activation="silu", residual=res)
        side.synchronize()
        assert torch.equal(ref, out)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            kaio.kaio_linear_w4a16(x, w, s, bias=b, activation="silu", residual=res, y=out)
        for i in range(3):
            x.mul_(0.5)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            got = out.clone()
            assert torch.equal(got, kaio.kaio_linear_w4a16(x, w, s, bias=b, activation="silu", residual=res))


@pytest.mark.parametrize("m,n,k", SIZES)
def test_every_form(m, n, k):
    run_case(m, n, k, "gelu_tanh", seed=7)
