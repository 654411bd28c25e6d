"""Pins of the oracles of the 8-bit product and of the mixture of experts: hand-worked values, exact rationals, and the
same operators stated another way."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import int4, linear8, moe


def test_quantize_by_hand():
    q, s = linear8.quantize(np.array([[127.0, -127.0, 0.5, 1.5, -0.5, 63.49], [0.0] * 6, [2.0, -1.0, 0.0, 1.0, 0.25, -2.0]]))
    assert q.tolist() == [[127, -127, 0, 2, 0, 63], [0] * 6, [127, -64, 0, 64, 16, -127]]   # 63.5 goes to 64, 15.875 to 16
    assert s.tolist() == [1.0, 0.0, np.float32(2 / 127)]
    q, s = linear8.quantize(np.array([[1.0, np.inf], [np.nan, 3.0]]))
    assert not q.any() and np.isnan(s).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_quantize_against_rationals(dtype):
    r = np.random.default_rng(0)
    x = torch.from_numpy(r.standard_normal((40, 16)) * 2.0 ** r.integers(-8, 9, (40, 16))).to(dtype).double().numpy()
    x[0] = np.arange(16) / 2 - 4      # with 127 a power of two away: many exact ties
    x[0, 0] = 127
    q, s = linear8.quantize(x)
    for row, qr, sr in zip(x, q, s):
        a = max(abs(Fraction(v)) for v in row)
        assert [round(127 * Fraction(v) / a) for v in row] == qr.tolist()     # Python rounds halves to even
        near = [abs(Fraction(float(c)) - a / 127) for c in (np.nextafter(sr, np.float32(0)), sr, np.nextafter(sr, np.float32(9e9)))]
        assert near[1] == min(near)


def test_linear8_against_whole_numbers():
    r = np.random.default_rng(1)
    xq, wq = r.integers(-128, 128, (5, 48)).astype(np.int8), r.integers(-128, 128, (7, 48)).astype(np.int8)
    y, z, p = linear8.linear(xq, np.full(5, 0.5, np.float32), wq, np.arange(1, 8).astype(np.float32), bias=np.arange(7.0))
    for i in range(5):
        for j in range(7):
            total = sum(int(a) * int(b) for a, b in zip(xq[i], wq[j]))
            assert y[i, j] == total * 0.5 * (j + 1) + j


def _experts(e, h, i, seed=0):
    r = np.random.default_rng(seed)
    w = lambda k, n: r.integers(0, 2 ** 32, (e, k // 8, n), dtype=np.uint64).astype(np.uint32)
    s = lambda k, n: r.uniform(0.005, 0.02, (e, k // 128, n)).astype(np.float16)
    return r.standard_normal((e, h)).astype(np.float16), w(h, i), s(h, i), w(h, i), s(h, i), w(i, h), s(i, h)


def test_moe_of_one_expert_is_a_feed_forward():
    from oracle import linear
    router, wg, sg, wu, su, wd, sd = _experts(1, 128, 256)
    x = np.random.default_rng(2).standard_normal((3, 128)).astype(np.float16)
    y, _ = moe.moe(x, router, wg, sg, wu, su, wd, sd, 1)
    gate, up = linear.linear(x, wg[0], sg[0], act="silu")[0], linear.linear(x, wu[0], su[0])[0]
    assert np.allclose(y, (gate * up) @ (int4.unpack_int4(wd[0]) * np.repeat(sd[0].astype(np.float64), 128, 0)), rtol=1e-12)


def test_moe_choice():
    x = np.array([[1.0, 0, 0, 0], [0, 1.0, 0, 0]])
    router = np.array([[1.0, 0, 0, 0], [2, 3, 0, 0], [2, 0, 0, 0], [0, 3, 0, 0]])
    chosen, shares = moe.choose(x, router, 2, True)
    assert chosen == [[1, 2], [1, 3]] and np.allclose(shares, 0.5)
    chosen, shares = moe.choose(x, router, 2, False)
    e = np.exp(1.0)
    assert np.allclose(shares[0], e ** 2 / (2 * e ** 2 + e + 1)) and np.allclose(shares[1], e ** 3 / (2 * e ** 3 + 2))
    # two experts that are the same: the shares of both add up to one of the two
    a = _experts(2, 128, 128)
    twin = [np.stack([t[0], t[0]]) for t in a]
    x = np.random.default_rng(3).standard_normal((2, 128)).astype(np.float16)
    assert np.allclose(moe.moe(x, *twin, 2)[0], moe.moe(x, *[t[:1] for t in twin], 1)[0], rtol=1e-12)
