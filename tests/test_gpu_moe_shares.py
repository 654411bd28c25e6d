"""Shares of the chosen experts to f32's bits."""
import numpy as np
import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from tests.gpu_util import DEV, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 64])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("e", [3, 70, 300, 512])
def test_shares_of_far_scores(t, normalize, e):
    """The best expert gives zero and the second, behind by 1 to 30, a power of two that brings its share near one; the
    residual takes away all but the share's last bits.  Its error: a step of f32 of the exponential and of what corrects it,
    half a step each of the sum, of the quotient, of the product and of the sum with the residual, below 2^-21 in all;
    half a step of f16 of what is left, 2^-24."""
    r = np.random.default_rng(t + e)
    h = i = 128
    x = np.zeros((t, h), np.float16)
    x[:, 0], x[:, 1], x[:, 2] = r.uniform(1, 30, t), r.uniform(0.01, 0.02, t), 1
    router = np.zeros((e, h), np.float16)
    router[:, 2] = -200                                   # the others: nowhere
    router[0, :3], router[1, :3] = [0, 0, 0], [-1, -1, 0]
    gap = x[:, 0].astype(np.float64) + x[:, 1].astype(np.float64)
    share = np.exp(-gap) / (1 + np.exp(-gap))
    times = 2.0 ** np.round(-np.log2(share))
    one = np.full((e, h // 8, i), 0, np.uint32)
    one[:, 0, 0] = 1 << 8                                 # column 0 is x[2]
    gate, up, down = one.copy(), one.copy(), np.zeros((e, i // 8, h), np.uint32)
    down[1, 0, :] = 1                                     # of expert 1 alone, from column 0
    s = np.ones((e, 1, 128), np.float16)
    # the power of two, one per token: by x[3] through the gate, as two factors of f16's range
    gate[:, 0, 0], up[:, 0, 0] = 1 << 12, 1 << 16
    half = np.round(np.log2(times / 2.0 ** 13) / 2)       # and 2^13 by the scale of the down product: up to 2^15 in each
    x[:, 3], x[:, 4] = 2.0 ** half, times / 2.0 ** 13 / 2.0 ** half
    assert np.isfinite(x).all() and (x[:, 3:5] > 0).all()
    router[:, 3:] = 0
    res = np.repeat((-(share * times)).astype(np.float16)[:, None], h, 1)
    y = kaio.kaio_moe_w4a16(to_dev(x), kaio.KaioExperts(*[to_dev(a) for a in (router, gate, s, up, s, down, s * np.float16(8192))]), 2,
                            normalize=normalize, activation="none", residual=to_dev(res))
    torch.cuda.synchronize()
    left = share * times + res[:, 0].astype(np.float64)
    assert np.abs(left).max() > 2.0 ** -15 or t == 1
    err = np.abs(y.double().cpu().numpy() - left[:, None]).max()
    assert err <= 2.0 ** -21 * 1.5 + 2.0 ** -24, err
