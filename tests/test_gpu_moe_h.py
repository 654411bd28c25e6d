"""h of the mixture of experts between its products: 22 bits and more, whatever its size (tolerance: oracle.moe.moe)."""
import numpy as np
import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from oracle import moe as om
from tests.gpu_util import DEV, to_dev
from tests.test_gpu_moe import compare, tokens, weights

pytestmark = pytest.mark.gpu


def run(x, ws, top, normalize=True, act="silu"):
    y = kaio.kaio_moe_w4a16(to_dev(x), kaio.KaioExperts(*[to_dev(a) for a in ws]), top, normalize=normalize, activation=act)
    torch.cuda.synchronize()
    return y


def check(x, ws, top, **kw):
    y = run(x, ws, top, **kw)
    want, tol = om.moe(x, *ws, top, **kw)
    assert np.isfinite(want).all() and (np.abs(want) < 65504).all()
    compare(y, want, tol)
    return want


def largest_h(x, ws, act):
    """of expert 0, in float64"""
    from oracle.linear import ACT
    from oracle.qkv import dequantize
    xr = x.astype(np.float64)
    return np.abs(ACT[act](xr @ dequantize(ws[1][0], ws[2][0])) * (xr @ dequantize(ws[3][0], ws[4][0])))


# rows of an expert: fewer than a tile of 8, more, more than 16
@pytest.mark.parametrize("t,e,top", [(1, 4, 1), (5, 4, 2), (12, 2, 1), (40, 2, 2), (64, 3, 1)])
@pytest.mark.parametrize("act", ["silu", "none", "relu"])
def test_h_past_the_range_of_f16_with_a_finite_result(t, e, top, act):
    ws, x = weights(e, 256, 384), tokens(t, 256)
    x[::2] *= np.float16(200)                     # every second token; the others are as ever
    ws[0] = (ws[0].astype(np.float32) / 100).astype(np.float16)
    ws[6] = (ws[6].astype(np.float32) / 1024).astype(np.float16)
    assert largest_h(x, ws, act)[0].max() > 65504
    check(x, ws, top, act=act)


@pytest.mark.parametrize("t,e,top", [(1, 4, 1), (5, 4, 2), (12, 2, 1), (40, 2, 2), (64, 3, 1)])
def test_h_below_the_normal_numbers_of_f16(t, e, top):
    ws, x = weights(e, 256, 384), tokens(t, 256)
    x = (x.astype(np.float32) / 256).astype(np.float16)
    ws[6] = (ws[6].astype(np.float32) * 2048).astype(np.float16)
    assert np.median(largest_h(x, ws, "silu")[0]) < 2.0 ** -14
    want = check(x, ws, top)
    assert np.median(np.abs(want)) > 2.0 ** -11   # the results are normal numbers, and their own half step is not what hides h's


@pytest.mark.parametrize("t,e,top", [(1, 4, 1), (6, 4, 2), (13, 2, 1), (40, 2, 2), (64, 2, 1)])
@pytest.mark.parametrize("normalize", [True, False])
def test_h_of_many_sizes_in_one_row(t, e, top, normalize):
    # scales of whole strips of inner columns, of single columns, and tokens, over 2^-20 to 2^8 each
    r = np.random.default_rng(t)
    ws, x = weights(e, 256, 512, 3), tokens(t, 256, 3)
    strips = 2.0 ** r.integers(-16, 7, (e, 1, 16)).repeat(32, -1)
    some = np.where(r.random((e, 1, 512)) < 0.1, 2.0 ** r.integers(-8, 3, (e, 1, 512)), 1.0)
    for i in (2, 4):
        ws[i] = (ws[i] * strips * some).astype(np.float16)
    ws[2][:, :, 64:96] = 0                        # a strip of zeros
    x = (x * 2.0 ** r.integers(-6, 3, (t, 1))).astype(np.float16)
    ws[6] = (ws[6].astype(np.float32) / 512).astype(np.float16)
    spread = largest_h(x, ws, "silu")[0].reshape(16, 32).max(-1)
    assert spread[spread > 0].min() * 2.0 ** 20 < spread.max()
    y, (want, tol) = run(x, ws, top, normalize=normalize), om.moe(x, *ws, top, normalize=normalize)
    fits = np.abs(want) < 60000
    assert fits.mean() > 0.9
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= tol)[fits].all(), f"{(~(err <= tol))[fits].sum()} of {fits.sum()} outside tolerance"


def test_infinities_among_h_of_many_sizes():
    # an inner column that is infinite, in a strip whose other columns are far below the rest: results are infinite, of the
    # down weight's sign, or not a number where that weight is zero
    ws, x = weights(2, 128, 256), tokens(3, 128)
    x[:] = np.abs(x)
    ws[0][0], ws[0][1] = 1, -1                    # all tokens to expert 0
    for i in (1, 3):
        ws[i][0, :, 32:64] = 0x11111111           # weights of one: gate and up are sums of x
    ws[2][0, 0, 32:64], ws[4][0, 0, 32:64] = 2.0 ** -20, 2.0 ** -10
    ws[2][0, 0, 40] = np.inf
    y = run(x, ws, 1).double().cpu().numpy()
    q = (ws[5][0, 40 // 8].astype(np.int64) >> 4 * (40 % 8)) & 15
    q = np.where(q > 7, q - 16, q)
    assert np.isnan(y[:, q == 0]).all() and (q == 0).any()
    assert (y[:, q > 0] == np.inf).all() and (y[:, q < 0] == -np.inf).all()


@pytest.mark.parametrize("t,e,top", [(4, 8, 2), (33, 16, 4), (60, 4, 2)])
def test_results_are_the_rounded_sums_but_near_a_border(t, e, top):
    """Products of 512 terms in f32 are off by some 2^-20 of a typical result (errors of a step's half, added like a walk:
    sqrt(512) 2^-24), twice, and h by 2^-22, so that about one result in 2^11 / 2^19 = 2^-8 lies close enough to the border
    between two f16 numbers to go to the other; one in 2^-5 is allowed.  (h in f16 is off by 2^-12 a term and shifts
    results by a quarter of their step: one in four or five.)"""
    ws, x = weights(e, 512, 512, 5), tokens(t, 512, 5)
    y = run(x, ws, top).cpu().numpy()
    want = om.moe(x, *ws, top)[0].astype(np.float16)
    assert (y != want).mean() < 2.0 ** -5


def test_mixed_rows_on_two_streams_and_in_a_graph():
    ws, x = weights(6, 256, 256), to_dev(tokens(30, 256))
    ws[2][:, :, :64] = (ws[2][:, :, :64] * np.float32(2.0 ** -9)).astype(np.float16)
    x[::3] *= 30
    experts = kaio.KaioExperts(*[to_dev(a) for a in ws])
    need = kaio.lib().kaio_moe_w4a16_workspace_size(experts._ref, 30, 2)
    scratch = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    ref = kaio.kaio_moe_w4a16(x, experts, 2)
    assert torch.equal(ref, kaio.kaio_moe_w4a16(x, experts, 2, workspace=scratch))
    torch.cuda.synchronize()
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(g):
        kaio.kaio_moe_w4a16(x, experts, 2, y=out, workspace=scratch)
    for factor in (1.0, 0.01, 100.0, 1.0):         # other bins than the call before: none is left over
        x.mul_(factor)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kaio.kaio_moe_w4a16(x, experts, 2))
        torch.cuda.synchronize()
