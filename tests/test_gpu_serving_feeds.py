"""The 8-bit and the expert feed-forward of examples/serve_layers.py: every call of them in a served run against the oracle with
that call's own inputs, and whole runs against the layers computed in float64 from the definitions."""
import numpy as np
import pytest
import torch

import int4_group_quantized_w4a16_amd as kaio
from oracle import linear as ol
from oracle import linear8, moe, paged
from oracle.qkv import dequantize
from tests.test_gpu_serving_example import host, serve

pytestmark = pytest.mark.gpu

KW = dict(layers=2, hidden=256, heads=2)
LENGTHS, TAIL = (70, 33, 1), 3
f64 = lambda t: None if t is None else t.cpu().numpy().astype(np.float64)


def expert_weights(e):
    return [t.cpu().numpy().view(np.uint32) if t.dtype == torch.int32 else t.cpu().numpy()
            for t in (e.router, e.w_gate, e.s_gate, e.w_up, e.s_up, e.w_down, e.s_down)]


@pytest.mark.parametrize("feed,calls", [("w8a8", {"kaio_quantize_rows": 1, "kaio_linear_w8a8": 2}), ("experts", {"kaio_moe_w4a16": 1})])
def test_every_call_of_a_run(feed, calls, monkeypatch):
    seen = []

    def record(name):
        real = getattr(kaio, name)

        def call(*a, **kw):
            out = real(*a, **kw)
            seen.append((name, a, kw, out))
            return out
        monkeypatch.setattr(kaio, name, call)

    for name in calls:
        record(name)
    serve.run(lengths=LENGTHS, tail=TAIL, window=24, sinks=3, seed=5, feed=feed, **KW)
    steps = 1 + 2 + TAIL   # whole; pieces
    assert {n: sum(s[0] == n for s in seen) for n in calls} == {n: c * KW["layers"] * steps for n, c in calls.items()}
    for name, a, kw, out in seen:
        if name == "kaio_quantize_rows":
            q, s = linear8.quantize(f64(a[0]))
            assert np.array_equal(out[0].cpu().numpy(), q) and np.array_equal(out[1].cpu().numpy(), s)
        elif name == "kaio_linear_w8a8":
            x, w, ws = a
            q, s = (x.cpu().numpy(), kw["x_scale"].cpu().numpy()) if "x_scale" in kw else linear8.quantize(f64(x))
            act, bias, res = kw.get("activation", "none"), f64(kw.get("bias")), f64(kw.get("residual"))
            y, z, p = linear8.linear(q, s, w.cpu().numpy(), ws.cpu().numpy(), bias, act, res)
            assert (np.abs(f64(out) - y) <= linear8.tolerance(y, z, p, act, 2.0 ** -11, 2.0 ** -25, bias, res)).all()
        else:
            x, e, top = a
            y, tol = moe.moe(x.cpu().numpy(), *expert_weights(e), top, residual=kw["residual"].cpu().numpy())
            assert (np.abs(f64(out) - y) <= tol).all()


def plain(server, x, feed):
    """One sequence [n, hidden] float64 through the server's layers; and the sum over roundings to 8 bits of half a step of the
    row's largest over the row's root mean square, the most of any row."""
    n, heads, dim = x.shape[0], server.heads, server.dim
    nrm = lambda y: y / np.sqrt((y * y).mean(-1, keepdims=True) + 1e-6)
    inv, pos, table = server.inv_freq.cpu().numpy(), np.arange(n)[None], np.zeros((1, 1), dtype=np.int64)
    steps = 0.0
    step = lambda y: float((np.abs(y).max(-1) / np.sqrt((y * y).mean(-1))).max() / 254)
    for layer in server.layers:
        q, k, v = (nrm(x) @ dequantize(*host(w)) for w in (layer.q, layer.k, layer.v))
        q, k = (paged.rotate(t.reshape(n, heads, dim), pos, inv, [dim // 2], False) for t in (q, k))
        a, _ = paged.attention(q, k[None], v.reshape(1, n, heads, dim), table, [0, n], [n], dim ** -0.5, 0, 0)
        x = ol.linear(a.reshape(n, -1), *host(layer.o))[0] + x
        if feed == "w8a8":
            w = lambda v: f64(v.w).T * f64(v.s)
            h = ol.ACT["silu"](nrm(x) @ w(layer.up) + f64(layer.bias))
            steps += step(nrm(x)) + step(h)
            x = h @ w(layer.down) + x
        else:
            x = moe.moe(nrm(x), *expert_weights(layer.experts), layer.top, residual=x)[0]
    return x, steps


@pytest.mark.parametrize("feed,more", [("w8a8", {}), ("experts", dict(count=4, top=4))])
def test_whole_and_in_pieces_against_float64(feed, more):
    # (All experts are chosen, so that the outputs are continuous in the inputs.)  Each layer rounds some ten tensors to f16
    # (2^-11 relative) and two to 8 bits (half of a 127th of the row's largest); relative errors in the norm of a row, added as
    # if they were one direction: 2 layers x 10 x 2^-11, and the sum of the other steps.  What a layer is given wrong it hands on
    # by the residual and by its own branches: twice, and three times where two projections of it are multiplied.
    whole, pieces = serve.run(lengths=LENGTHS, tail=TAIL, seed=3, feed=feed, **more, **KW)
    server = serve.Server(KW["layers"], KW["hidden"], KW["heads"], len(LENGTHS), max(LENGTHS) + TAIL, seed=3, feed=feed, **more)
    gen = torch.Generator(device="cuda").manual_seed(4)
    for n, a, b in zip(LENGTHS, whole, pieces):
        x = torch.randn(n + TAIL, KW["hidden"], generator=gen, device="cuda").half()
        want, steps = plain(server, f64(x), feed)
        for y in (a, b):
            err = np.linalg.norm(f64(y) - want, axis=-1) / np.linalg.norm(want, axis=-1)
            assert y.shape == x.shape and err.max() <= (2 if feed == "w8a8" else 3) * (2 * 10 * 2.0 ** -11 + steps), err.max()
