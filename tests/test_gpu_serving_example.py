"""The serving operators together: examples/serve_layers.py against the layers computed in float64 from the definitions."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import linear as ol
from oracle import paged
from oracle.qkv import dequantize

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "serve_layers", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_layers.py"))
serve = importlib.util.module_from_spec(spec)
spec.loader.exec_module(serve)


def host(w):
    return w.w.cpu().numpy().view(np.uint32), w.s.cpu().numpy()


def plain(server, x, window, sinks):
    """One sequence [n, hidden] float64 through the server's layers, every token at once."""
    n, heads, dim = x.shape[0], server.heads, server.dim
    nrm = lambda y: y / np.sqrt((y * y).mean(-1, keepdims=True) + 1e-6)
    inv = server.inv_freq.cpu().numpy()
    pos = np.arange(n)[None]
    table = np.zeros((1, 1), dtype=np.int64)
    for layer in server.layers:
        q, k, v = (nrm(x) @ dequantize(*host(w)) for w in (layer.q, layer.k, layer.v))
        q, k = (paged.rotate(t.reshape(n, heads, dim), pos, inv, [dim // 2], False) for t in (q, k))
        a, _ = paged.attention(q, k[None], v.reshape(1, n, heads, dim), table, [0, n], [n], dim ** -0.5, window, sinks)
        x = ol.linear(a.reshape(n, -1), *host(layer.o))[0] + x
        h = ol.linear(nrm(x), *host(layer.up), bias=layer.bias.cpu().numpy(), act="silu")[0]
        x = ol.linear(h, *host(layer.down))[0] + x
    return x


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_whole_and_in_pieces_against_float64(window, sinks):
    # Each layer rounds some ten tensors to f16 on the way (half a step: 2^-11 relative); their relative errors add in
    # root mean square where they are independent, in sum at worst: 2 layers x 10 x 2^-11 of a vector's norm.
    kw = dict(layers=2, hidden=256, heads=2)
    lengths, tail = (70, 33, 1), 3
    whole, pieces = serve.run(lengths=lengths, tail=tail, window=window, sinks=sinks, seed=3, **kw)
    server = serve.Server(kw["layers"], kw["hidden"], kw["heads"], len(lengths), max(lengths) + tail, window=window,
                          sinks=sinks, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    for n, a, b in zip(lengths, whole, pieces):
        x = torch.randn(n + tail, kw["hidden"], generator=gen, device="cuda").half()
        want = plain(server, x.cpu().numpy().astype(np.float64), window, sinks)
        for y in (a, b):
            err = np.linalg.norm(y.cpu().numpy().astype(np.float64) - want, axis=-1) / np.linalg.norm(want, axis=-1)
            assert y.shape == x.shape and err.max() <= 2 * 10 * 2.0 ** -11, err.max()
