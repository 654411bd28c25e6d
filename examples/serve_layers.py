"""A stack of quantized transformer layers served over one paged cache: prompts in pieces, then tokens one at a time.

    python examples/serve_layers.py [--layers 4] [--hidden 1024] [--heads 8] [--feed w4a16 | w8a8 | experts]

Each layer is six calls of the library:

    q, k, v = kaio_qkv_w4a16(norm(x))              the fused projection
    q       = kaio_rope_append(q, k, v, ...)       rotary positions; K and V go to the layer's pages
    a       = kaio_paged_attention(q, ...)         over everything the sequence has in the cache
    x       = kaio_linear_w4a16(a, residual=x)     the projection after attention
    h       = kaio_linear_w4a16(norm(x), activation="silu", bias=...)
    x       = kaio_linear_w4a16(h, residual=x)     the feed-forward block

With ``--feed w8a8`` the last two are products in 8-bit integers:

    xq, xs  = kaio_quantize_rows(norm(x))          rows rounded to 8 bits
    h       = kaio_linear_w8a8(xq, x_scale=xs, activation="silu", bias=...)
    x       = kaio_linear_w8a8(h, residual=x)      (which rounds h itself)

and with ``--feed experts`` a mixture of experts, in one call:

    x       = kaio_moe_w4a16(norm(x), experts, top_k, residual=x)

Weights are random.  The same tokens are run whole, in pieces and one by one; the answers agree to f16's rounding.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int4_group_quantized_w4a16_amd as kaio  # noqa: E402

GROUP = kaio.GROUP_SIZE


def norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Weight:
    """A packed INT4 weight [k, n] with its scales, random, of a gain near one."""

    def __init__(self, k, n, gen):
        self.w = torch.randint(-2 ** 31, 2 ** 31, (k // 8, n), generator=gen, device=gen.device, dtype=torch.int64).int()
        self.s = ((torch.rand((k // GROUP, n), generator=gen, device=gen.device) + 0.5) * (0.2 / math.sqrt(k))).half()


class Weight8:
    """An int8 weight [n, k] with a scale for each row, random, of a gain near one."""

    def __init__(self, k, n, gen):
        self.w = torch.randint(-127, 128, (n, k), generator=gen, device=gen.device, dtype=torch.int8)
        self.s = (torch.rand(n, generator=gen, device=gen.device) + 0.5) * (0.014 / math.sqrt(k))


def experts(hidden, inner, count, gen):
    """``count`` feed-forward experts of ``inner`` columns and their router, random."""
    some = lambda k, n: [Weight(k, n, gen) for _ in range(count)]
    w = lambda ws: (torch.stack([x.w for x in ws]), torch.stack([x.s for x in ws]))
    router = (torch.randn((count, hidden), generator=gen, device=gen.device) / math.sqrt(hidden)).half()
    return kaio.KaioExperts(router, *w(some(hidden, inner)), *w(some(hidden, inner)), *w(some(inner, hidden)))


class Layer:
    def __init__(self, hidden, gen, feed="w4a16", count=8, top=2):
        self.q, self.k, self.v, self.o = (Weight(hidden, hidden, gen) for _ in range(4))
        self.feed = {"w4a16": self.feed4, "w8a8": self.feed8, "experts": self.feed_experts}[feed]
        if feed == "experts":
            self.experts, self.top = experts(hidden, hidden, count, gen), top
            return
        kind = Weight if feed == "w4a16" else Weight8
        self.up, self.down = kind(hidden, 2 * hidden, gen), kind(2 * hidden, hidden, gen)
        self.bias = torch.randn(2 * hidden, generator=gen, device=gen.device).half() * 0.1

    def feed4(self, x):
        h = kaio.kaio_linear_w4a16(norm(x), self.up.w, self.up.s, bias=self.bias, activation="silu")
        return kaio.kaio_linear_w4a16(h, self.down.w, self.down.s, residual=x)

    def feed8(self, x):
        xq, xs = kaio.kaio_quantize_rows(norm(x))
        h = kaio.kaio_linear_w8a8(xq, self.up.w, self.up.s, x_scale=xs, bias=self.bias, activation="silu")
        return kaio.kaio_linear_w8a8(h, self.down.w, self.down.s, residual=x)

    def feed_experts(self, x):
        return kaio.kaio_moe_w4a16(norm(x), self.experts, self.top, residual=x)


class Server:
    """Layers, a paged cache for each, and the pages that the sequences hold."""

    def __init__(self, layers, hidden, heads, seqs, most_tokens, page=16, window=0, sinks=0, seed=0, device="cuda", **feed):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.layers = [Layer(hidden, gen, **feed) for _ in range(layers)]
        self.heads, self.dim, self.page, self.window, self.sinks = heads, hidden // heads, page, window, sinks
        width = -(-most_tokens // page)
        self.free = torch.randperm(seqs * width, generator=torch.Generator().manual_seed(seed)).tolist()
        self.table = torch.full((seqs, width), -1, dtype=torch.int32)
        self.len = [0] * seqs
        # what the kernels read: kept for the server's life and updated in place, so that a graph may hold the calls
        self.dev = dict(table=self.table.to(device), q_start=torch.zeros(seqs + 1, dtype=torch.int32, device=device),
                        lens=torch.zeros(seqs, dtype=torch.int32, device=device))
        shape = (seqs * width, page, heads, self.dim)
        self.paged = [kaio.KaioPagedKV(torch.zeros(shape, dtype=torch.half, device=device),
                                       torch.zeros(shape, dtype=torch.half, device=device),
                                       self.dev["table"], self.dev["q_start"], self.dev["lens"]) for _ in range(layers)]
        half = self.dim // 2
        self.inv_freq = (1e4 ** (-torch.arange(half, dtype=torch.float64) / half)).to(device)

    def step(self, pieces):
        """pieces: each sequence's new tokens, f16 [n, hidden] (n may be 0); returns their outputs in one tensor."""
        new = [p.shape[0] for p in pieces]
        positions = torch.cat([torch.arange(have, have + n) for have, n in zip(self.len, new)]).int()
        for s, n in enumerate(new):
            for c in range(-(-self.len[s] // self.page), -(-(self.len[s] + n) // self.page)):
                self.table[s, c] = self.free.pop()
            self.len[s] += n
        self.dev["table"].copy_(self.table)
        self.dev["q_start"].copy_(torch.tensor([0] + new).cumsum(0).int())
        self.dev["lens"].copy_(torch.tensor(self.len, dtype=torch.int32))
        x = torch.cat(pieces)
        out = self.forward(x, positions[None].to(x.device), max(new))
        for s in range(len(new)):
            self.release(s)
        return out

    def forward(self, x, positions, max_new):
        split = lambda t: t.view(t.shape[0], self.heads, self.dim)
        for layer, paged in zip(self.layers, self.paged):
            ws = (layer.q, layer.k, layer.v)
            q, k, v = (split(t) for t in kaio.kaio_qkv_w4a16(norm(x), *[w.w for w in ws], *[w.s for w in ws]))
            q = kaio.kaio_rope_append(q, k, v, positions, self.inv_freq, [self.dim // 2], paged, q_out=q)
            a = kaio.kaio_paged_attention(q, paged, max_new, self.dim ** -0.5, window=self.window, sinks=self.sinks)
            x = kaio.kaio_linear_w4a16(a.view(x.shape), layer.o.w, layer.o.s, residual=x)
            x = layer.feed(x)
        return x

    def release(self, s):
        """With a window: gives back pages that no later token sees (the first ``sinks`` tokens stay)."""
        if not self.window:
            return
        for c in range(-(-self.sinks // self.page), max(0, self.len[s] - self.window + 1) // self.page):
            if self.table[s, c] >= 0:
                self.free.append(int(self.table[s, c]))
                self.table[s, c] = -1


def run(layers=4, hidden=1024, heads=8, lengths=(300, 77, 1), tail=5, window=0, sinks=0, seed=0, **feed):
    """The same tokens whole, and in pieces with the last ``tail`` one by one; returns both outputs, sequence by sequence.

    ``feed``: of the layers (feed="w8a8", or feed="experts" with count and top)."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    tokens = [torch.randn(n + tail, hidden, generator=gen, device="cuda").half() for n in lengths]
    make = lambda: Server(layers, hidden, heads, len(lengths), max(lengths) + tail, window=window, sinks=sinks, seed=seed, **feed)
    whole = make().step(tokens).split([t.shape[0] for t in tokens])
    server, got = make(), [[] for _ in tokens]

    def step(pieces):
        for s, y in enumerate(server.step(pieces).split([p.shape[0] for p in pieces])):
            got[s].append(y)

    cuts = [n // 3 for n in lengths]
    step([t[:c] for t, c in zip(tokens, cuts)])
    step([t[c:n] for t, c, n in zip(tokens, cuts, lengths)])
    for i in range(tail):
        step([t[n + i:n + i + 1] for t, n in zip(tokens, lengths)])
    torch.cuda.synchronize()
    return whole, [torch.cat(g) for g in got]


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--layers", type=int, default=4)
    a.add_argument("--hidden", type=int, default=1024)
    a.add_argument("--heads", type=int, default=8)
    a.add_argument("--feed", choices=("w4a16", "w8a8", "experts"), default="w4a16")
    a = a.parse_args()
    for window, sinks in ((0, 0), (64, 4)):
        whole, pieces = run(a.layers, a.hidden, a.heads, window=window, sinks=sinks, feed=a.feed)
        for s, (x, y) in enumerate(zip(whole, pieces)):
            diff = (x.float() - y.float()).norm() / x.float().norm()
            print(f"window {window:3d}, sequence {s}: {x.shape[0]} tokens, whole against pieces: relative difference {diff:.2e}")
