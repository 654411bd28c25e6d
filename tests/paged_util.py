"""Batches over a paged cache for the GPU tests: pages anywhere, a table with room, lengths given."""
import numpy as np
import torch

from tests.gpu_util import DEV

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# spacing at 1 and smallest normal number of the output types
EPS = {"f16": (2.0 ** -10, 2.0 ** -14), "bf16": (2.0 ** -7, 2.0 ** -126)}


def f64(t):
    return t.detach().cpu().double().numpy()


class Batch:
    """new[s] new tokens and lens[s] tokens of each sequence; ``pad`` rows of q in no sequence."""

    def __init__(self, new, lens, hq, hkv, d, page, dtype="f16", seed=0, window=0, sinks=0, pad=0, extra_width=1,
                 release=True):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens, self.window, self.sinks, self.dtype = list(new), list(lens), window, sinks, dtype
        self.tokens = sum(new) + pad
        need = [(x + page - 1) // page for x in lens]
        self.pages = sum(need) + 2
        width = max(need, default=0) + extra_width
        order = torch.randperm(self.pages, generator=g)
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n].int()
            at += n
            if window and release:   # pages no row can see any more
                first = max(0, lens[s] - new[s] - window + 1) // page
                table[s, min(first, (sinks + page - 1) // page):first] = -1
        self.table = table
        self.q_start = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        dt = DT[dtype]
        rnd = lambda *shape: torch.randn(*shape, generator=g).to(dt)
        self.k_cache, self.v_cache = rnd(self.pages, page, hkv, d), rnd(self.pages, page, hkv, d)
        self.q, self.k, self.v = rnd(self.tokens, hq, d), rnd(self.tokens, hkv, d), rnd(self.tokens, hkv, d)
        self.scale = d ** -0.5

    def used(self):
        """Boolean mask [pages * page] of the slots some sequence has a token in."""
        from oracle import paged
        page = self.k_cache.shape[1]
        m = torch.zeros(self.pages * page, dtype=torch.bool)
        for s, n in enumerate(self.lens):
            for c in range(n):
                i = paged.slot(self.table.numpy(), page, self.pages, s, c)
                if i >= 0:
                    m[i] = True
        return m

    def on_gpu(self):
        import int4_group_quantized_w4a16_amd as kaio
        self.dk, self.dv = self.k_cache.to(DEV), self.v_cache.to(DEV)
        self.dq = self.q.to(DEV)
        self.paged = kaio.KaioPagedKV(self.dk, self.dv, self.table.to(DEV), self.q_start.to(DEV),
                                      torch.tensor(self.lens, dtype=torch.int32, device=DEV))
        return self.paged

    def attention(self, **kw):
        import int4_group_quantized_w4a16_amd as kaio
        self.on_gpu()
        out = torch.full_like(self.dq, float("nan"))
        kaio.kaio_paged_attention(self.dq, self.paged, max(max(self.new, default=1), 1), self.scale, window=self.window,
                                  sinks=self.sinks, out=out, **kw)
        torch.cuda.synchronize()
        return out

    def expected(self):
        from oracle import paged
        y, terms = paged.attention(f64(self.q), f64(self.k_cache), f64(self.v_cache), self.table.numpy(),
                                   self.q_start.numpy(), self.lens, self.scale, self.window, self.sinks)
        return y, paged.attention_tolerance(y, terms, *EPS[self.dtype])

    def check(self, out, rows=None):
        y, tol = self.expected()
        got = f64(out)
        if rows is not None:
            got, y, tol = got[rows], y[rows], tol[rows]
        err = np.abs(got - y)
        assert np.isfinite(got).all(), "not finite"
        bad = err > tol
        worst = float((err / np.where(tol > 0, tol, 1)).max()) if err.size else 0.0
        assert not bad.any(), f"{bad.sum()} of {bad.size} outside tolerance, max |d|/tol = {worst:.3f}, " \
                              f"first at {tuple(int(i[0]) for i in np.nonzero(bad))}"
        return worst
