"""Measured cases of the serving operators that stand around the W4A16 QKV projection.

Three operators, used one after the other in every layer of a served model:

* ``rope_append``: rotary positions (one or several axes) on Q and K, with K and V written to a paged cache;
* ``attention``: the new tokens' attention over that cache (decode, chunks, whole prompts; sliding window with sinks);
* ``linear``: the W4A16 product with bias, activation and residual in its epilogue.

Where ``own`` is false ``run`` computes them from elementary torch operations in 32 bits (angles in 64), where it is
true through the library's entry points.  A sequence s of a batch has n_s new tokens (rows q_start[s] .. q_start[s+1]
of q) and lens[s] tokens in the cache, the new ones last; its token c lies in slot c % page_size of page
page_table[s][c // page_size].
"""
import math

import torch

own = False

GROUP = 128
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


# ---------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step of a few chats: one new token each, as many K/V heads as Q heads (the projection's own form)
        dict(name="append decode", op="rope_append", dtype="f16", seqs=4, new=4, cached=900, hq=32, hkv=32, d=128, page=16,
             axes=1, rotary=128, interleaved=False),
        # image and video tokens: three axes, neighbouring pairs, a partly rotated head, ragged prompts
        dict(name="append image", op="rope_append", dtype="bf16", seqs=5, new=2357, cached=3000, hq=16, hkv=4, d=64, page=32,
             axes=3, rotary=48, interleaved=True),
        # a long prompt in one piece, grouped heads
        dict(name="append prompt", op="rope_append", dtype="f16", seqs=1, new=16384, cached=0, hq=32, hkv=8, d=128, page=64,
             axes=1, rotary=128, interleaved=False),
        # a decode step of a few chats over short caches: latency
        dict(name="decode few", op="attention", dtype="f16", seqs=4, new=4, cached=900, hq=32, hkv=32, d=128, page=16,
             window=0, sinks=0),
        # a full decode batch with caches of very different lengths
        dict(name="decode batch", op="attention", dtype="bf16", seqs=64, new=64, cached=8000, hq=32, hkv=8, d=128, page=16,
             window=0, sinks=0),
        # one long document being continued: few rows, a long axis
        dict(name="decode long", op="attention", dtype="f16", seqs=1, new=1, cached=131000, hq=32, hkv=8, d=128, page=64,
             window=0, sinks=0),
        # a prompt in one piece: no cached tokens, causal
        dict(name="prompt", op="attention", dtype="f16", seqs=1, new=8192, cached=0, hq=32, hkv=32, d=128, page=64,
             window=0, sinks=0),
        # pieces of several prompts over what is cached already, odd sizes
        dict(name="chunks", op="attention", dtype="bf16", seqs=3, new=1535, cached=12001, hq=32, hkv=8, d=128, page=32,
             window=0, sinks=0),
        # a piece of a long stream: sliding window, the first tokens stay, pages between them released
        dict(name="window", op="attention", dtype="f16", seqs=2, new=2049, cached=30000, hq=16, hkv=4, d=64, page=16,
             window=4096, sinks=4),
        # the product after attention in a decode step: bias and residual
        dict(name="linear decode", op="linear", m=8, n=4096, k=4096, act="none", bias=True, residual=True),
        # the widening product of a small batch, odd rows and columns
        dict(name="linear batch", op="linear", m=61, n=11004, k=4096, act="silu", bias=False, residual=False),
        # a prompt's product, everything in the epilogue
        dict(name="linear prompt", op="linear", m=2048, n=4096, k=4096, act="gelu_tanh", bias=True, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    hkv = rng.choice((1, 2, 4, 8, 16, 32))
    return hkv * rng.choice([g for g in (1, 2, 3, 4, 7, 8) if hkv * g <= 32]), hkv


def draw(rng):
    op = rng.choice(("rope_append", "attention", "attention", "linear"))
    if op == "linear":
        return dict(op=op, m=_log(rng, 1, 2048), n=rng.choice((512, 1000, 2048, 4088, 4096)) + rng.choice((0, 0, 4, 1)),
                    k=GROUP * rng.choice((4, 6, 8, 11, 16, 21, 28, 32)), act=rng.choice(ACTIVATIONS), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    hq, hkv = _heads(rng)
    d = rng.choice((64, 128))
    dtype = rng.choice(("f16", "bf16"))
    page = rng.choice((8, 16, 32, 64, 128))
    seqs = _log(rng, 1, 32)
    if op == "rope_append":
        return dict(op=op, dtype=dtype, seqs=seqs, new=seqs + _log(rng, 1, 8192) - 1, cached=_log(rng, 1, 4000), hq=hq, hkv=hkv,
                    d=d, page=page, axes=rng.choice((1, 2, 3)), rotary=rng.choice((d // 2, d)),
                    interleaved=rng.random() < 0.5)
    windowed = rng.random() < 0.4
    window, sinks = (_log(rng, 16, 4096), rng.choice((0, 1, 4, 70))) if windowed else (0, 0)
    if rng.random() < 0.5:   # decode
        return dict(op=op, dtype=dtype, seqs=seqs, new=seqs, cached=_log(rng, 1, 120000 // seqs), hq=hq, hkv=hkv, d=d,
                    page=page, window=window, sinks=sinks)
    seqs = rng.choice((1, 2, 3, 5))
    new = seqs + _log(rng, 2, 2048)
    return dict(op=op, dtype=dtype, seqs=seqs, new=new, cached=_log(rng, 1, 12000 // seqs), hq=hq, hkv=hkv, d=d, page=page,
                window=window, sinks=sinks)


# ---------------------------------------------------------------------------------------------- their sizes
def _lengths(case):
    """New and cached tokens of each sequence: the case's totals, dealt out unevenly and always alike."""
    n = case["seqs"]
    new = [case["new"] // n] * n
    new[-1] += case["new"] - sum(new)
    if case["new"] > n and n > 1:      # a ragged batch: move tokens from each sequence to its neighbour
        for i in range(0, n - 1, 2):
            step = min(new[i] - 1, (new[i] * (i + 1)) // (2 * n))
            new[i] -= step
            new[i + 1] += step
    cached = [max(0, case["cached"] * (n - i) // n) if n > 1 else case["cached"] for i in range(n)]
    return new, cached


def _visible(pos, window, sinks):
    """Visible tokens of a query at position pos."""
    if window == 0 or pos < window:
        return pos + 1
    return window + min(sinks, pos + 1 - window)


def _visible_sum(first, count, window, sinks):
    return sum(_visible(p, window, sinks) for p in range(first, first + count))


def work(case):
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        b = k * n // 2 + (k // GROUP) * n * 2 + 2 * m * k + 2 * m * n
        return {"bytes": b + 2 * n * case["bias"] + 2 * m * n * case["residual"], "flops": 2.0 * m * n * k}
    t, hq, hkv, d = case["new"], case["hq"], case["hkv"], case["d"]
    new, cached = _lengths(case)
    if case["op"] == "rope_append":
        return {"bytes": 2 * 2 * t * (hq + 2 * hkv) * d + 4 * t * case["axes"] + 4 * case["rotary"],
                "flops": 3.0 * t * (hq + hkv) * case["rotary"]}
    w, s = case["window"], case["sinks"]
    seen = sum(_visible_sum(c, n, w, s) for n, c in zip(new, cached))
    keys = sum(n + c if w == 0 else min(n + c, n - 1 + w + min(s, c + n)) for n, c in zip(new, cached))
    return {"bytes": 2 * 2 * keys * hkv * d + 2 * 2 * t * hq * d, "flops": 4.0 * d * hq * seen}


# ---------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=torch.float16):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        st = dict(case, x=normal(m, k),
                  w=torch.randint(-2 ** 31, 2 ** 31, (k // 8, n), generator=gen, device=dev, dtype=torch.int64).to(torch.int32),
                  s=(torch.rand((k // GROUP, n), generator=gen, device=dev) * 0.015 + 0.005).to(torch.float16))
        st["b"] = normal(n) if case["bias"] else None
        st["r"] = normal(m, n) if case["residual"] else None
        return st

    dtype, page, hkv, d = DTYPES[case["dtype"]], case["page"], case["hkv"], case["d"]
    new, cached = _lengths(case)
    lens = [a + b for a, b in zip(new, cached)]
    width = max((x + page - 1) // page for x in lens)
    pages = sum((x + page - 1) // page for x in lens) + 3
    order = torch.randperm(pages, generator=host)      # a cache in use: a sequence's pages lie anywhere
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for i, x in enumerate(lens):
        c = (x + page - 1) // page
        table[i, :c] = order[at:at + c]
        at += c
        if case.get("window"):                          # pages that no query can see any more were given back
            first = max(0, lens[i] - new[i] - case["window"] + 1) // page
            table[i, min(first, (case["sinks"] + page - 1) // page):first] = -1
    starts = [0]
    for x in new:
        starts.append(starts[-1] + x)
    t = starts[-1]
    st = dict(case, k_cache=torch.empty((pages, page, hkv, d), device=dev, dtype=dtype),
              v_cache=torch.empty((pages, page, hkv, d), device=dev, dtype=dtype),
              table=table.to(dev), q_start=torch.tensor(starts, dtype=torch.int32).to(dev),
              lens=torch.tensor(lens, dtype=torch.int32).to(dev), most_new=max(new), most_len=max(lens),
              q=normal(t, case["hq"], d, dtype=dtype))
    st["k_cache"].normal_(generator=gen)
    st["v_cache"].normal_(generator=gen)
    if case["op"] == "rope_append":
        st["k"], st["v"] = normal(t, hkv, d, dtype=dtype), normal(t, hkv, d, dtype=dtype)
        half, axes = case["rotary"] // 2, case["axes"]
        st["sections"] = [half // axes + (half % axes if a == 0 else 0) for a in range(axes)]
        p = torch.arange(half, dtype=torch.float64)
        st["inv_freq"] = (1e4 ** (-p / half)).to(dev)
        pos = torch.cat([torch.arange(c, c + n) for n, c in zip(new, cached)])
        if axes > 1:                                    # time, then rows and columns of a picture 40 patches wide
            pos = torch.stack([pos] + [pos // 40, pos % 40][:axes - 1])
        st["positions"] = pos.reshape(axes, t).to(torch.int32).to(dev)
    else:
        st["scale"] = d ** -0.5
    if own:
        # what a serving program keeps from step to step: the description of its cache's and its batch's buffers
        from int4_group_quantized_w4a16_amd import KaioPagedKV
        st["paged"] = KaioPagedKV(st["k_cache"], st["v_cache"], st["table"], st["q_start"], st["lens"])
    return st


# ---------------------------------------------------------------------------------------------- one pass
def run(state):
    if not own:
        return {"rope_append": _append, "attention": _attention, "linear": _linear}[state["op"]](state)
    import int4_group_quantized_w4a16_amd as kaio
    st = state
    if st["op"] == "linear":
        return kaio.kaio_linear_w4a16(st["x"], st["w"], st["s"], bias=st["b"], activation=st["act"], residual=st["r"])
    if st["op"] == "rope_append":
        q = kaio.kaio_rope_append(st["q"], st["k"], st["v"], st["positions"], st["inv_freq"], st["sections"], st["paged"],
                                  interleaved=st["interleaved"])
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    return kaio.kaio_paged_attention(st["q"], st["paged"], max_new=st["most_new"], scale=st["scale"], window=st["window"],
                                     sinks=st["sinks"])


def _rows(st):
    """Sequence and cache position of each new token."""
    t = torch.arange(st["q"].shape[0], device=st["q"].device, dtype=torch.int32)
    seq = torch.searchsorted(st["q_start"][1:], t, right=True)
    pos = t - st["q_start"][1:][seq] + st["lens"][seq]
    return seq, pos.long()


def _append(st):
    half = st["rotary"] // 2
    axis = torch.repeat_interleave(torch.arange(st["axes"], device=st["q"].device),
                                   torch.tensor(st["sections"], device=st["q"].device), output_size=half)
    angle = st["positions"].double()[axis].T * st["inv_freq"]           # [T, half]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x):
        y = x.float()
        r = y[..., :2 * half]
        a, b = (r[..., 0::2], r[..., 1::2]) if st["interleaved"] else (r[..., :half], r[..., half:])
        a, b = a * cos - b * sin, a * sin + b * cos
        r = torch.stack((a, b), -1).flatten(-2) if st["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((r, y[..., 2 * half:]), -1).to(x.dtype)

    seq, pos = _rows(st)
    page = st["table"][seq, pos // st["page"]].long()
    st["k_cache"][page, pos % st["page"]] = turn(st["k"])
    st["v_cache"][page, pos % st["page"]] = st["v"]
    return {"q": turn(st["q"]), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _attention(st):
    q, table, page = st["q"], st["table"].long(), st["page"]
    t, hq, d = q.shape
    hkv, n, most = st["hkv"], st["seqs"], st["most_new"]
    g = hq // hkv
    seq, pos = _rows(st)
    row = torch.arange(t, device=q.device) - st["q_start"].long()[seq]
    qs = torch.zeros((n, most, hq, d), device=q.device)
    qs[seq, row] = q.float()
    at = torch.full((n, most), -1, device=q.device)
    at[seq, row] = pos
    there = (table >= 0).repeat_interleave(page, 1)                     # [n, L]
    ks = st["k_cache"][table.clamp(min=0)].flatten(1, 2).float()         # [n, L, hkv, d]
    vs = st["v_cache"][table.clamp(min=0)].flatten(1, 2).float()
    j = torch.arange(there.shape[1], device=q.device)
    sees = there[:, None] & (j <= at[..., None])                        # [n, most, L]
    vs = torch.where((there & (j < st["lens"][:, None]))[..., None, None], vs, 0.0)
    if st["window"]:
        sees &= (j > at[..., None] - st["window"]) | (j < st["sinks"])
    qs = qs.reshape(n, most, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * most, d)
    p = qs @ ks.permute(0, 2, 3, 1).contiguous()                        # [n, hkv, g * most, L]
    p = p.reshape(n, hkv, g, most, -1).mul_(st["scale"]).masked_fill_(~sees[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1)
    o = (p.reshape(n, hkv, g * most, -1) @ vs.permute(0, 2, 1, 3).contiguous()).reshape(n, hkv, g, most, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(n, most, hq, d)[seq, row].to(q.dtype)


def _act(y, name):
    if name == "relu":
        return torch.where(y < 0, torch.zeros_like(y), y)
    if name == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y * torch.sigmoid(y) if name == "silu" else y


def _linear(st):
    shift = torch.arange(0, 32, 4, device=st["w"].device, dtype=torch.int32)
    nib = (st["w"][:, None] >> shift[None, :, None]) & 15               # [k/8, 8, n]
    q = ((nib ^ 8) - 8).reshape(-1, st["w"].shape[1]).float()
    y = st["x"].float() @ (q * st["s"].float().repeat_interleave(GROUP, 0))
    if st["b"] is not None:
        y = y + st["b"].float()
    y = _act(y, st["act"])
    return (y + st["r"].float() if st["r"] is not None else y).half()


# ---------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        w = st["w"].long() & 0xFFFFFFFF
        cols = []
        for i in range(8):
            v = (w >> (4 * i)) % 16
            cols.append(torch.where(v >= 8, v - 16, v))
        w = torch.stack(cols, 1).reshape(case["k"], case["n"]).double()
        w *= st["s"].double().repeat_interleave(GROUP, 0)
        y = st["x"].double() @ w
        if case["bias"]:
            y += st["b"].double()
        if case["act"] == "relu":
            y = y.clamp(min=0)
        elif case["act"] == "gelu":
            y = y / 2 * torch.erfc(-y / math.sqrt(2.0))
        elif case["act"] == "gelu_tanh":
            y = y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
        elif case["act"] == "silu":
            y = y / (1 + torch.exp(-y))
        return y + st["r"].double() if case["residual"] else y
    new, cached = _lengths(case)
    page, hq, hkv, d = case["page"], case["hq"], case["hkv"], case["d"]
    table = st["table"].cpu().tolist()
    starts = st["q_start"].cpu().tolist()
    if case["op"] == "rope_append":
        half = case["rotary"] // 2
        turn = torch.empty((starts[-1], half), dtype=torch.complex128, device=st["q"].device)
        p0 = 0
        for a, c in enumerate(st["sections"]):
            ang = st["positions"][a].double()[:, None] * st["inv_freq"][p0:p0 + c]
            turn[:, p0:p0 + c] = torch.polar(torch.ones_like(ang), ang)
            p0 += c
        i0 = torch.arange(half, device=turn.device) * (2 if case["interleaved"] else 1)
        i1 = i0 + (1 if case["interleaved"] else half)

        def rotate(x):
            y = x.double()
            z = torch.complex(y[..., i0], y[..., i1]) * turn[:, None]
            y[..., i0], y[..., i1] = z.real, z.imag
            return y

        kc, vc, kr = st["k_cache"].double(), st["v_cache"].double(), rotate(st["k"])
        for s, (n, c) in enumerate(zip(new, cached)):
            where = [table[s][x // page] * page + x % page for x in range(c, c + n)]
            where = torch.tensor(where, device=kc.device)
            kc.view(-1, hkv, d)[where] = kr[starts[s]:starts[s + 1]]
            vc.view(-1, hkv, d)[where] = st["v"][starts[s]:starts[s + 1]].double()
        return {"q": rotate(st["q"]), "k_cache": kc, "v_cache": vc}
    out = torch.empty((starts[-1], hq, d), dtype=torch.float64, device=st["q"].device)
    kf, vf = st["k_cache"].view(-1, hkv, d), st["v_cache"].view(-1, hkv, d)
    for s, (n, c) in enumerate(zip(new, cached)):
        keys = [x for x in range(c + n) if table[s][x // page] >= 0]
        slots = torch.tensor([table[s][x // page] * page + x % page for x in keys], device=out.device)
        keys = torch.tensor(keys, device=out.device)
        at = torch.arange(c, c + n, device=out.device)
        hidden = keys[None] > at[:, None]
        if case["window"]:
            hidden |= (at[:, None] - keys[None] >= case["window"]) & (keys[None] >= case["sinks"])
        for h in range(hq):
            kh, vh = kf[slots, h * hkv // hq].double(), vf[slots, h * hkv // hq].double()
            z = st["q"][starts[s]:starts[s + 1], h].double() @ kh.T.contiguous() * st["scale"]
            out[starts[s]:starts[s + 1], h] = torch.softmax(z.masked_fill_(hidden, -math.inf), -1) @ vh
    return out
