"""Measured cases of the products that a served layer on quantized weights makes besides the W4A16 ones.

* ``quantize``: tokens rounded to 8 bits, each with a scale of its own;
* ``linear``: the product in 8-bit integers with a scale for each token and each channel, with bias, activation and
  residual; a 16-bit x is rounded within the call;
* ``experts``: a mixture-of-experts feed-forward on packed W4A16 weights, from the router to the weighted sum.

Where ``own`` is false ``run`` computes them from elementary torch operations in 32 bits (the router's scores, whose
order decides, in 64), where it is true through the library's entry points.  Weights of the 8-bit product are int8 [n, k];
those of the experts int4 as u32 [experts, k / 8, n], low nibble first, with f16 scales [experts, k / 128, n].
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
        # the rounding before a decode step's products: latency
        dict(name="quantize decode", op="quantize", dtype="f16", m=8, k=4096),
        # the rounding before a prompt's down product, odd rows
        dict(name="quantize prompt", op="quantize", dtype="bf16", m=8191, k=8192),
        # one new token through the projection after attention: the weights are the work
        dict(name="linear token", op="linear", dtype="f16", m=1, n=4096, k=4096, act="none", bias=True, residual=True),
        # a decode batch through a widening product, odd rows and columns
        dict(name="linear batch", op="linear", dtype="bf16", m=61, n=11004, k=4096, act="silu", bias=False, residual=False),
        # short prompts gathered, odd rows
        dict(name="linear chunk", op="linear", dtype="f16", m=509, n=4096, k=4096, act="gelu", bias=True, residual=False),
        # a prompt's product, everything in the epilogue
        dict(name="linear prompt", op="linear", dtype="bf16", m=2048, n=4096, k=8192, act="gelu_tanh", bias=True, residual=True),
        # Q, K and V of a long prompt in one product, of tokens rounded before
        dict(name="linear long", op="linear", dtype="int8", m=8192, n=12288, k=4096, act="none", bias=False, residual=False),
        # one new token, many small experts: latency
        dict(name="experts token", op="experts", t=1, experts=64, top=8, hidden=2048, inner=1024, act="silu", normalize=True,
             residual=True),
        # a few chats, few large experts
        dict(name="experts few", op="experts", t=8, experts=8, top=2, hidden=4096, inner=8192, act="silu", normalize=True,
             residual=False),
        # a decode batch, many small experts, most of them with a token or two
        dict(name="experts batch", op="experts", t=33, experts=128, top=8, hidden=2048, inner=768, act="silu", normalize=True,
             residual=True),
        # the largest decode batch, weights of the chosen not brought to a sum of one, sizes off the powers of two
        dict(name="experts full", op="experts", t=64, experts=60, top=4, hidden=2048, inner=1408, act="gelu", normalize=False,
             residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "experts", "experts"))
    if op == "quantize":
        return dict(op=op, dtype=rng.choice(("f16", "bf16")), m=_log(rng, 1, 8191), k=16 * _log(rng, 8, 512))
    if op == "linear":
        return dict(op=op, dtype=rng.choice(("f16", "bf16", "int8")), m=_log(rng, 1, 4096),
                    n=rng.choice((512, 1000, 2048, 4088, 4096, 8192, 11000)) + rng.choice((0, 0, 4, 1)),
                    k=16 * _log(rng, 16, 512), act=rng.choice(ACTIVATIONS), bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5)
    experts = rng.choice((4, 8, 16, 30, 64, 128))
    top = rng.choice([k for k in (1, 2, 3, 4, 6, 8) if k <= experts])
    hidden = GROUP * rng.choice((4, 7, 8, 16, 21, 32))
    most = 400e6 / (1.6 * experts * hidden)     # columns of an expert that keep the weights under 400 MB
    inner = GROUP * max(1, _log(rng, 1, min(64, max(1, most / GROUP))))
    return dict(op=op, t=_log(rng, 1, 64), experts=experts, top=top, hidden=hidden, inner=inner, act=rng.choice(("silu", "gelu", "relu")),
                normalize=rng.random() < 0.5, residual=rng.random() < 0.5)


def work(case):
    if case["op"] == "quantize":
        m, k = case["m"], case["k"]
        return {"bytes": 3 * m * k + 4 * m, "flops": 3.0 * m * k}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        b = n * k + 4 * n + (m * k + 4 * m if case["dtype"] == "int8" else 2 * m * k) + 2 * m * n
        return {"bytes": b + 2 * n * case["bias"] + 2 * m * n * case["residual"], "flops": 2.0 * m * n * k}
    t, e, h, i = case["t"], case["experts"], case["hidden"], case["inner"]
    # experts that some token chooses, when every set of choices is alike
    chosen = e * (1 - (1 - case["top"] / e) ** t)
    b = chosen * 3 * h * i * (0.5 + 2 / GROUP) + 2 * e * h + 2 * 2 * t * h
    return {"bytes": b + 2 * t * h * case["residual"], "flops": 6.0 * t * case["top"] * h * i + 2.0 * t * e * h}


# ---------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=torch.float16, scale=1.0):
        return (torch.randn(shape, generator=gen, device=dev, dtype=torch.float32) * scale).to(dtype)

    def tokens(m, k, dtype):
        """Activations as a layer has them: rows of different sizes, a few channels that stand out."""
        x = torch.randn((m, k), generator=gen, device=dev)
        x *= torch.rand((m, 1), generator=gen, device=dev) * 3 + 0.25
        x *= torch.where(torch.rand((k,), generator=gen, device=dev) < 0.002, 8.0, 1.0)
        return x.to(dtype)

    if case["op"] == "quantize":
        return dict(case, x=tokens(case["m"], case["k"], DTYPES[case["dtype"]]))
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        dtype = DTYPES.get(case["dtype"], torch.float16)
        st = dict(case, out=dtype,
                  w=torch.randint(-127, 128, (n, k), generator=gen, device=dev, dtype=torch.int8),
                  ws=torch.rand((n,), generator=gen, device=dev) * 4e-4 + 1e-4)
        if case["dtype"] == "int8":
            st["x"] = torch.randn((m, k), generator=gen, device=dev).mul_(32).round_().clamp_(-127, 127).to(torch.int8)
            st["xs"] = torch.rand((m,), generator=gen, device=dev) * 0.04 + 0.01
        else:
            st["x"], st["xs"] = tokens(m, k, dtype), None
        st["b"] = normal(n, dtype=dtype) if case["bias"] else None
        st["r"] = normal(m, n, dtype=dtype) if case["residual"] else None
        return st
    t, e, h, i = case["t"], case["experts"], case["hidden"], case["inner"]

    def packed(k, n):
        w = torch.empty((e, k // 8, n), device=dev, dtype=torch.int32)
        w.view(torch.uint8).random_(0, 256, generator=gen)
        return w, (torch.rand((e, k // GROUP, n), generator=gen, device=dev) * 0.015 + 0.005).to(torch.float16)

    st = dict(case, x=normal(t, h), router=normal(e, h, scale=2 / math.sqrt(h)))
    for name, (k, n) in dict(gate=(h, i), up=(h, i), down=(i, h)).items():
        st["w_" + name], st["s_" + name] = packed(k, n)
    st["r"] = normal(t, h) if case["residual"] else None
    if own:
        # what a serving program keeps for each layer: the description of its experts' buffers
        from int4_group_quantized_w4a16_amd import KaioExperts
        st["e"] = KaioExperts(st["router"], st["w_gate"], st["s_gate"], st["w_up"], st["s_up"], st["w_down"], st["s_down"])
    return st


# ---------------------------------------------------------------------------------------------- one pass
def run(state):
    if not own:
        return {"quantize": _quantize_case, "linear": _linear, "experts": _experts}[state["op"]](state)
    import int4_group_quantized_w4a16_amd as kaio
    st = state
    if st["op"] == "quantize":
        q, scale = kaio.kaio_quantize_rows(st["x"])
        return {"q": q, "scale": scale}
    if st["op"] == "linear":
        return kaio.kaio_linear_w8a8(st["x"], st["w"], st["ws"], x_scale=st["xs"], bias=st["b"], activation=st["act"],
                                     residual=st["r"])
    return kaio.kaio_moe_w4a16(st["x"], st["e"], st["top"], normalize=st["normalize"], activation=st["act"], residual=st["r"])


def _quantize(x):
    """Rounded tokens and their scales.  127 x is exact in 32 bits, and a quotient of a 16-bit number's 127-fold and
    another lies further from any border between two integers than 32 bits round, unless it lies on it."""
    y = x.float()
    most = y.abs().amax(-1, keepdim=True)
    fine = torch.isfinite(most)
    q = torch.where(fine & (most > 0), y * 127 / most, 0.0).round().to(torch.int8)
    return q, torch.where(fine, most / 127, math.nan)[:, 0]


def _quantize_case(st):
    q, scale = _quantize(st["x"])
    return {"q": q, "scale": scale}


def _act(y, name):
    if name == "relu":
        return torch.where(y < 0, torch.zeros_like(y), y)
    if name == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y * torch.sigmoid(y) if name == "silu" else y


def _linear(st):
    q, scale = (st["x"], st["xs"]) if st["xs"] is not None else _quantize(st["x"])
    y = (q.float() @ st["w"].float().T) * scale[:, None] * st["ws"]
    if st["b"] is not None:
        y = y + st["b"].float()
    y = _act(y, st["act"])
    return (y + st["r"].float() if st["r"] is not None else y).to(st["out"])


def _dequant(w, s):
    """[..., k / 8, n] words and [..., k / 128, n] scales -> [..., k, n] in 32 bits."""
    shift = torch.arange(0, 32, 4, device=w.device, dtype=torch.int32)
    nib = (w[..., None, :] >> shift[:, None]) & 15
    q = ((nib ^ 8) - 8).flatten(-3, -2).float()
    return (q.unflatten(-2, (-1, GROUP)) * s.float()[..., None, :]).flatten(-3, -2)


def _experts(st):
    x, t, e = st["x"], st["t"], st["experts"]
    z = x.double() @ st["router"].double().T
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :st["top"]]    # ties: the lowest index
    p = torch.exp(z - z.amax(-1, keepdim=True)).float()
    share = p.gather(1, order)
    share = share / (share if st["normalize"] else p).sum(-1, keepdim=True)
    if t * st["top"] < e:      # the weights of each choice, gathered
        pick = order.flatten()
        rows = x.float().repeat_interleave(st["top"], 0)[:, None]                      # [choices, 1, hidden]
        share = share.flatten()[:, None, None]
        gate, up, down = (_dequant(st["w_" + n][pick], st["s_" + n][pick]) for n in ("gate", "up", "down"))
    else:                      # every expert on every token; a share of zero where it was not chosen
        rows = x.float()[None]
        share = torch.zeros((t, e), device=x.device).scatter_(1, order, share).T[:, :, None]
        gate, up, down = (_dequant(st["w_" + n], st["s_" + n]) for n in ("gate", "up", "down"))
    y = ((_act(rows @ gate, st["act"]) * (rows @ up)) @ down) * share
    y = y.reshape(t, st["top"], -1).sum(1) if t * st["top"] < e else y.sum(0)
    return (y + st["r"].float() if st["r"] is not None else y).half()


# ---------------------------------------------------------------------------------------------- in 64 bits
def _act64(y, name):
    if name == "relu":
        return y.clamp(min=0)
    if name == "gelu":
        return y / 2 * torch.erfc(-y / math.sqrt(2.0))
    if name == "gelu_tanh":
        return y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y / (1 + torch.exp(-y)) if name == "silu" else y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "experts":
        return _experts64(case, st)
    x = st["x"].double()
    if case["dtype"] == "int8":
        scale = st["xs"].double()
    else:
        most = torch.maximum(x.amax(1), -x.amin(1))
        x = torch.round(x * 127 / torch.where(most > 0, most, 1.0)[:, None])
        scale = most / 127
    if case["op"] == "quantize":
        return {"q": x.to(torch.int8), "scale": scale}
    y = x @ st["w"].double().T.contiguous()
    y *= scale[:, None]
    y *= st["ws"].double()
    if case["bias"]:
        y += st["b"].double()
    y = _act64(y, case["act"])
    return y + st["r"].double() if case["residual"] else y


def _experts64(case, st):
    t, e = case["t"], case["experts"]

    def weight(name, i):
        w = st["w_" + name][i].long()
        parts = [((w >> (4 * j)) + 8) % 16 - 8 for j in range(8)]
        return torch.stack(parts, 1).flatten(0, 1).double() * st["s_" + name][i].double().repeat_interleave(GROUP, 0)

    x = st["x"].double()
    z = x @ st["router"].double().T.contiguous()
    rows = z.cpu().tolist()
    y = st["r"].double() if case["residual"] else torch.zeros((t, case["hidden"]), dtype=torch.float64, device=x.device)
    wants = [[] for _ in range(e)]
    for i, row in enumerate(rows):
        best = sorted(range(e), key=lambda j: (-row[j], j))[:case["top"]]
        part = [math.exp(row[j] - row[best[0]]) for j in (best if case["normalize"] else range(e))]
        for j in best:
            wants[j].append((i, math.exp(row[j] - row[best[0]]) / math.fsum(part)))
    for j, want in enumerate(wants):
        if want:
            at = torch.tensor([i for i, _ in want], device=x.device)
            share = torch.tensor([p for _, p in want], device=x.device, dtype=torch.float64)
            h = _act64(x[at] @ weight("gate", j), case["act"]) * (x[at] @ weight("up", j))
            y.index_add_(0, at, (h @ weight("down", j)) * share[:, None])
    return y
