"""More operators of a 1-bit decoder's step, as they are timed and checked.

Keys and values are held as q8_0 in the paged cache (``rope_append_q8`` writes
them, ``cache_read_q8`` reads them back, ``paged_attention_q8`` attends to
them), the gated activation between the up and the down product gives the down
product's q8_0 input (``gated_act``), and the next token is drawn from the
output product's logits (``sample``).  ``listed`` and ``draw`` give cases of
each, ``prepare`` a case's inputs, ``run`` one pass: the plain form, in
elementary torch operations, or (``own``) the library's.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
Q8 = 1 + 2 / 32  # bytes of a q8_0 value: its quant, and its part of a block's scale


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # 64 sequences write one token each and read it back: latency.
        dict(name="cache-64", op="cache", batch=64, new=1, kv=4096, hq=32, hkv=8, dim=128, page=16, dtype="bf16",
             pairs=False, lens=1),
        # Prompts of different lengths enter the cache: 64-wide heads, neighbouring pairs rotated.
        dict(name="cache-prompts", op="cache", batch=7, new=2048, kv=5000, hq=32, hkv=8, dim=64, page=64, dtype="f16",
             pairs=True, lens=2),
        # One user's next token over a long conversation: few rows, one long axis.
        dict(name="attend-1", op="attend", batch=1, new=1, kv=8191, hq=32, hkv=8, dim=128, page=16, dtype="bf16",
             lens=3),
        # The next token of 64 users with caches of all lengths, 1.1 GB of keys and values: the cache is read once.
        dict(name="attend-64", op="attend", batch=64, new=1, kv=16384, hq=32, hkv=8, dim=128, page=16, dtype="bf16",
             lens=4),
        # A chunk of a long prompt over what came before it: matrix products decide.
        dict(name="attend-chunk", op="attend", batch=1, new=2048, kv=16001, hq=32, hkv=8, dim=128, page=64,
             dtype="bf16", lens=5),
        # A mixed batch, some requests a few tokens and some hundreds, one head of k and v per head of q.
        dict(name="attend-mixed", op="attend", batch=16, new=509, kv=3001, hq=16, hkv=16, dim=64, page=32, dtype="f16",
             lens=6),
        # One token between up and down: the products' outputs, the down product's input.
        dict(name="gate-1", op="gate", nvec=1, n=14336, dtype="f32", act="silu", q8=True, y=False),
        # A prompt's tokens, an odd number of them.
        dict(name="gate-prompt", op="gate", nvec=4095, n=14336, dtype="f32", act="silu", q8=True, y=False),
        # 16-bit inputs and output, a width that is no multiple of a launch's.
        dict(name="gate-16", op="gate", nvec=2000, n=11008, dtype="bf16", act="gelu", q8=False, y=True),
        # One user's next token, the usual settings.
        dict(name="sample-1", op="sample", rows=1, vocab=128256, dtype="f32", spread=2.0, masked=False, mixed=False,
             temperature=0.8, top_k=50, top_p=0.95, min_p=0.0, lens=7),
        # 64 users, each with settings of their own, greedy ones among them.
        dict(name="sample-64", op="sample", rows=64, vocab=128256, dtype="f32", spread=2.0, masked=False, mixed=True,
             temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, lens=8),
        # Many rows of 16-bit logits, a flat distribution and a large nucleus, half of the tokens masked.
        dict(name="sample-256", op="sample", rows=256, vocab=151937, dtype="bf16", spread=1.5, masked=True, mixed=False,
             temperature=1.2, top_k=0, top_p=0.9, min_p=0.0, lens=9),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges above, at most as costly as the largest listed ones."""
    op = rng.choice(["cache", "attend", "attend", "gate", "sample", "sample"])
    if op == "gate":
        n = 32 * _spread(rng, 4, 448)
        q8 = rng.random() < 0.6
        return dict(op=op, nvec=_spread(rng, 1, max(1, 4095 * 14336 // n)), n=n, dtype=rng.choice(["f32", "bf16", "f16"]),
                    act=rng.choice(["silu", "gelu"]), q8=q8, y=not q8 or rng.random() < 0.3)
    if op == "sample":
        vocab = _spread(rng, 50, 262144)
        return dict(op=op, rows=_spread(rng, 1, max(1, min(512, 256 * 151937 // vocab))), vocab=vocab,
                    dtype=rng.choice(["f32", "bf16", "f16"]), spread=rng.choice([1.0, 2.0, 4.0]), masked=rng.random() < 0.3,
                    mixed=rng.random() < 0.5, temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.5]),
                    top_k=rng.choice([0, 0, _spread(rng, 1, 2000)]), top_p=rng.choice([1.0, 1.0, round(rng.uniform(0.3, 0.99), 3)]),
                    min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.3), 4)]), lens=rng.randint(10, 1 << 20))
    dim, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
    case = dict(op=op, batch=_spread(rng, 1, 64), new=1 if rng.random() < 0.5 else _spread(rng, 2, 2048),
                kv=_spread(rng, 16, 16384), hq=hq, hkv=hkv, dim=dim, page=page, dtype=rng.choice(["bf16", "f16"]))
    if op == "cache":
        case["pairs"] = rng.random() < 0.5
    case["lens"] = rng.randint(10, 1 << 20)
    case["kv"] = max(case["kv"], case["new"])
    while _too_much(case):
        big = max(("batch", case["batch"] * 256), ("new", case["new"]), ("kv", case["kv"]), key=lambda p: p[1])[0]
        case[big] = max(1, case[big] * 5 // 7)
        case["kv"] = max(case["kv"], case["new"])
    return case


def _too_much(c):
    cache = c["batch"] * c["kv"] * c["hkv"] * c["dim"]                  # k and v values at the longest lengths
    scores = c["batch"] * c["new"] * c["kv"] * c["hq"]
    return (cache > 64 * 16384 * 8 * 128 or scores > 2048 * 16001 * 32 or scores * c["dim"] > 2048 * 16001 * 32 * 128 or
            c["batch"] * c["new"] * c["hq"] * c["dim"] > 7 * 2048 * 32 * 64)


def _lengths(c):
    """Per sequence: new tokens and cached tokens, the new ones among them.  The first has the largest of both."""
    r = random.Random(c["lens"])
    new = [c["new"]] + [_spread(r, 1, c["new"]) for _ in range(c["batch"] - 1)]
    kv = [c["kv"]] + [r.randint(t, c["kv"]) for t in new[1:]]
    return new, kv


def _settings(c):
    """Per row: temperature, top_k, top_p, min_p; the case's, or (mixed) what different users ask for."""
    one = (c["temperature"], c["top_k"], c["top_p"], c["min_p"])
    if not c["mixed"]:
        return [one] * c["rows"]
    r = random.Random(c["lens"])
    return [one] + [(r.choice([0.0, 0.6, 0.8, 1.0, 1.3]), r.choice([0, 0, 20, 50, 200]), r.choice([1.0, 0.9, 0.95]),
                     r.choice([0.0, 0.0, 0.05])) for _ in range(c["rows"] - 1)]


# ----------------------------------------------------------------- inputs --
def _quantized(x):
    """The q8_0 form of x's last axis in blocks of 32: quants, and the blocks' 16-bit scales."""
    b = x.unflatten(-1, (x.shape[-1] // 32, 32))
    d = b.abs().amax(-1, keepdim=True) / 127
    t = b * torch.where(d != 0, 1 / d, 0)
    low = t.abs().floor()
    q = torch.sign(t) * (low + (t.abs() - low >= 0.5))  # half away from zero
    return q.flatten(-2).to(torch.int8), d.squeeze(-1).half()


def _values(q, d):
    return (q.unflatten(-1, (q.shape[-1] // 32, 32)).float() * d.float()[..., None]).flatten(-2)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = TYPES[c["dtype"]]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev).mul_(std).to(dtype)

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    s = dict(case=c)
    if c["op"] == "gate":
        s.update(gate=normal(c["nvec"], c["n"], std=2.0, dtype=t), up=normal(c["nvec"], c["n"], dtype=t))
        return s
    if c["op"] == "sample":
        x = normal(c["rows"], c["vocab"], std=c["spread"])
        # what the context makes likely stands out, a few tokens most
        likely = torch.randint(c["vocab"], (c["rows"], 30), generator=g, device=dev)
        x.scatter_add_(1, likely, torch.rand(likely.shape, generator=g, device=dev) * 4 * c["spread"])
        if c["masked"]:
            x.masked_fill_(torch.rand(x.shape, generator=g, device=dev) < 0.5, -math.inf)
            x[:, seed % c["vocab"]] = 0.5
        temperature, top_k, top_p, min_p = zip(*_settings(c))
        s.update(logits=x.to(t), uniform=torch.rand(c["rows"], generator=g, device=dev))
        if c["mixed"]:
            s.update(temperature=torch.tensor(temperature, device=dev), top_k=whole(top_k), top_p=torch.tensor(top_p, device=dev),
                     min_p=torch.tensor(min_p, device=dev))
        else:
            s.update(temperature=c["temperature"], top_k=c["top_k"], top_p=c["top_p"], min_p=c["min_p"])
        return s
    new, kv = _lengths(c)
    width = -(-c["kv"] // c["page"])
    pages = sum(-(-k // c["page"]) for k in kv) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(c["batch"], width, dtype=torch.int32, device=dev)
    used = 0
    for i, k in enumerate(kv):
        m = -(-k // c["page"])
        table[i, :m] = order[used:used + m]
        used += m
    total = sum(new)
    s.update(table=table, kv_len=whole(kv), cu_q=whole(np.cumsum([0] + new).tolist()))
    # The cache, a head's tokens of a page side by side.  Some of the keys' channels are larger than the others.
    if c["op"] == "attend":
        loud = torch.where(torch.rand(c["hkv"], 1, c["dim"], generator=g, device=dev) < 0.05, 4.0, 1.0)
        k, ks = _quantized(normal(pages, c["hkv"], c["page"], c["dim"]).mul_(loud))
        v, vs = _quantized(normal(pages, c["hkv"], c["page"], c["dim"]))
    else:
        k, v = (torch.zeros(pages, c["hkv"], c["page"], c["dim"], dtype=torch.int8, device=dev) for _ in range(2))
        ks, vs = (torch.zeros(pages, c["hkv"], c["page"], c["dim"] // 32, dtype=torch.float16, device=dev) for _ in range(2))
    s.update(cache_k=k.transpose(1, 2), cache_v=v.transpose(1, 2), scale_k=ks.transpose(1, 2), scale_v=vs.transpose(1, 2))
    if c["op"] == "attend":
        s.update(q=normal(total, c["hq"], c["dim"], dtype=t))
        return s
    angle = (np.arange(max(kv))[:, None] * 10000.0 ** (-np.arange(0, c["dim"], 2) / c["dim"]))
    s.update(q=normal(total, c["hq"] * c["dim"]), k=normal(total, c["hkv"] * c["dim"]),
             v=normal(total, c["hkv"] * c["dim"]),
             cos_sin=torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).to(dev))
    return s


# ------------------------------------------------------------ plain forms --
def _sequence_of(s, total):
    """Per token: its sequence, and its position there."""
    token = torch.arange(total, device=s["cu_q"].device)
    seq = torch.searchsorted(s["cu_q"], token, right=True) - 1
    return seq, s["kv_len"][seq] - s["cu_q"][seq + 1] + token


def _plain_cache(s):
    c = s["case"]
    total, half = s["q"].shape[0], c["dim"] // 2
    seq, pos = _sequence_of(s, total)
    cos, sin = s["cos_sin"][pos, None, :half], s["cos_sin"][pos, None, half:]

    def rotate(x, heads):
        x = x.view(total, heads, c["dim"])
        a, b = (x[..., 0::2], x[..., 1::2]) if c["pairs"] else (x[..., :half], x[..., half:])
        u, v = a * cos - b * sin, b * cos + a * sin
        return torch.stack([u, v], -1).flatten(-2) if c["pairs"] else torch.cat([u, v], -1)

    page, slot = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    out = dict(q=rotate(s["q"], c["hq"]).to(TYPES[c["dtype"]]))
    for name, x in (("k", rotate(s["k"], c["hkv"])), ("v", s["v"].view(total, c["hkv"], c["dim"]))):
        quants, scale = _quantized(x)
        s["cache_" + name][page, slot] = quants
        s["scale_" + name][page, slot] = scale
        out[name] = _values(quants, scale).to(TYPES[c["dtype"]])
    return out


def _plain_attend(s):
    c = s["case"]
    total, group, rows = s["q"].shape[0], c["hq"] // c["hkv"], c["new"]
    seq, pos = _sequence_of(s, total)
    row = torch.arange(total, device=seq.device) - s["cu_q"][seq]
    q = torch.zeros(c["batch"], rows, c["hkv"], group, c["dim"], device=seq.device)
    q[seq, row] = s["q"].float().view(total, c["hkv"], group, c["dim"])
    q = q.permute(0, 2, 1, 3, 4).reshape(c["batch"], c["hkv"], rows * group, c["dim"])
    k = _values(s["cache_k"][s["table"]], s["scale_k"][s["table"]]).flatten(1, 2)[:, :c["kv"]].permute(0, 2, 3, 1)
    v = _values(s["cache_v"][s["table"]], s["scale_v"][s["table"]]).flatten(1, 2)[:, :c["kv"]].transpose(1, 2)
    p = torch.matmul(q, k).mul_(c["dim"] ** -0.5).view(c["batch"], c["hkv"], rows, group, c["kv"])
    last = torch.full((c["batch"], rows), -1, dtype=torch.int64, device=seq.device)
    last[seq, row] = pos
    seen = torch.arange(c["kv"], device=seq.device) <= last[:, :, None]
    p.masked_fill_(~seen[:, None, :, None], -1e30)
    p = p.sub_(p.amax(-1, keepdim=True)).exp_().view(c["batch"], c["hkv"], rows * group, c["kv"])
    o = torch.matmul(p, v).div_(p.sum(-1, keepdim=True))
    o = o.view(c["batch"], c["hkv"], rows, group, c["dim"]).transpose(1, 2)
    return o[seq, row].reshape(total, c["hq"], c["dim"]).to(s["q"].dtype)


def _plain_gate(s):
    c = s["case"]
    x, up = s["gate"].float(), s["up"].float()
    if c["act"] == "silu":
        y = x / (1 + torch.exp(-x)) * up
    else:  # x / (1 + e^-2u) is x (1 + tanh(u)) / 2
        u = math.sqrt(2 / math.pi) * (x + 0.044715 * (x * x * x))
        y = x / (1 + torch.exp(-2 * u)) * up
    out = {}
    if c["q8"]:
        out["values"] = _values(*_quantized(y)).half()
    if c["y"]:
        out["y"] = y.to(s["gate"].dtype)
    return out


def _plain_sample(s):
    """In 64 bits: a token is drawn where long sums cross a border."""
    c = s["case"]
    temperature, top_k, top_p, min_p = (
        v.double()[:, None] if isinstance(v, torch.Tensor) else torch.full((c["rows"], 1), float(np.float32(v)), dtype=torch.float64, device="cuda")
        for v in (s["temperature"], s["top_k"], s["top_p"], s["min_p"]))
    x = s["logits"].double()
    ordered, index = torch.sort(x, dim=-1, descending=True, stable=True)
    w = torch.exp((ordered - ordered[:, :1]) / torch.where(temperature > 0, temperature, 1))
    place = torch.arange(c["vocab"], device=x.device)
    w = w * ((top_k <= 0) | (place < top_k))
    above = torch.cumsum(w, -1) - w
    enough = top_p * w.sum(-1, keepdim=True)
    keep = ((top_p >= 1) | (above < enough)) & (w >= min_p)
    keep[:, 0] = True
    w = torch.zeros_like(w).scatter_(1, index, w * keep)  # in the vocabulary's order
    sums = torch.cumsum(w, -1)
    drawn = (sums <= s["uniform"].double()[:, None] * sums[:, -1:]).sum(-1)
    return torch.where(temperature[:, 0] > 0, drawn, index[:, 0]).to(torch.int32)


# -------------------------------------------------------------------- run --
def run(state):
    s, c = state, state["case"]
    if not own:
        return {"cache": _plain_cache, "attend": _plain_attend, "gate": _plain_gate, "sample": _plain_sample}[c["op"]](s)
    from decode_q1_gemv_gb300 import binding

    if c["op"] == "cache":
        cache = (s["cache_k"], s["cache_v"], s["scale_k"], s["scale_v"], s["table"], s["kv_len"], s["cu_q"])
        q = binding.rope_append_q8(s["q"], s["k"], s["v"], s["cos_sin"], *cache, interleaved=c["pairs"], dtype=TYPES[c["dtype"]])
        k, v = binding.cache_read_q8(*cache, s["q"].shape[0], dtype=TYPES[c["dtype"]])
        return dict(q=q, k=k, v=v)
    if c["op"] == "attend":
        return binding.paged_attention_q8(s["q"], s["cache_k"], s["cache_v"], s["scale_k"], s["scale_v"], s["table"],
                                          s["kv_len"], s["cu_q"], max_new=c["new"])
    if c["op"] == "gate":
        r = binding.gated_act(s["gate"], s["up"], c["act"], out="both" if c["q8"] and c["y"] else "q8" if c["q8"] else "y")
        out = {}
        if c["q8"]:  # the quants with their scales, as the values they stand for
            out["values"] = (r.q.view(c["nvec"], -1, 32) * r.d.view(torch.float16)[:, :, None]).view(c["nvec"], c["n"])
        if c["y"]:
            out["y"] = r.y
        return out
    return binding.sample(s["logits"], s["uniform"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])


# ------------------------------------------------------------------- work --
def work(case):
    c = case
    e = BYTES[c["dtype"]]
    if c["op"] == "gate":
        m = c["nvec"] * c["n"]
        return dict(bytes=m * (2 * e + (e if c["y"] else 0)) + int(m * Q8 if c["q8"] else 0), flops=m * 12)
    if c["op"] == "sample":
        return dict(bytes=c["rows"] * (c["vocab"] * e + 8), flops=c["rows"] * c["vocab"] * 4)
    new, kv = _lengths(c)
    if c["op"] == "cache":
        m = sum(new) * c["dim"]
        return dict(bytes=int(m * (c["hq"] * (4 + e) + 2 * c["hkv"] * (4 + Q8 + Q8 + e)) + 4 * m),
                    flops=3 * m * (c["hq"] + c["hkv"]) + 8 * m * c["hkv"])
    pairs = sum(t * k - t * (t - 1) // 2 for t, k in zip(new, kv))
    return dict(bytes=int(2 * (Q8 * sum(kv) * c["hkv"] + e * sum(new) * c["hq"]) * c["dim"]),
                flops=4 * pairs * c["hq"] * c["dim"])


# ------------------------------------------------------------------ exact --
def _exact_q8(x):
    """The q8_0 values of x [..., n], in 64 bits but for the scale, which is 16 bits wide."""
    b = x.reshape(-1, 32)
    top = b.abs().max(1, keepdim=True).values / 127
    quants = torch.copysign(torch.floor((b / top.clamp(min=1e-300)).abs() + 0.5), b)
    return (quants * top.half().to(torch.float64)).reshape(x.shape)


def _exact_sample(c, s):
    logits = s["logits"].double().cpu().numpy()
    uniform = s["uniform"].double().cpu().numpy()
    out = np.empty(c["rows"], dtype=np.int32)
    for r, settings in enumerate(_settings(c)):
        t, k, p, m = (float(np.float32(v)) for v in settings)
        x = logits[r]
        best = int(np.argmax(x))  # the first of the largest
        if t <= 0:
            out[r] = best
            continue
        tokens = np.flatnonzero(x > -np.inf)
        tokens = tokens[np.argsort(-x[tokens], kind="stable")]
        if k > 0:
            tokens = tokens[:int(k)]
        w = np.exp((x[tokens] - x[best]) / t)
        if p < 1:
            count = int(np.searchsorted(np.cumsum(w), p * w.sum(), side="left")) + 1
            tokens, w = tokens[:count], w[:count]
        stay = w >= m
        stay[0] = True
        tokens, w = tokens[stay], w[stay]
        back = np.argsort(tokens)
        sums = np.cumsum(w[back])
        out[r] = tokens[back][min(len(tokens) - 1, int(np.searchsorted(sums, uniform[r] * sums[-1], side="right")))]
    return torch.from_numpy(out).cuda()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f = torch.float64
    if c["op"] == "sample":
        return _exact_sample(c, s)
    if c["op"] == "gate":
        x, up = s["gate"].to(f), s["up"].to(f)
        if c["act"] == "silu":
            y = x * torch.sigmoid(x) * up
        else:
            y = 0.5 * x * (1 + torch.tanh((2 / math.pi) ** 0.5 * (x + 0.044715 * x ** 3))) * up
        out = {}
        if c["q8"]:
            out["values"] = _exact_q8(y)
        if c["y"]:
            out["y"] = y
        return out
    kv, cu, table = s["kv_len"].tolist(), s["cu_q"].tolist(), s["table"].tolist()
    if c["op"] == "cache":
        half = c["dim"] // 2
        first = torch.arange(0, c["dim"], 2, device="cuda") if c["pairs"] else torch.arange(half, device="cuda")
        second = first + 1 if c["pairs"] else first + half

        def turned(x, heads):
            x = x.to(f).reshape(cu[-1], heads, c["dim"])
            y = torch.empty_like(x)
            for i in range(c["batch"]):
                a, b = cu[i], cu[i + 1]
                at = torch.arange(kv[i] - (b - a), kv[i], device="cuda")
                cos, sin = (s["cos_sin"][at, o:o + half].to(f)[:, None] for o in (0, half))
                y[a:b][..., first] = x[a:b][..., first] * cos - x[a:b][..., second] * sin
                y[a:b][..., second] = x[a:b][..., first] * sin + x[a:b][..., second] * cos
            return y

        return dict(q=turned(s["q"], c["hq"]), k=_exact_q8(turned(s["k"], c["hkv"])),
                    v=_exact_q8(s["v"].to(f).reshape(cu[-1], c["hkv"], c["dim"])))
    if work(c)["flops"] > 8e11:
        return None
    out = torch.empty(s["q"].shape, dtype=f, device="cuda")
    for i in range(c["batch"]):
        a, b = cu[i], cu[i + 1]
        page = torch.tensor(table[i], device="cuda")
        k, v = ((s["cache_" + x][page].to(f).reshape(-1, c["hkv"], c["dim"] // 32, 32) *
                 s["scale_" + x][page].to(f).reshape(-1, c["hkv"], c["dim"] // 32, 1)).reshape(-1, c["hkv"], c["dim"])[:kv[i]]
                for x in "kv")
        hidden = torch.arange(kv[i], device="cuda")[None, :] > torch.arange(kv[i] - (b - a), kv[i], device="cuda")[:, None]
        for h in range(c["hq"]):
            g = h // (c["hq"] // c["hkv"])
            z = s["q"][a:b, h].to(f) @ k[:, g].T / c["dim"] ** 0.5
            out[a:b, h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v[:, g]
    return out
