"""The operators that stand between a decoder layer's 1-bit products, as they are timed and checked.

A layer of a 1-bit decoder adds the residual, norms and quantizes an
activation (``add_rms_norm``), multiplies it with the packed q, k and v
weights and their requests' low-rank adapters (``lora_add``), rotates q and k
and puts k and v into a paged cache (``rope_append``) and lets the new tokens
attend to that cache (``paged_attention``).  ``listed`` and ``draw`` give cases
of each, ``prepare`` a case's inputs, ``run`` one call: the plain form, in
elementary torch operations on 32-bit values, or (``own``) the library's.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # One decode step of one user: the hidden state of a single token, whose launch is all latency.
        dict(name="norm-1", op="norm", nvec=1, n=4096, dtype="f32", y=False),
        # 64 sequences decode together, 16-bit hidden states; the adapters need the float values too.
        dict(name="norm-64", op="norm", nvec=64, n=4096, dtype="bf16", y=True),
        # A long prompt's hidden states, a width that is no multiple of the launch's, f32 as the products give them.
        dict(name="norm-prompt", op="norm", nvec=8191, n=4128, dtype="f32", y=False),
        # 64 sequences write one token each.
        dict(name="rope-64", op="rope", batch=64, new=1, kv=4096, hq=32, hkv=8, dim=128, page=16, dtype="bf16",
             pairs=False, lens=1),
        # Prompts of different lengths enter the cache: 64-wide heads, neighbouring pairs rotated.
        dict(name="rope-prompts", op="rope", batch=7, new=2048, kv=5000, hq=32, hkv=8, dim=64, page=64, dtype="f16",
             pairs=True, lens=2),
        # One user's next token over a long conversation: few rows, one long axis.
        dict(name="attend-1", op="attend", batch=1, new=1, kv=8191, hq=32, hkv=8, dim=128, page=16, dtype="bf16",
             lens=3),
        # The next token of 64 users with caches of all lengths: the cache is read once, 2 GB of it.
        dict(name="attend-64", op="attend", batch=64, new=1, kv=16384, hq=32, hkv=8, dim=128, page=16, dtype="bf16",
             lens=4),
        # A chunk of a long prompt over what came before it: matrix products decide.
        dict(name="attend-chunk", op="attend", batch=1, new=2048, kv=16001, hq=32, hkv=8, dim=128, page=64,
             dtype="bf16", lens=5),
        # A mixed batch, some requests a few tokens and some hundreds, one head of k and v per head of q.
        dict(name="attend-mixed", op="attend", batch=16, new=509, kv=3001, hq=16, hkv=16, dim=64, page=32, dtype="f16",
             lens=6),
        # One request's adapter beside the o projection: latency.
        dict(name="lora-1", op="lora", nvec=1, n=4096, rows=4096, rank=16, adapters=8, run=1, dtype="bf16", lens=7),
        # 64 requests, most with an adapter of their own, beside the gate projection; ranks differ.
        dict(name="lora-64", op="lora", nvec=64, n=4096, rows=14336, rank=64, adapters=48, run=1, dtype="f16", lens=8),
        # Tokens of a few prompts, each in one piece, beside the down projection.
        dict(name="lora-prompts", op="lora", nvec=1000, n=14336, rows=4096, rank=32, adapters=6, run=170, dtype="bf16",
             lens=9),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n if n != 3072 else n - 1


def draw(rng):
    """One more case of the ranges above, at most as costly as the largest listed ones."""
    op = rng.choice(["norm", "rope", "attend", "attend", "lora"])
    if op == "norm":
        n = 32 * rng.choice([_spread(rng, 4, 95), _spread(rng, 97, 448)])
        return dict(op=op, nvec=_spread(rng, 1, max(1, min(8191, 8191 * 4128 // n))), n=n,
                    dtype=rng.choice(["f32", "bf16", "f16"]), y=rng.random() < 0.5)
    if op == "lora":
        n = 8 * rng.choice([_spread(rng, 64, 383), _spread(rng, 385, 1792)])
        rows = _spread(rng, 512, 14336)
        rank = 8 * rng.randint(1, 8)
        nvec = _spread(rng, 1, max(1, min(1000, 1000 * 32 * 18432 // (rank * (n + rows)))))
        return dict(op=op, nvec=nvec, n=n, rows=rows, rank=rank, adapters=rng.randint(1, 64),
                    run=rng.choice([1, 1, 2, 50, 170]), dtype=rng.choice(["bf16", "f16"]), lens=rng.randint(10, 1 << 20))
    dim, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
    case = dict(op=op, batch=_spread(rng, 1, 64), new=1 if rng.random() < 0.4 else _spread(rng, 2, 2048),
                kv=_spread(rng, 16, 16384), hq=hq, hkv=hkv, dim=dim, page=page, dtype=rng.choice(["bf16", "f16"]))
    if op == "rope":
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


def _adapter_of(c):
    """Per token: its adapter, or -1; `run` consecutive tokens are of one request."""
    r = random.Random(c["lens"])
    ids = [r.choice([-1] + list(range(c["adapters"])) * 2) for _ in range(c["nvec"] // c["run"] + 1)]
    ids[0] = c["adapters"] - 1
    return [ids[v // c["run"]] for v in range(c["nvec"])]


def _ranks(c):
    r = random.Random(c["lens"] + 1)
    return [c["rank"]] + [max(1, c["rank"] // r.choice([1, 1, 2, 4])) for _ in range(c["adapters"] - 1)]


# ----------------------------------------------------------------- inputs --
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
    if c["op"] == "norm":
        x = normal(c["nvec"], c["n"])
        x[torch.rand(x.shape, generator=g, device=dev) < 0.01] *= 20  # hidden states have outliers
        s.update(x=x.to(t), residual=normal(c["nvec"], c["n"], std=2.0, dtype=t), weight=1 + normal(c["n"], std=0.2),
                 residual_out=torch.empty(c["nvec"], c["n"], dtype=t, device=dev))
        return s
    if c["op"] == "lora":
        s.update(x=normal(c["nvec"], c["n"]), base=normal(c["nvec"], c["rows"]),
                 a=normal(c["adapters"], c["rank"], c["n"], std=c["n"] ** -0.5, dtype=t),
                 b=normal(c["adapters"], c["rows"], c["rank"], std=0.3, dtype=t),
                 scale=torch.rand(c["adapters"], generator=g, device=dev) + 0.5,
                 ranks=whole(_ranks(c)), index=whole(_adapter_of(c)))
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
    shape = (pages, c["page"], c["hkv"], c["dim"])
    s.update(cache_k=normal(*shape, dtype=t), cache_v=normal(*shape, dtype=t), table=table, kv_len=whole(kv),
             cu_q=whole(np.cumsum([0] + new).tolist()))
    total = sum(new)
    if c["op"] == "attend":
        s.update(q=normal(total, c["hq"], c["dim"], dtype=t))
        return s
    angle = (np.arange(max(kv))[:, None] * 10000.0 ** (-np.arange(0, c["dim"], 2) / c["dim"]))
    s.update(q=normal(total, c["hq"] * c["dim"]), k=normal(total, c["hkv"] * c["dim"]),
             v=normal(total, c["hkv"] * c["dim"]),
             cos_sin=torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).to(dev))
    return s


# ------------------------------------------------------------- plain forms --
def _plain_norm(s):
    c = s["case"]
    h = s["x"].float() + s["residual"].float()
    y = h * (1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)) * s["weight"]
    b = y.view(c["nvec"], c["n"] // 32, 32)
    d = b.abs().amax(-1, keepdim=True) / 127
    t = b * torch.where(d != 0, 1 / d, 0)
    low = t.abs().floor()
    q = torch.sign(t) * (low + (t.abs() - low >= 0.5))  # half away from zero
    out = dict(residual=h.to(s["x"].dtype), values=(q * d.half().float()).half().view(c["nvec"], c["n"]))
    if c["y"]:
        out["y"] = y.to(s["x"].dtype)
    return out


def _sequence_of(s, total):
    """Per token: its sequence, and its position there."""
    token = torch.arange(total, device=s["cu_q"].device)
    seq = torch.searchsorted(s["cu_q"], token, right=True) - 1
    return seq, s["kv_len"][seq] - s["cu_q"][seq + 1] + token


def _plain_rope(s):
    c = s["case"]
    total, half = s["q"].shape[0], c["dim"] // 2
    seq, pos = _sequence_of(s, total)
    cos, sin = s["cos_sin"][pos, None, :half], s["cos_sin"][pos, None, half:]

    def rotate(x, heads):
        x = x.view(total, heads, c["dim"])
        a, b = (x[..., 0::2], x[..., 1::2]) if c["pairs"] else (x[..., :half], x[..., half:])
        u, v = a * cos - b * sin, b * cos + a * sin
        return (torch.stack([u, v], -1).flatten(-2) if c["pairs"] else torch.cat([u, v], -1)).to(s["cache_k"].dtype)

    page, slot = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    s["cache_k"][page, slot] = rotate(s["k"], c["hkv"])
    s["cache_v"][page, slot] = s["v"].view(total, c["hkv"], c["dim"]).to(s["cache_v"].dtype)
    return dict(q=rotate(s["q"], c["hq"]), k=s["cache_k"], v=s["cache_v"])


def _plain_attend(s):
    c = s["case"]
    total, group, rows = s["q"].shape[0], c["hq"] // c["hkv"], c["new"]
    seq, pos = _sequence_of(s, total)
    row = torch.arange(total, device=seq.device) - s["cu_q"][seq]
    q = torch.zeros(c["batch"], rows, c["hkv"], group, c["dim"], device=seq.device)
    q[seq, row] = s["q"].float().view(total, c["hkv"], group, c["dim"])
    q = q.permute(0, 2, 1, 3, 4).reshape(c["batch"], c["hkv"], rows * group, c["dim"])
    k = s["cache_k"][s["table"]].flatten(1, 2)[:, :c["kv"]].float().permute(0, 2, 3, 1)
    v = s["cache_v"][s["table"]].flatten(1, 2)[:, :c["kv"]].float().transpose(1, 2)
    p = torch.matmul(q, k).mul_(c["dim"] ** -0.5).view(c["batch"], c["hkv"], rows, group, c["kv"])
    last = torch.full((c["batch"], rows), -1, dtype=torch.int64, device=seq.device)
    last[seq, row] = pos
    seen = torch.arange(c["kv"], device=seq.device) <= last[:, :, None]
    p.masked_fill_(~seen[:, None, :, None], -1e30)
    p = p.sub_(p.amax(-1, keepdim=True)).exp_().view(c["batch"], c["hkv"], rows * group, c["kv"])
    o = torch.matmul(p, v).div_(p.sum(-1, keepdim=True))
    o = o.view(c["batch"], c["hkv"], rows, group, c["dim"]).transpose(1, 2)
    return o[seq, row].reshape(total, c["hq"], c["dim"]).to(s["q"].dtype)


def _plain_lora(s):
    c = s["case"]
    at = s["index"].clamp(min=0).long()
    t = torch.matmul(s["a"][at].float(), s["x"][:, :, None])
    live = (torch.arange(c["rank"], device=at.device) < s["ranks"][at, None]) & (s["index"] >= 0)[:, None]
    t = t * (live * s["scale"][at, None])[:, :, None]
    return s["base"] + torch.matmul(s["b"][at].float(), t)[:, :, 0]


# -------------------------------------------------------------------- run --
def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "rope": _plain_rope, "attend": _plain_attend, "lora": _plain_lora}[c["op"]](s)
    from decode_q1_gemv_gb300 import binding

    if c["op"] == "norm":
        r = binding.add_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["residual_out"],
                                 out="both" if c["y"] else "q8")
        # the quants with their scales, as the values they stand for
        values = (r.q.view(c["nvec"], -1, 32) * r.d.view(torch.float16)[:, :, None]).view(c["nvec"], c["n"])
        out = dict(residual=r.residual, values=values)
        if c["y"]:
            out["y"] = r.y
        return out
    if c["op"] == "rope":
        q = binding.rope_append(s["q"], s["k"], s["v"], s["cos_sin"], s["cache_k"], s["cache_v"], s["table"],
                                s["kv_len"], s["cu_q"], interleaved=c["pairs"])
        return dict(q=q, k=s["cache_k"], v=s["cache_v"])
    if c["op"] == "attend":
        return binding.paged_attention(s["q"], s["cache_k"], s["cache_v"], s["table"], s["kv_len"], s["cu_q"],
                                       max_new=c["new"])
    return binding.lora_add(s["x"], s["a"], s["b"], s["index"], s["scale"], ranks=s["ranks"], base=s["base"])


# ------------------------------------------------------------------- work --
def work(case):
    c = case
    e = BYTES[c["dtype"]]
    if c["op"] == "norm":
        m = c["nvec"] * c["n"]
        return dict(bytes=m * (3 * e + 1 + (e if c["y"] else 0)) + m // 16 + 4 * c["n"], flops=m * 8)
    if c["op"] == "lora":
        index, ranks = _adapter_of(c), _ranks(c)
        used = sum(ranks[a] for a in set(index) if a >= 0)
        each = sum(ranks[a] for a in index if a >= 0)
        return dict(bytes=4 * c["nvec"] * (c["n"] + 2 * c["rows"]) + e * used * (c["n"] + c["rows"]),
                    flops=2 * each * (c["n"] + c["rows"]))
    new, kv = _lengths(c)
    if c["op"] == "rope":
        m = sum(new) * c["dim"]
        return dict(bytes=m * (c["hq"] + 2 * c["hkv"]) * (4 + e) + 4 * m, flops=3 * m * (c["hq"] + c["hkv"]))
    pairs = sum(t * k - t * (t - 1) // 2 for t, k in zip(new, kv))
    return dict(bytes=2 * e * (sum(kv) * c["hkv"] + sum(new) * c["hq"]) * c["dim"], flops=4 * pairs * c["hq"] * c["dim"])


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    c, s = case, prepare(case, seed)
    f = torch.float64
    if c["op"] == "norm":
        h = s["x"].to(f) + s["residual"].to(f)
        y = h / ((h ** 2).sum(1, keepdim=True) / c["n"] + EPS) ** 0.5 * s["weight"].to(f)
        top = y.reshape(-1, 32).abs().max(1, keepdim=True).values / 127
        quants = torch.copysign(torch.floor((y.reshape(-1, 32) / top.clamp(min=1e-300)).abs() + 0.5), y.reshape(-1, 32))
        out = dict(residual=h, values=(quants * top.half().to(f)).reshape(c["nvec"], c["n"]))
        if c["y"]:
            out["y"] = y
        return out
    if c["op"] == "lora":
        out = s["base"].to(f)
        index, ranks = s["index"].tolist(), s["ranks"].tolist()
        for a in sorted(set(index) - {-1}):
            at = torch.tensor([v for v, i in enumerate(index) if i == a], device=out.device)
            t = s["x"][at].to(f) @ s["a"][a, :ranks[a]].to(f).T
            out[at] += float(s["scale"][a]) * (t @ s["b"][a, :, :ranks[a]].to(f).T)
        return out
    kv, cu, table = s["kv_len"].tolist(), s["cu_q"].tolist(), s["table"].tolist()
    if c["op"] == "rope":
        k, v = s["cache_k"].to(f), s["cache_v"].to(f)
        q = torch.empty(cu[-1], c["hq"], c["dim"], dtype=f, device=k.device)
        half = c["dim"] // 2
        first = torch.arange(0, c["dim"], 2, device=k.device) if c["pairs"] else torch.arange(half, device=k.device)
        second = first + 1 if c["pairs"] else first + half

        def turned(x, where):
            cos, sin = (s["cos_sin"][where, at:at + half].to(f)[:, None] for at in (0, half))
            y = torch.empty_like(x)
            y[..., first] = x[..., first] * cos - x[..., second] * sin
            y[..., second] = x[..., first] * sin + x[..., second] * cos
            return y

        for i in range(c["batch"]):
            a, b = cu[i], cu[i + 1]
            where = torch.arange(kv[i] - (b - a), kv[i], device=k.device)
            page = torch.tensor([table[i][p // c["page"]] for p in where.tolist()], device=k.device)
            q[a:b] = turned(s["q"][a:b].to(f).reshape(b - a, c["hq"], c["dim"]), where)
            k[page, where % c["page"]] = turned(s["k"][a:b].to(f).reshape(b - a, c["hkv"], c["dim"]), where)
            v[page, where % c["page"]] = s["v"][a:b].to(f).reshape(b - a, c["hkv"], c["dim"])
        return dict(q=q, k=k, v=v)
    if work(c)["flops"] > 8e11:
        return None
    out = torch.empty(s["q"].shape, dtype=f, device="cuda")
    for i in range(c["batch"]):
        a, b = cu[i], cu[i + 1]
        page = torch.tensor(table[i], device="cuda")
        k = s["cache_k"][page].reshape(-1, c["hkv"], c["dim"])[:kv[i]].to(f)
        v = s["cache_v"][page].reshape(-1, c["hkv"], c["dim"])[:kv[i]].to(f)
        hidden = torch.arange(kv[i], device="cuda")[None, :] > torch.arange(kv[i] - (b - a), kv[i], device="cuda")[:, None]
        for h in range(c["hq"]):
            g = h // (c["hq"] // c["hkv"])
            z = s["q"][a:b, h].to(f) @ k[:, g].T / c["dim"] ** 0.5
            out[a:b, h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v[:, g]
    return out
