"""One decoder layer around the 1-bit products: prompts, then tokens one by one.

    python -m decode_q1_gemv_gb300.layer [--prompt 300] [--sequences 4] [--steps 16] [--cache bf16|q8_0] [--vocab 32000]

The path of a layer of a 1-bit decoder, every step of it a call of the binding:
residual and norm with the q8_0 activation (add_rms_norm), the q, k and v
products (gemv_multi or gemm_small) with their requests' low-rank adapters
(lora_add), rotary positions and the cache's new entries (rope_append),
attention over the paged cache (paged_attention), the o product, the second
norm, gate and up, silu(gate) * up with its q8_0 form (gated_act), and down.

``PagedCache`` hands out pages and keeps the index tensors of the current call
on the device; of type int8 it holds keys and values as q8_0 (rope_append_q8,
paged_attention_q8, cache_read_q8).  ``DecoderLayer`` holds the packed weights,
``Head`` those of the output product, from whose logits it draws the next
tokens (sample).  The command builds one layer of the Llama-3-8B shape and a
head from seeded synthetic weights (no checkpoint is read) and times them.
"""
from __future__ import annotations

import argparse

import torch

from . import binding, synth

MAX_VECTORS = 64  # of one batched product
MAX_ADAPTED = 65535  # of one lora_add


class PagedCache:
    """Keys and values of `sequences` sequences in pages of `page_size` tokens, of
    `dtype` bf16 or f16, or int8: q8_0 quants with the f16 scales `ks` and `vs`,
    a head's tokens of a page side by side."""

    def __init__(self, sequences: int, pages: int, page_size: int, kv_heads: int, dim: int, max_tokens: int,
                 dtype=torch.bfloat16, device="cuda"):
        self.page_size = page_size
        self.quantized = dtype == torch.int8
        if self.quantized:
            if dim % 32:
                raise ValueError("a q8_0 cache's dim is a multiple of 32")

            def storage(last, dtype):
                return torch.empty((pages, kv_heads, page_size, last), dtype=dtype, device=device).transpose(1, 2)

            self.k, self.v = storage(dim, torch.int8), storage(dim, torch.int8)
            self.ks, self.vs = storage(dim // 32, torch.float16), storage(dim // 32, torch.float16)
        else:
            self.k = torch.empty((pages, page_size, kv_heads, dim), dtype=dtype, device=device)
            self.v = torch.empty_like(self.k)
        width = -(-max_tokens // page_size)
        self.table = torch.zeros((sequences, width), dtype=torch.int32, device=device)
        self.kv_len = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.new_start = torch.zeros(sequences + 1, dtype=torch.int32, device=device)
        self.lengths = [0] * sequences
        self.pages = [[] for _ in range(sequences)]
        self.free = list(range(pages))
        self.max_new = 0

    def extend(self, new) -> None:
        """Room for new[i] more tokens of sequence i: the next call's new tokens."""
        if len(new) != len(self.lengths):
            raise ValueError("one count of new tokens a sequence")
        if min(new) < 0:
            raise ValueError("a count of new tokens is below zero")
        need = [-(-(n + m) // self.page_size) - len(p) for n, m, p in zip(self.lengths, new, self.pages)]
        if any(n + m > self.table.shape[1] * self.page_size for n, m in zip(self.lengths, new)):
            raise ValueError("a sequence outgrows its table")
        if sum(max(n, 0) for n in need) > len(self.free):
            raise ValueError("the cache has no free pages left")
        for i, n in enumerate(need):
            if n > 0:
                first = len(self.pages[i])
                self.pages[i] += [self.free.pop() for _ in range(n)]
                self.table[i, first:first + n] = torch.tensor(self.pages[i][first:], dtype=torch.int32)
        self.lengths = [n + m for n, m in zip(self.lengths, new)]
        starts = [0]
        for m in new:
            starts.append(starts[-1] + m)
        self.kv_len.copy_(torch.tensor(self.lengths, dtype=torch.int32))
        self.new_start.copy_(torch.tensor(starts, dtype=torch.int32))
        self.max_new = max(new)

    def release(self, sequence: int) -> None:
        """Sequence `sequence` is empty and its pages are free: the next extend may
        hand them out (work on the current stream that reads them comes before).
        Its row of the table keeps old entries, which no call reads."""
        self.free += self.pages[sequence]
        self.pages[sequence] = []
        self.lengths[sequence] = 0
        self.kv_len.copy_(torch.tensor(self.lengths, dtype=torch.int32))
        self.new_start.zero_()  # nothing is new until the next extend
        self.max_new = 0

    def args(self):
        """The cache's tensors as rope_append and paged_attention take them, or their q8_0 forms."""
        if self.quantized:
            return self.k, self.v, self.ks, self.vs, self.table, self.kv_len, self.new_start
        return self.k, self.v, self.table, self.kv_len, self.new_start

    def read(self, sequence: int, dtype=torch.float32):
        """Keys and values [tokens, kv_heads, dim] of a sequence, a copy of type `dtype`."""
        n = self.lengths[sequence]
        if n == 0:
            return tuple(torch.empty((0, *self.k.shape[2:]), dtype=dtype, device=self.k.device) for _ in range(2))
        row = slice(sequence, sequence + 1)
        if self.quantized:
            whole = torch.tensor([0, n], dtype=torch.int32, device=self.k.device)
            return binding.cache_read_q8(self.k, self.v, self.ks, self.vs, self.table[row], self.kv_len[row], whole, n, dtype=dtype)
        pages = self.table[sequence, :len(self.pages[sequence])].long()
        return tuple(t[pages].flatten(0, 1)[:n].to(dtype) for t in (self.k, self.v))


class DecoderLayer:
    """blocks: Q1_0 blocks (uint8 [rows, n/128, 18]) of q, k, v, o, gate, up and
    down; norms: two f32 [hidden] weights; cos_sin: f32 [positions, rot];
    adapters: {product: (a, b, scale)} or {product: (a, b, scale, ranks)} of
    low-rank adapters, or None; ranks int32 [adapters] are the ranks in use."""

    PRODUCTS = ("q", "k", "v", "o", "gate", "up", "down")

    def __init__(self, blocks: dict, norms, cos_sin: torch.Tensor, dim: int = 128, adapters: dict | None = None,
                 eps: float = 1e-5):
        self.shape = {p: (blocks[p].shape[0], blocks[p].shape[1] * 128) for p in self.PRODUCTS}
        self.packed = {p: binding.pack(blocks[p], *self.shape[p]) for p in self.PRODUCTS}
        self.norms, self.cos_sin, self.dim, self.eps = norms, cos_sin, dim, eps
        self.adapters = adapters or {}

    def _products(self, names, q, d):
        """The named products of one quantized activation [tokens, n]."""
        tokens = q.shape[0]
        out = [torch.empty((tokens, self.shape[p][0]), dtype=torch.float32, device=q.device) for p in names]
        if tokens == 1:  # all of them in one launch
            binding.gemv_multi([(self.packed[p], *self.shape[p], None, q[0], d[0], o[0]) for p, o in zip(names, out)])
            return out
        for p, o in zip(names, out):
            for t in range(0, tokens, MAX_VECTORS):
                e = min(tokens, t + MAX_VECTORS)
                binding.gemm_small(self.packed[p], *self.shape[p], q[t:e], d[t:e], o[t:e])
        return out

    def _adapt(self, name, x, out, index):
        if name in self.adapters and index is not None:
            a, b, scale, *ranks = self.adapters[name]
            for t in range(0, x.shape[0], MAX_ADAPTED):
                e = t + MAX_ADAPTED
                binding.lora_add(x[t:e], a, b, index[t:e], scale, *ranks, out=out[t:e])
        return out

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None, cache: PagedCache,
                 index: torch.Tensor | None = None):
        """x, residual f32 [tokens, hidden] (the new tokens of all sequences,
        packed as cache.extend was told); index int32 [tokens]: each token's
        adapter.  Returns the layer's output and the residual it is added to."""
        adapted = bool(self.adapters) and index is not None
        n = binding.add_rms_norm(x, self.norms[0], self.eps, residual=residual, out="both" if adapted else "q8")
        residual = x if residual is None else n.residual
        q, k, v = self._products(("q", "k", "v"), n.q, n.d)
        for name, out in (("q", q), ("k", k), ("v", v)):
            self._adapt(name, n.y, out, index)
        if cache.quantized:
            heads = binding.rope_append_q8(q, k, v, self.cos_sin, *cache.args())
            a = binding.paged_attention_q8(heads, *cache.args(), max_new=cache.max_new)
        else:
            heads = binding.rope_append(q, k, v, self.cos_sin, *cache.args())
            a = binding.paged_attention(heads, *cache.args(), max_new=cache.max_new)
        a = a.view(a.shape[0], -1).float()
        out, = self._products(("o",), *binding.quantize(a))
        self._adapt("o", a, out, index)
        n = binding.add_rms_norm(out, self.norms[1], self.eps, residual=residual, out="both" if adapted else "q8")
        gate, up = self._products(("gate", "up"), n.q, n.d)
        self._adapt("gate", n.y, gate, index)
        self._adapt("up", n.y, up, index)
        h = binding.gated_act(gate, up, out="both" if adapted and "down" in self.adapters else "q8")
        out, = self._products(("down",), h.q, h.d)
        return self._adapt("down", h.y, out, index), n.residual


class Head:
    """blocks: Q1_0 blocks (uint8 [vocab, n/128, 18]) of the output product; norm: f32 [n]."""

    def __init__(self, blocks: torch.Tensor, norm: torch.Tensor, eps: float = 1e-5):
        self.vocab, self.n = blocks.shape[0], blocks.shape[1] * 128
        self.packed, self.norm, self.eps = binding.pack(blocks, self.vocab, self.n), norm, eps

    def logits(self, x: torch.Tensor, residual: torch.Tensor | None) -> torch.Tensor:
        """f32 [tokens, vocab] of the last layer's output and residual [tokens, n]."""
        n = binding.add_rms_norm(x, self.norm, self.eps, residual=residual)
        out = torch.empty((x.shape[0], self.vocab), dtype=torch.float32, device=x.device)
        if x.shape[0] == 1:
            binding.gemv(self.packed, self.vocab, self.n, n.q[0], n.d[0], out[0])
            return out
        for t in range(0, x.shape[0], MAX_VECTORS):
            e = min(x.shape[0], t + MAX_VECTORS)
            binding.gemm_small(self.packed, self.vocab, self.n, n.q[t:e], n.d[t:e], out[t:e])
        return out

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None, uniform: torch.Tensor, **settings) -> torch.Tensor:
        """The next token (int32) of each row of x, drawn with uniform f32 [rows]; settings as of sample."""
        return binding.sample(self.logits(x, residual), uniform, **settings)


def rope_table(positions: int, dim: int, theta: float = 500000.0, device="cuda") -> torch.Tensor:
    """f32 [positions, dim]: cosines then sines of position * theta^(-2i/dim)."""
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * theta ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def synthetic_layer(shapes=synth.LLAMA3_8B_LAYER, dim: int = 128, positions: int = 8192, adapters: int = 0, rank: int = 16,
                    seed: int = 5) -> DecoderLayer:
    """A layer of seeded synthetic weights; with `adapters`, that many of rank
    `rank` beside q and v.  Block scales are 1/sqrt(n), which keeps the
    activations' magnitude from product to product."""
    blocks, sizes = {}, {name: (rows, n) for name, rows, n in shapes}
    for i, (name, (rows, n)) in enumerate(sizes.items()):
        b = synth.weight_blocks(synth.rng_for(seed, i), rows, n, "ones")
        b[:, :, :2] = synth.fp16_bits([n ** -0.5]).view("uint8")
        blocks[name] = torch.from_numpy(b).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    hidden = sizes["q"][1]
    low = {p: (normal(adapters, rank, sizes[p][1], std=sizes[p][1] ** -0.5, dtype=torch.bfloat16),
               normal(adapters, sizes[p][0], rank, std=0.1, dtype=torch.bfloat16),
               torch.ones(adapters, device="cuda")) for p in ("q", "v")} if adapters else None
    return DecoderLayer(blocks, [1 + normal(hidden, std=0.1) for _ in range(2)], rope_table(positions, dim), dim, low)


def synthetic_head(vocab: int, hidden: int, seed: int = 6) -> Head:
    """A head of seeded synthetic weights."""
    b = synth.weight_blocks(synth.rng_for(seed, 0), vocab, hidden, "ones")
    b[:, :, :2] = synth.fp16_bits([2 * hidden ** -0.5]).view("uint8")
    return Head(torch.from_numpy(b).cuda(), torch.ones(hidden, device="cuda"))


def main() -> None:
    ap = argparse.ArgumentParser(description="One decoder layer and a head: prompts, then tokens one by one.")
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--cache", choices=("bf16", "q8_0"), default="bf16")
    ap.add_argument("--vocab", type=int, default=32000)
    args = ap.parse_args()
    layer = synthetic_layer(adapters=3)
    hidden, dim = layer.shape["q"][1], layer.dim
    head = synthetic_head(args.vocab, hidden)
    most = args.prompt + args.steps
    cache = PagedCache(args.sequences, args.sequences * (-(-most // 16)), 16, layer.shape["k"][0] // dim, dim, most,
                       torch.int8 if args.cache == "q8_0" else torch.bfloat16)
    of = torch.arange(args.sequences, dtype=torch.int32, device="cuda") % 4 - 1  # one sequence in four has no adapter

    def run(new):
        cache.extend([new] * args.sequences)
        x = torch.randn(new * args.sequences, hidden, device="cuda")
        start, end, drawn = (torch.cuda.Event(enable_timing=True) for _ in range(3))
        start.record()
        out, residual = layer(x, None, cache, of.repeat_interleave(new))
        end.record()
        last = slice(new - 1, None, new)  # of each sequence
        tokens = head(out[last], residual[last], torch.rand(args.sequences, device="cuda"), temperature=0.8, top_k=50, top_p=0.95)
        drawn.record()
        torch.cuda.synchronize()
        assert torch.isfinite(out).all() and torch.isfinite(residual).all() and binding.device_status() == 0
        assert ((tokens >= 0) & (tokens < args.vocab)).all()
        return start.elapsed_time(end), end.elapsed_time(drawn), tokens.tolist()

    layer_ms, head_ms, tokens = run(args.prompt)
    print(f"prompt: {args.sequences} x {args.prompt} tokens, {layer_ms:.3f} ms, head {head_ms:.3f} ms (first call), next {tokens}")
    times = [run(1)[:2] for _ in range(args.steps)]
    layer_ms, head_ms = (sorted(t)[len(times) // 2] for t in zip(*times))
    print(f"steps: {args.sequences} tokens each, median {layer_ms:.3f} ms, head {head_ms:.3f} ms of {args.steps}")


if __name__ == "__main__":
    main()
