"""The operators between the products against plain forms in 64 bits.

Tolerances are bounds from the operators' arithmetic, not fits.  Rounding to p
significant bits is off by 2^-p of the value at most: u = 2^-24 for f32, U =
2^-8 for bf16 and 2^-11 for f16 (an f16 value below 2^-14 by 2^-25 at most).  Where an operator has an exact definition (the q8_0 form of y, cache
entries that are copied, rows that must not change) the comparison is by bits.
"""
import math

import numpy as np
import pytest
import torch

from decode_q1_gemv_gb300 import binding

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
U = {torch.float32: U32, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    binding.device_status()


def normal(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def within(got, want, tol):
    """|got - want| <= tol everywhere, and every value is a number."""
    got = got.to(F64)
    assert torch.isfinite(got).all()
    off = (got - want).abs() - tol
    assert off.max() <= 0, f"{(off > 0).sum()} of {off.numel()} values off, worst by {off.max().item():.3g}"


# ------------------------------------------------------------------- norm --
def norm_reference(x, residual, weight, eps):
    h = x.to(F64) + (residual.to(F64) if residual is not None else 0)
    return h, h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * weight.to(F64)


# The sum of squares: a chain of at most 6 groups of 8 a thread (the long form:
# n / threads), 5 butterfly steps, 32 warps; its relative error is half as
# large in the square root; then eight more roundings.
def norm_tol(n, y, dtype):
    chain = max(48, n // 256) + 5 + 32
    return (chain / 2 + 8) * U32 * y.abs() + U[dtype] * y.abs() + TINY[dtype]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nvec,n", [(1, 32), (1, 4096), (3, 96), (5, 1024), (2, 4128), (64, 4096), (7, 14336),
                                    (2, 24608), (300, 256), (1, 131072)])
def test_norm(nvec, n, dtype):
    x, r = normal(1, nvec, n, dtype=dtype), normal(2, nvec, n, std=3.0, dtype=dtype)
    w = 1 + normal(3, n, std=0.3)
    got = binding.add_rms_norm(x, w, 1e-5, residual=r, out="both")
    h, y = norm_reference(x, r, w, 1e-5)
    within(got.residual, h, (U32 + U[dtype] * (dtype != torch.float32)) * h.abs() + TINY[dtype])
    within(got.y, y, norm_tol(n, y, dtype))
    if dtype == torch.float32:  # the fused q8_0 form is that of the quantize call on y
        q, d = binding.quantize(got.y)
        assert torch.equal(q, got.q) and torch.equal(d, got.d)
    scale = got.d.view(torch.float16).to(F64).repeat_interleave(32, -1)
    # half a step (and a little of the next), the step itself off by 2^-11 of itself or 2^-25
    within(got.q.to(F64) * scale, y, 0.501 * scale + 127 * (2.0 ** -11 * scale + 2.0 ** -25) + norm_tol(n, y, torch.float32))
    only = binding.add_rms_norm(x, w, 1e-5, residual=r)
    assert only.y is None and torch.equal(only.q, got.q) and torch.equal(only.d, got.d)
    assert torch.equal(only.residual, got.residual)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 3, 7, 33, 1001, 4097])
def test_norm_odd_widths_and_strides(n, dtype):
    """Widths of no whole group and rows of any stride, without a residual."""
    x = normal(4, 5, n + 3, dtype=dtype)[:, 1:n + 1]
    w = 1 + normal(5, n, std=0.3)
    buf = torch.full((5, n + 2), 7.0, dtype=dtype, device="cuda")
    got = binding.add_rms_norm(x, w, 1e-6, out="y", y=buf[:, :n])
    _, y = norm_reference(x, None, w, 1e-6)
    within(got.y, y, norm_tol(n, y, dtype))
    assert got.residual is None and (buf[:, n:] == 7).all()


def test_norm_scalar_path_gives_the_same_bits():
    """Rows that allow no 16-byte access: the same sums in the same order."""
    x, r, w = normal(6, 4, 4096), normal(7, 4, 4096), 1 + normal(8, 4096, std=0.1)
    want = binding.add_rms_norm(x, w, residual=r, out="both")
    wide = torch.empty(4, 4099, device="cuda")
    wide[:, 1:4097] = x
    got = binding.add_rms_norm(wide[:, 1:4097], w, residual=r, out="both")
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [4096, 49152])
def test_norm_in_place_and_batch_invariant(n):
    x, r, w = normal(9, 33, n), normal(10, 33, n), 1 + normal(11, n, std=0.1)
    want = binding.add_rms_norm(x, w, residual=r, out="both")
    one = binding.add_rms_norm(x[17:18], w, residual=r[17:18], out="both")
    for a, b in zip(want, one):
        assert torch.equal(a[17:18], b)
    r2, x2 = r.clone(), x.clone()
    got = binding.add_rms_norm(x2, w, residual=r2, residual_out=r2, y=x2, out="both")
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_norm_of_zeros_and_large_values():
    x = torch.zeros(2, 64, device="cuda")
    x[1] = 1e15
    got = binding.add_rms_norm(x, torch.ones(64, device="cuda"), 1e-5, out="both")
    assert (got.q[0] == 0).all() and (got.d[0] == 0).all() and (got.y[0] == 0).all()
    within(got.y[1], torch.ones(64, dtype=F64, device="cuda"), 64 * U32)


# ------------------------------------------------------------------- lora --
def lora_reference(x, a, b, index, scale, ranks, base):
    """Values, and the sum of magnitudes that every rounding is relative to."""
    out, mag = base.to(F64).clone(), base.to(F64).abs()
    for v, i in enumerate(index.tolist()):
        if 0 <= i < a.shape[0]:
            r = a.shape[1] if ranks is None else int(ranks[i])
            s = 1.0 if scale is None else float(scale[i])
            A, B, xv = a[i, :r].to(F64), b[i, :, :r].to(F64), x[v].to(F64)
            out[v] += s * (B @ (A @ xv))
            mag[v] += abs(s) * (B.abs() @ (A.abs() @ xv.abs()))
    return out, mag


# A chain of n/8 / 256 * 8 values a lane, 5 + 3 + 8 joins, a chain of 8, 4 joins,
# the scale and the base.
def lora_tol(n, mag):
    return (n / 256 + 40) * U32 * mag


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nvec,n,rows,rank,adapters", [
    (1, 8, 1, 8, 1), (1, 4096, 4096, 16, 4), (5, 520, 333, 8, 2), (64, 1024, 1030, 64, 40), (3, 14336, 4096, 128, 2),
    (65, 2048, 515, 24, 3), (130, 264, 77, 40, 1), (17, 4104, 1000, 16, 3), (700, 128, 256, 8, 5)])
def test_lora(nvec, n, rows, rank, adapters, dtype):
    rng = np.random.default_rng(nvec + n)
    index = torch.from_numpy(rng.integers(-1, adapters, nvec).astype(np.int32)).cuda()
    ranks = torch.from_numpy(rng.integers(0, rank + 1, adapters).astype(np.int32)).cuda()
    x, base = normal(20, nvec, n), normal(21, nvec, rows)
    a, b = normal(22, adapters, rank, n, std=0.05, dtype=dtype), normal(23, adapters, rows, rank, dtype=dtype)
    scale = normal(24, adapters)
    for i in range(adapters):  # what lies past a rank may be anything
        a[i, ranks[i]:] = math.nan
        b[i, :, ranks[i]:] = math.inf
    got = binding.lora_add(x, a, b, index, scale, ranks=ranks, base=base)
    want, mag = lora_reference(x, a, b, index, scale, ranks, base)
    within(got, want, lora_tol(n, mag))
    none = (index < 0).nonzero()[:, 0]
    assert torch.equal(got[none], base[none])
    again = binding.lora_add(x, a, b, index, scale, ranks=ranks, base=base)
    assert torch.equal(got, again)
    inplace = base.clone()
    binding.lora_add(x, a, b, index, scale, ranks=ranks, out=inplace)
    assert torch.equal(got, inplace)


@pytest.mark.parametrize("count", [1, 2, 4, 5, 8, 9, 63, 64, 65, 129])
def test_lora_buckets(count):
    """Runs of one adapter of every length around a bucket and a window, no scale or ranks."""
    x, base = normal(25, count + 1, 512), normal(26, count + 1, 300)
    a, b = normal(27, 2, 16, 512, std=0.05, dtype=torch.bfloat16), normal(28, 2, 300, 16, dtype=torch.bfloat16)
    index = torch.ones(count + 1, dtype=torch.int32, device="cuda")
    index[count // 2] = 0
    got = binding.lora_add(x, a, b, index, base=base)
    want, mag = lora_reference(x, a, b, index, None, None, base)
    within(got, want, lora_tol(512, mag))


def test_lora_strided_rows_and_bad_index():
    x, wide = normal(29, 6, 600)[:, :256], normal(30, 6, 555)
    a, b = normal(31, 3, 8, 256, std=0.1, dtype=torch.float16), normal(32, 3, 501, 8, dtype=torch.float16)
    index = torch.tensor([0, 3, -1, 2, -7, 1 << 30], dtype=torch.int32, device="cuda")
    out = torch.full((6, 777), 5.0, device="cuda")
    got = binding.lora_add(x, a, b, index, base=wide[:, 3:504], out=out[:, 1:502])
    want, mag = lora_reference(x, a, b, index, None, None, wide[:, 3:504])
    within(got, want, lora_tol(256, mag))
    assert (out[:, :1] == 5).all() and (out[:, 502:] == 5).all()
    assert binding.device_status() == 2 and binding.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nvec, adapters, run, n, rows, rank", [
    (129, 16, 1, 520, 301, 24),      # buckets of sixteen, rows that start off 16 bytes
    (129, 17, 1, 520, 304, 24),      # buckets of eight
    (1100, 2, 37, 264, 132, 64),     # more than one round of windows
    (700, 90, 1, 136, 66, 8),        # more buckets than run at once
    (300, 5, 50, 2056, 516, 72),     # a rank beyond the buckets of sixteen
    (600, 1, 600, 40, 8, 16),        # slices without values and without rows
    (140, 3, 140, 1032, 1030, 56),
])
def test_lora_many_vectors(nvec, adapters, run, n, rows, rank, dtype):
    rng = np.random.default_rng(nvec + rank)
    which = np.repeat(rng.integers(-1, adapters, -(-nvec // run)), run)[:nvec].astype(np.int32)
    bad = rng.choice(nvec, 3, replace=False)
    which[bad] = [adapters, -2, 1 << 30]
    index = torch.from_numpy(which).cuda()
    ranks = torch.from_numpy(rng.integers(0, rank + 1, adapters).astype(np.int32)).cuda()
    ranks[0] = rank
    x, base = normal(33, nvec, n), normal(34, nvec, rows)
    a, b = normal(35, adapters, rank, n, std=0.05, dtype=dtype), normal(36, adapters, rows, rank, dtype=dtype)
    for i in range(adapters):
        a[i, ranks[i]:] = math.nan
        b[i, :, ranks[i]:] = math.inf
    scale = normal(37, adapters)
    got = binding.lora_add(x, a, b, index, scale, ranks=ranks, base=base)
    assert binding.device_status() == 2 and binding.device_status() == 0
    want, mag = lora_reference(x, a, b, index, scale, ranks, base)
    within(got, want, lora_tol(n, mag))
    none = ((index < 0) | (index >= adapters)).nonzero()[:, 0]
    assert torch.equal(got[none], base[none])
    assert torch.equal(got, binding.lora_add(x, a, b, index, scale, ranks=ranks, base=base))
    binding.device_status()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rank", [88, 96, 104, 120, 128])
def test_lora_high_ranks(rank, dtype):
    """x of very different sizes, up to 2^100, with ranks beyond a stage's room for sums."""
    x, base = normal(38, 9, 1416), normal(39, 9, 520)
    x *= torch.tensor([2.0 ** e for e in (0, 100, -60, 20, -20, 10, 1, 2, 3)], device="cuda")[:, None]
    a, b = normal(40, 2, rank, 1416, std=0.05, dtype=dtype), normal(41, 2, 520, rank, dtype=dtype)
    index = torch.tensor([0, 1, 1, 0, 1, 1, 1, 1, 1], dtype=torch.int32, device="cuda")
    got = binding.lora_add(x, a, b, index, base=base)
    want, mag = lora_reference(x, a, b, index, None, None, base)
    within(got, want, lora_tol(1416, mag))


# ----------------------------------------------------------------- paged --
class Cache:
    """A paged cache with random content, random pages and poison wherever no token lies."""

    least_tokens = 0  # that a row of the table covers

    def __init__(self, seqs, heads, kv_heads, dim, page, dtype, layout="token", width=None, seed=40, spare=2):
        self.new, self.len = [s[0] for s in seqs], [s[1] for s in seqs]
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in self.len]
        self.width = max(width or max(1, max(need)), -(-self.least_tokens // page))
        pages = sum(need) + spare
        order = rng.permutation(pages).astype(np.int32)
        table = rng.choice(np.array([-5, pages, 1 << 30], dtype=np.int32), (len(seqs), self.width))
        used = 0
        for i, m in enumerate(need):
            table[i, :m] = order[used:used + m]
            used += m
        shape = (pages, page, kv_heads, dim) if layout == "token" else (pages, kv_heads, page, dim)
        self.k, self.v = (torch.full(shape, math.nan, dtype=dtype, device="cuda") for _ in range(2))
        if layout == "head":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.table = torch.from_numpy(table).cuda()
        self.kv_len = torch.tensor(self.len, dtype=torch.int32, device="cuda")
        self.new_start = torch.tensor(np.cumsum([0] + self.new), dtype=torch.int32, device="cuda")
        self.total = sum(self.new)
        self.dense = []
        for i, n in enumerate(self.len):
            k, v = (normal(seed + 10 * i + j, n, kv_heads, dim, dtype=dtype) for j in (1, 2))
            self.dense.append((k, v))
            pos = torch.arange(n, device="cuda")
            at = self.table[i, pos // page].long(), pos % page
            self.k[at], self.v[at] = k, v

    def args(self):
        return self.k, self.v, self.table, self.kv_len, self.new_start


def attend_reference(c, q, scale):
    """Values, the rows' sums of |weight * v|, sums of weights relative to the largest, and visible keys."""
    out = torch.zeros(q.shape, dtype=F64, device="cuda")
    mag, total, seen = out.clone(), torch.ones(q.shape[:2], dtype=F64, device="cuda"), out[:, 0, 0].clone()
    group = q.shape[1] // c.k.shape[2]
    at = 0
    for (k, v), new, n in zip(c.dense, c.new, c.len):
        k, v = (t.to(F64).repeat_interleave(group, 1) for t in (k, v))
        for j in range(new):
            p = n - new + j + 1
            if p > 0:
                s = torch.einsum("hd,khd->hk", q[at + j].to(F64), k[:p]) * scale
                w = torch.exp(s - s.amax(1, keepdim=True))
                total[at + j] = w.sum(1)
                w = w / w.sum(1, keepdim=True)
                out[at + j] = torch.einsum("hk,khd->hd", w, v[:p])
                mag[at + j] = torch.einsum("hk,khd->hd", w, v[:p].abs())
                seen[at + j] = p
        at += new
    return out, mag, total, seen


# Each weight is rounded once for its product with v (U, or 2^-25 of the largest
# weight for a small one in f16) and the sum of the products is divided by a sum
# of unrounded ones; scores are sums of dim f32 products of magnitude
# scale * sum |q k| < 40 here, so a weight is off by 2 * dim * 40 * u at most; then the output's rounding.
def attend_tol(c, q, out, mag, total, seen):
    dtype, dim = q.dtype, q.shape[2]
    small = TINY[dtype] * seen[:, None] / total * 6  # |v| < 6
    return (U[dtype] + 80 * dim * U32) * mag + small[:, :, None] + U[dtype] * out.abs() + TINY[dtype] + 1e-6 * mag


def check_attend(c, heads, dtype, dim, max_new=None, scale=None, seed=70):
    q = normal(seed, c.total, heads, dim, dtype=dtype)
    got = binding.paged_attention(q, *c.args(), max_new=max_new or max(c.new), scale=scale)
    want = attend_reference(c, q, dim ** -0.5 if scale is None else scale)
    within(got, want[0], attend_tol(c, q, *want))
    assert binding.device_status() == 0  # no wait ran into its limit
    return q, got


TYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (4, 4), (7, 1), (32, 2)])
@pytest.mark.parametrize("length", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000])
def test_attend_one_token(length, heads, kv_heads, dim, dtype):
    check_attend(Cache([(1, length)], heads, kv_heads, dim, 16, dtype), heads, dtype, dim)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (16, 1), (32, 8), (36, 12)])
@pytest.mark.parametrize("width", [4, 8, 17, 40, 110, 200])
def test_attend_whatever_the_table_holds(width, heads, kv_heads, dim):
    """The length of the table chooses how the work is split, the lengths do not: short and full
    sequences in short and long tables, fewer units than a cluster has CTAs, nothing new, several rows."""
    full = min(width * 64, 7000)
    for seqs in ([(1, 1)], [(1, full)], [(1, 200), (0, 77), (1, full - 63)], [(0, 9)], [(3, 2), (2, 130)]):
        c = Cache(seqs, heads, kv_heads, dim, 64, torch.bfloat16, width=width)
        for max_new in {max(1, max(c.new)), 1}:
            if c.total:
                check_attend(c, heads, torch.bfloat16, dim, max_new=max_new)
            else:
                q = normal(77, 1, heads, dim, dtype=torch.bfloat16)  # a row of no sequence
                out = torch.full_like(q, 3.0)
                binding.paged_attention(q, *c.args(), max_new=max_new, out=out)
                assert (out == 3).all()
    assert binding.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 64, 128, 256])
def test_attend_ragged_batch(page, dim, dtype):
    """Single tokens, chunks, whole prompts, sequences without new tokens, lengths around pages and tiles."""
    seqs = [(1, 300), (5, 5), (0, 40), (17, 129), (1, 1), (33, 64), (2, 2000), (0, 0), (70, 70), (1, page + 1), (3, page)]
    check_attend(Cache(seqs, 8, 2, dim, page, dtype), 8, dtype, dim)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 128), (2, 2, 64), (5, 1, 128), (8, 1, 64), (3, 1, 64)])
@pytest.mark.parametrize("new,length", [(15, 200), (64, 64), (65, 700), (127, 129), (128, 128), (129, 1025), (257, 300)])
def test_attend_chunk(new, length, heads, kv_heads, dim, dtype):
    check_attend(Cache([(new, length)], heads, kv_heads, dim, 32, dtype), heads, dtype, dim)


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 16, 16), (128, 16, 4)])
def test_attend_many_items_a_cta(dim, heads, kv_heads):
    """More items than CTAs, of one and two tiles and of few rows in turn: the kernels' barriers pass
    from item to item.  No wait may have run into its limit."""
    rng = np.random.default_rng(5)
    seqs = [(int(n), int(n + rng.integers(0, 300))) for n in np.exp(rng.uniform(0, np.log(300), 40))]
    check_attend(Cache(seqs, heads, kv_heads, dim, 32, torch.float16), heads, torch.float16, dim)
    assert binding.device_status() == 0


@pytest.mark.parametrize("new,length", [(1, 0), (4, 2), (40, 10), (300, 1), (130, 129)])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_rows_that_see_nothing(new, length, dim):
    """More new tokens than cached ones: the first see no key and are zero."""
    c = Cache([(2, 9), (new, length), (1, 30)], 4, 2, dim, 16, torch.bfloat16, width=2 if length < 33 else None)
    q, got = check_attend(c, 4, torch.bfloat16, dim)
    empty = got[2:2 + new - length]
    assert empty.shape[0] == new - length and (empty == 0).all()


@pytest.mark.parametrize("width", [None, 500])
@pytest.mark.parametrize("max_new", [1 << 40, (1 << 63) - 1])
def test_attend_max_new_beyond_any_sequence(max_new, width):
    c = Cache([(1, 100), (40, 333), (7, 50)], 8, 2, 64, 16, torch.float16, width=width)
    check_attend(c, 8, torch.float16, 64, max_new=max_new)


@pytest.mark.parametrize("dim", [64, 128])
def test_attend_mixed_calls_one_after_another(dim):
    """Calls of short and long sequences back to back on one workspace, in a graph: each starts before the
    one before it has ended, and none may see the other's parts or outputs."""
    heads, calls = 16, 12
    cs = [Cache([(200, 1500), (1, 900), (3, 2500), (130, 131), (16, 40)], heads, 4, dim, 32, torch.bfloat16, seed=90 + i,
                width=250) for i in range(3)]
    qs = [normal(95 + i, cs[0].total, heads, dim, dtype=torch.bfloat16) for i in range(3)]
    ws = torch.empty(binding.paged_attention_workspace(200, heads, 4, dim), dtype=torch.uint8, device="cuda")
    want = [binding.paged_attention(q, *c.args(), max_new=200) for q, c in zip(qs, cs)]
    for q, c, w in zip(qs, cs, want):
        ref = attend_reference(c, q, dim ** -0.5)
        within(w, ref[0], attend_tol(c, q, *ref))
    outs = [torch.empty_like(qs[0]) for _ in range(calls)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(calls):
            binding.paged_attention(qs[i % 3], *cs[i % 3].args(), max_new=200, out=outs[i], workspace=ws)
    for _ in range(5):
        for o in outs:
            o.fill_(7.0)
        g.replay()
        for i, o in enumerate(outs):
            assert torch.equal(o, want[i % 3])
    assert binding.device_status() == 0


@pytest.mark.parametrize("max_new", [1, 40, 4096])
def test_attend_max_new_is_only_a_hint(max_new):
    c = Cache([(1, 100), (40, 333), (7, 50)], 8, 2, 128, 16, torch.bfloat16)
    check_attend(c, 8, torch.bfloat16, 128, max_new=max_new)


@pytest.mark.parametrize("new", [1, 100])
def test_attend_layouts_and_strides(new):
    """Heads before slots in the cache, strided q and out, rows of no sequence left alone."""
    dtype, dim, heads = torch.float16, 128, 8
    c = Cache([(new, 500), (1, 33)], heads, 2, dim, 64, dtype, layout="head")
    wide = normal(71, c.total + 3, heads + 2, dim + 8, dtype=dtype)
    q = wide[:, 1:-1, 8:]
    buf = torch.full((c.total + 3, heads, dim + 16), 9.0, dtype=dtype, device="cuda")
    got = binding.paged_attention(q, *c.args(), max_new=new, out=buf[..., 8:-8])
    want = attend_reference(c, q[:c.total].contiguous(), dim ** -0.5)
    within(got[:c.total], want[0], attend_tol(c, q[:c.total], *want))
    assert (buf[..., :8] == 9).all() and (buf[..., -8:] == 9).all() and (buf[c.total:] == 9).all()


@pytest.mark.parametrize("new", [1, 64])
def test_attend_sharp_and_growing_scores(new):
    """Large scores of both signs: one key takes all weight, and the maximum grows along the keys."""
    dtype, dim = torch.bfloat16, 128
    c = Cache([(new, 900)], 4, 1, dim, 16, dtype)
    q = normal(72, c.total, 4, dim, dtype=dtype)
    k, v = c.dense[0]
    ramp = (q[0, 0].to(F64) / q[0, 0].to(F64).norm() * torch.linspace(-20, 20, 900, dtype=F64, device="cuda")[:, None])
    k = (k.to(F64) * 0.1 + ramp[:, None]).to(dtype)
    c.dense[0] = (k, v)
    pos = torch.arange(900, device="cuda")
    c.k[c.table[0, pos // 16].long(), pos % 16] = k
    for scale in (0.3, -0.3):
        got = binding.paged_attention(q, *c.args(), max_new=new, scale=scale)
        want, mag, total, seen = attend_reference(c, q, scale)
        # magnitudes of q.k reach about 20 * 11.5 + noise, scale 0.3: 80 a score
        within(got, want, 4 * dim * 80 * U32 * mag + attend_tol(c, q, want, mag, total, seen))


@pytest.mark.parametrize("new", [1, 90])
def test_attend_scale_zero(new):
    """All weights equal: the mean of the visible values (masked keys stay masked)."""
    check_attend(Cache([(new, 300)], 4, 1, 128, 16, torch.bfloat16), 4, torch.bfloat16, 128, scale=0.0)


@pytest.mark.parametrize("most", [1, 12])
def test_attend_many_sequences(most):
    """More sequences than lanes of a warp, some of them without new tokens."""
    rng = np.random.default_rng(most)
    seqs = []
    for _ in range(300):
        n = int(rng.integers(0, most + 1))
        seqs.append((n, int(n + rng.integers(0, 90))))
    check_attend(Cache(seqs, 8, 2, 64, 16, torch.float16), 8, torch.float16, 64, max_new=most)


@pytest.mark.parametrize("max_new", [1, 100])
def test_attend_nothing_new(max_new):
    """No sequence has a new token: every row is left as it is."""
    c = Cache([(0, 40), (0, 0)], 4, 2, 64, 16, torch.float16)
    q = normal(76, 3, 4, 64, dtype=torch.float16)
    out = torch.full_like(q, 3.0)
    binding.paged_attention(q, *c.args(), max_new=max_new, out=out)
    assert (out == 3).all() and binding.device_status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_attend_nan_in_a_row_stays_there(new):
    """A NaN in one row of q makes that row's output NaN and no other's."""
    c = Cache([(new, 600), (1, 77)], 4, 2, 128, 16, torch.bfloat16)
    q = normal(77, c.total, 4, 128, dtype=torch.bfloat16)
    want = binding.paged_attention(q, *c.args(), max_new=new)
    q[0, 1, 5] = math.nan
    got = binding.paged_attention(q, *c.args(), max_new=new)
    assert torch.isnan(got[0, 1]).all()
    keep = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("new,max_new", [(1, 1), (200, 200)])
def test_attend_repeats_bit_for_bit_and_on_another_stream(new, max_new):
    c = Cache([(new, 3000), (1, 500)], 8, 2, 128, 16, torch.bfloat16)
    q = normal(73, c.total, 8, 128, dtype=torch.bfloat16)
    want = binding.paged_attention(q, *c.args(), max_new=max_new)
    assert torch.equal(want, binding.paged_attention(q, *c.args(), max_new=max_new))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(q) for _ in range(4)]
    for o in outs:
        binding.paged_attention(q, *c.args(), max_new=max_new, out=o, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for o in outs:
        assert torch.equal(want, o)


def test_attend_in_a_graph_with_changing_lengths():
    """Lengths live on the device: a captured call follows them."""
    c = Cache([(1, 700), (1, 90)], 8, 2, 64, 16, torch.float16)
    q = normal(74, 2, 8, 64, dtype=torch.float16)
    out = torch.empty_like(q)
    ws = torch.empty(binding.paged_attention_workspace(1, 8, 2, 64), dtype=torch.uint8, device="cuda")
    call = lambda: binding.paged_attention(q, *c.args(), max_new=1, out=out, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([700, 90], [1, 64], [650, 17]):
        c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        full, c.dense, c.len = (c.dense, c.len), [(k[:n], v[:n]) for (k, v), n in zip(c.dense, lens)], lens
        g.replay()
        want = attend_reference(c, q, 64 ** -0.5)
        within(out, want[0], attend_tol(c, q, *want))
        c.dense, c.len = full


def test_attend_pages_past_32_bit_offsets():
    """A cache of more than 2^32 elements: pages at its far end."""
    page, kv_heads, dim = 256, 8, 128
    pages = (1 << 32) // (page * kv_heads * dim) + 8
    k, v = (torch.empty(pages, page, kv_heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = Cache([(1, 600), (20, 500)], 16, kv_heads, dim, page, torch.bfloat16, spare=0)
    used = c.k.shape[0]
    k[pages - used:], v[pages - used:] = c.k, c.v
    c.table = torch.where((c.table >= 0) & (c.table < used), c.table + (pages - used), c.table)
    c.k, c.v = k, v
    check_attend(c, 16, torch.bfloat16, dim)
    check_attend(c, 16, torch.bfloat16, dim, max_new=1)


@pytest.mark.parametrize("max_new", [1, 64])
def test_attend_bad_pages_are_not_followed(max_new):
    """A page out of range among the keys: no fault, the status bit, other sequences as they were."""
    binding.device_status()
    c = Cache([(1, 100), (1, 100)], 4, 2, 64, 16, torch.bfloat16)
    q = normal(75, 2, 4, 64, dtype=torch.bfloat16)
    want = binding.paged_attention(q, *c.args(), max_new=max_new)
    assert binding.device_status() == 0
    c.table[1, 3] = 1 << 28
    got = binding.paged_attention(q, *c.args(), max_new=max_new)
    assert binding.device_status() == 2 and torch.equal(got[0], want[0]) and torch.isfinite(got).all()


LONG_TABLE = [(test_attend_chunk, (new, length, *heads, dtype))
              for new, length in [(15, 200), (64, 64), (65, 700), (127, 129), (128, 128), (129, 1025), (257, 300)]
              for heads in [(4, 1, 128), (2, 2, 64), (5, 1, 128), (8, 1, 64), (3, 1, 64)] for dtype in TYPES]
LONG_TABLE += [(test_attend_one_token, (length, *heads, dim, torch.bfloat16)) for length in [1, 16, 65, 129, 1000]
               for heads in [(8, 2), (7, 1)] for dim in [64, 128]]
LONG_TABLE += [(test_attend_rows_that_see_nothing, (*seq, dim))
               for seq in [(1, 0), (4, 2), (40, 10), (300, 1), (130, 129)] for dim in [64, 128]]
LONG_TABLE += [(test_attend_ragged_batch, (64, dim, torch.float16)) for dim in [64, 128]]
LONG_TABLE += [(test_attend_max_new_is_only_a_hint, (n,)) for n in [1, 40, 4096]]
LONG_TABLE += [(test_attend_layouts_and_strides, (n,)) for n in [1, 100]]
LONG_TABLE += [(test_attend_sharp_and_growing_scores, (n,)) for n in [1, 64]]
LONG_TABLE += [(test_attend_scale_zero, (n,)) for n in [1, 90]]
LONG_TABLE += [(test_attend_nothing_new, (n,)) for n in [1, 100]]
LONG_TABLE += [(test_attend_nan_in_a_row_stays_there, (n,)) for n in [1, 40]]
LONG_TABLE += [(test_attend_repeats_bit_for_bit_and_on_another_stream, n) for n in [(1, 1), (200, 200)]]
LONG_TABLE += [(test_attend_in_a_graph_with_changing_lengths, ())]
LONG_TABLE += [(test_attend_bad_pages_are_not_followed, (n,)) for n in [1, 64]]


@pytest.mark.parametrize("case", range(len(LONG_TABLE)))
def test_attend_in_a_long_table(case, monkeypatch):
    """A table for more tokens than clusters take: the same calls by shares of the keys or on the tensor cores."""
    monkeypatch.setattr(Cache, "least_tokens", 7300)
    test, args = LONG_TABLE[case]
    test(*args)


# ------------------------------------------------------------------- rope --
def rope_table(positions, rot):
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()


def rope_reference(x, table, pos, pairs):
    x, rot = x.to(F64).clone(), table.shape[1]
    cos, sin = (t.to(F64)[:, None] for t in table[pos].split(rot // 2, 1))
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    mag = torch.zeros_like(x)
    if pairs:
        mag[..., 0:rot:2], mag[..., 1:rot:2] = a.abs() + b.abs(), a.abs() + b.abs()
        x[..., 0:rot:2], x[..., 1:rot:2] = u, v
    else:
        mag[..., :rot // 2], mag[..., rot // 2:rot] = a.abs() + b.abs(), a.abs() + b.abs()
        x[..., :rot // 2], x[..., rot // 2:rot] = u, v
    return x, mag


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dim,rot,page,layout", [(128, 128, 16, "token"), (64, 64, 64, "head"), (128, 32, 8, "head"),
                                                 (64, 8, 16, "token")])
def test_rope_append(dim, rot, page, layout, pairs, dtype):
    heads, kv_heads = 6, 2
    seqs = [(1, 77), (0, 5), (20, 20), (3, 400), (1, 1), (16, 2 * page)]
    c = Cache(seqs, heads, kv_heads, dim, page, dtype, layout=layout)
    rows = normal(50, c.total + 2, (heads + 2 * kv_heads) * dim)  # one product's output, split by columns
    q, k, v = rows.split([heads * dim, kv_heads * dim, kv_heads * dim], 1)
    table = rope_table(400, rot)
    before_k, before_v = c.k.clone(), c.v.clone()
    binding.device_status()
    got = binding.rope_append(q, k, v, table, *c.args(), interleaved=pairs)
    assert binding.device_status() == 0
    assert (got[c.total:] == 0).all()  # tokens of no sequence
    at = 0
    for i, (new, n) in enumerate(seqs):
        pos = torch.arange(n - new, n, device="cuda")
        where = c.table[i, pos // page].long(), pos % page
        for x, out, h in ((q, got[at:at + new], heads), (k, c.k[where], kv_heads)):
            want, mag = rope_reference(x[at:at + new].view(new, h, dim), table, pos, pairs)
            if new:
                within(out, want, 4 * U32 * mag + U[dtype] * want.abs() + TINY[dtype])
        assert torch.equal(c.v[where], v[at:at + new].view(new, kv_heads, dim).to(dtype))
        before_k[where], before_v[where] = c.k[where], c.v[where]
        at += new
    for a, b in ((before_k, c.k), (before_v, c.v)):  # nothing else has changed
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_rope_positions_and_pages_out_of_range():
    c = Cache([(3, 1), (1, 60), (1, 20), (1, 33)], 2, 1, 64, 16, torch.bfloat16, width=4)
    c.table[2, 1] = -1
    x = normal(51, 6, 2 * 64)
    k = v = x[:, :64]
    before = c.k.clone()
    binding.device_status()
    got = binding.rope_append(x, k, v, rope_table(40, 64), *c.args())
    assert binding.device_status() == 2
    bad = [0, 1, 3, 4]  # positions -2 and -1, position 59 of 40, a page of -1
    assert (got[bad] == 0).all() and (got[2] != 0).any() and (got[5] != 0).any()
    changed = (before.view(torch.int16) != c.k.view(torch.int16)).flatten(2).any(-1).sum()
    assert changed == 2


def test_new_keys_then_attention():
    """The cache as rope_append leaves it is what paged_attention reads."""
    dtype, dim, heads, kv_heads = torch.bfloat16, 128, 8, 2
    c = Cache([(1, 50), (30, 200)], heads, kv_heads, dim, 16, dtype)
    q, k, v = normal(52, 31, heads * dim), normal(53, 31, kv_heads * dim), normal(54, 31, kv_heads * dim)
    turned = binding.rope_append(q, k, v, rope_table(200, dim), *c.args())
    got = binding.paged_attention(turned, *c.args(), max_new=30)
    for i, n in enumerate(c.len):
        pos = torch.arange(n, device="cuda")
        where = c.table[i, pos // 16].long(), pos % 16
        c.dense[i] = (c.k[where], c.v[where])
    want = attend_reference(c, turned, dim ** -0.5)
    within(got, want[0], attend_tol(c, turned, *want))
