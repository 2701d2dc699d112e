"""The q8_0 cache: what is written to it and read back, and attention over it,
against plain forms in 64 bits.  Tolerances are bounds from the arithmetic, as in
test_gpu_ops.py; what has an exact definition is compared by bits."""
import math

import numpy as np
import pytest
import torch

from decode_q1_gemv_gb300 import binding
from tests.test_gpu_ops import F64, TINY, U, U32, normal, rope_reference, rope_table, within

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    binding.device_status()


def quantized(x):
    """binding.quantize of blocks along x's last axis: quants and scales' bits, of x's shape."""
    q, d = binding.quantize(x.contiguous().view(-1, x.shape[-1]))
    return q.view(x.shape), d.view(*x.shape[:-1], -1)


def values(q, d):
    """Quants times scales, exact in 64 bits (and in f32)."""
    return (q.to(F64).unflatten(-1, (-1, 32)) * d.view(torch.float16).to(F64)[..., None]).flatten(-2)


ORDERS = {"token": (0, 1, 2), "head": (0, 2, 1), "slot": (1, 0, 2), "last": (2, 1, 0)}  # storage of (page, slot, head)


class Cache8:
    """A paged q8_0 cache with random content and pages; no token's slots hold scales that are NaN, no page's entries lie in range."""

    least_tokens = 0

    def __init__(self, seqs, kv_heads, dim, page, layout="head", scales=None, width=None, seed=40, spare=2, std=1.0):
        self.new, self.len = [s[0] for s in seqs], [s[1] for s in seqs]
        self.page, self.kv_heads, self.dim = page, kv_heads, dim
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
        shape = (pages, page, kv_heads)

        def stored(name, last, value, dtype):
            o = ORDERS[name]
            t = torch.full([shape[a] for a in o] + [last], value, dtype=dtype, device="cuda")
            back = [o.index(a) for a in range(3)]
            return t.permute(*back, 3)

        self.k, self.v = (stored(layout, dim, 127, torch.int8) for _ in range(2))
        self.ks, self.vs = (stored(scales or layout, dim // 32, math.nan, torch.float16) for _ in range(2))
        self.table = torch.from_numpy(table).cuda()
        self.kv_len = torch.tensor(self.len, dtype=torch.int32, device="cuda")
        self.new_start = torch.tensor(np.cumsum([0] + self.new), dtype=torch.int32, device="cuda")
        self.total = sum(self.new)
        self.dense = []
        for i, n in enumerate(self.len):
            if n:
                self.put(i, *(normal(seed + 10 * i + j, n, kv_heads, dim, std=std) for j in (1, 2)), fresh=True)
            else:
                self.dense.append((torch.zeros(0, kv_heads, dim, dtype=F64, device="cuda"),) * 2)

    def where(self, i, pos):
        return self.table[i, pos // self.page].long(), pos % self.page

    def put(self, i, k, v, fresh=False):
        """Sequence i's keys and values, given as floats."""
        at = self.where(i, torch.arange(k.shape[0], device="cuda"))
        (kq, kd), (vq, vd) = quantized(k), quantized(v)
        self.k[at], self.v[at], self.ks[at], self.vs[at] = kq, vq, kd.view(torch.float16), vd.view(torch.float16)
        pair = values(kq, kd), values(vq, vd)
        if fresh:
            self.dense.append(pair)
        else:
            self.dense[i] = pair

    def args(self):
        return self.k, self.v, self.ks, self.vs, self.table, self.kv_len, self.new_start


def attend_reference(c, q, scale):
    """Values, the rows' sums of |weight * v|, sums of weights relative to the largest, visible keys, and the
    largest |scale| sum |q k| of a row."""
    out = torch.zeros(q.shape, dtype=F64, device="cuda")
    mag, total, seen = out.clone(), torch.ones(q.shape[:2], dtype=F64, device="cuda"), out[:, 0, 0].clone()
    size = torch.zeros(q.shape[:2], dtype=F64, device="cuda")
    group = q.shape[1] // c.kv_heads
    at = 0
    for (k, v), new, n in zip(c.dense, c.new, c.len):
        if new and n:
            k, v = (t.repeat_interleave(group, 1) for t in (k, v))
            x = q[at:at + new].to(F64)
            hidden = torch.arange(n, device="cuda") > torch.arange(n - new, n, device="cuda")[:, None]
            s = (torch.einsum("rhd,khd->rhk", x, k) * scale).masked_fill(hidden[:, None], -math.inf)
            some = ~hidden.all(1)
            w = torch.exp(s[some] - s[some].amax(-1, keepdim=True))
            rows = torch.arange(at, at + new, device="cuda")[some]
            total[rows] = w.sum(-1)
            w = w / w.sum(-1, keepdim=True)
            out[rows], mag[rows] = torch.einsum("rhk,khd->rhd", w, v), torch.einsum("rhk,khd->rhd", w, v.abs())
            seen[rows] = (~hidden[some]).sum(1).to(F64)
            size[at:at + new] = (torch.einsum("rhd,khd->rhk", x.abs(), k.abs()) * abs(scale)).amax(-1)
        at += new
    return out, mag, total, seen, size


# A weight (few rows: its product with a scale) is rounded once to f16: 2^-11 of itself, small ones 2^-25 of
# the largest.  Few rows: keys and values are exact.  Many rows: with bf16 q keys (which moves a
# score by 2^-11 of its sum of magnitudes, and a weight twice that, with the sum of all) and values are
# rounded to f16, with f16 q to two of them.  Sums of dim products in f32: a score off by dim 2^-24 of its magnitudes at most,
# and 1e-6 as in test_gpu_ops.py; then the output's rounding.
def attend_tol(c, q, out, mag, total, seen, size, many=True):
    dtype, dim = q.dtype, q.shape[2]
    bf = dtype == torch.bfloat16
    weights = 2.0 ** -11
    key = value = 2.0 ** -11 if many and bf else 2.0 ** -22
    most = max((v.abs().max().item() for _, v in c.dense if v.numel()), default=0.0)
    small = 2.0 ** -25 * seen[:, None] / total * most
    part = (weights + value + 1e-6) + (2 * key + 2 * dim * U32) * size
    return part[..., None] * mag + small[..., None] + U[dtype] * out.abs() + TINY[dtype]


def check_attend(c, heads, dtype, max_new=None, scale=None, seed=70, many=True):
    q = normal(seed, max(1, c.total), heads, c.dim, dtype=dtype)[:c.total]
    got = binding.paged_attention_q8(q, *c.args(), max_new=max_new or max(c.new), scale=scale)
    want = attend_reference(c, q, c.dim ** -0.5 if scale is None else scale)
    within(got, want[0], attend_tol(c, q, *want, many=many))
    assert binding.device_status() == 0  # no wait ran into its limit, no index was out of range
    return q, got


# ------------------------------------------------------- append and read --
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dim,rot,page,layout,scales", [(128, 128, 16, "token", "head"), (64, 64, 64, "head", "token"),
                                                        (128, 24, 8, "slot", "last"), (64, 8, 16, "last", "slot"),
                                                        (128, 96, 4096, "head", "head")])
def test_append(dim, rot, page, layout, scales, pairs, dtype):
    heads, kv_heads = 6, 2
    seqs = [(1, 77), (0, 5), (20, 20), (3, 400), (1, 1), (16, 2 * min(page, 64))]
    c = Cache8(seqs, kv_heads, dim, page, layout, scales)
    rows = normal(50, c.total + 2, (heads + 2 * kv_heads) * dim)  # one product's output, split by columns
    q, k, v = rows.split([heads * dim, kv_heads * dim, kv_heads * dim], 1)
    table = rope_table(400, rot)
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    got = binding.rope_append_q8(q, k, v, table, *c.args(), interleaved=pairs, dtype=dtype)
    assert binding.device_status() == 0 and got.dtype == dtype
    # q as rope_append turns it
    page16 = torch.zeros(c.k.shape, dtype=dtype, device="cuda")
    assert torch.equal(got, binding.rope_append(q, k, v, table, page16, page16.clone(), c.table, c.kv_len, c.new_start, interleaved=pairs))
    assert (got[c.total:] == 0).all()  # tokens of no sequence
    at = 0
    for i, (new, n) in enumerate(seqs):
        pos = torch.arange(n - new, n, device="cuda")
        where = c.where(i, pos)
        if new:
            vq, vd = quantized(v[at:at + new].reshape(new, kv_heads, dim))
            assert torch.equal(c.v[where], vq) and torch.equal(c.vs[where].view(torch.int16), vd)
            want, mag = rope_reference(k[at:at + new].reshape(new, kv_heads, dim), table, pos, pairs)
            # half a quant, of the scale before its rounding to f16 (2^-11 of a value), and the turn's rounding
            top = want.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
            within(values(c.k[where], c.ks[where]), want, (0.5 / 127) * top * (1 + 2.0 ** -20) + 2.0 ** -11 * top + 4 * U32 * mag)
            assert ((c.ks[where].to(F64) * 127 - top[..., ::32]).abs() <= (2.0 ** -11 + 8 * U32) * top[..., ::32] + 2.0 ** -18).all()
        for old, now in zip(before, (c.k, c.v, c.ks, c.vs)):
            old[where] = now[where]
        at += new
    for old, now in zip(before, (c.k, c.v, c.ks, c.vs)):  # nothing else has changed
        assert torch.equal(old.view(torch.int8 if old.dtype == torch.int8 else torch.int16), now.view(torch.int8 if now.dtype == torch.int8 else torch.int16))


def test_append_positions_and_pages_out_of_range():
    c = Cache8([(3, 1), (1, 60), (1, 20), (1, 33)], 1, 64, 16, width=4)
    c.table[2, 1] = -1
    x = normal(51, 6, 2 * 64)
    k = v = x[:, :64]
    before = c.ks.clone()
    got = binding.rope_append_q8(x, k, v, rope_table(40, 64), *c.args())
    assert binding.device_status() == 2
    bad = [0, 1, 3, 4]  # positions -2 and -1, position 59 of 40, a page of -1
    assert (got[bad] == 0).all() and (got[2] != 0).any() and (got[5] != 0).any()
    assert (before.view(torch.int16) != c.ks.view(torch.int16)).flatten(2).any(-1).sum() == 2


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf, 1e9, 0.0, 1e-9, 3.4e38])
def test_append_unusual_blocks(value):
    """A block with a value that is no number is NaN as read; one too large for its f16 scale no number; others as they are."""
    c = Cache8([(4, 4)], 2, 64, 16)
    k, v = normal(5, 4, 128), normal(6, 4, 128)
    plain = k.clone()
    k[1, 40], v[2, 3] = value, value
    if value in (0.0, 1e-9):
        k[1, 32:64], v[2, :32] = value, value
    zero = torch.zeros(4, 64, device="cuda")
    zero[:, :32] = 1  # cos 1, sin 0
    binding.rope_append_q8(plain, k, v, zero, *c.args())
    for x, got in zip((k, v), binding.cache_read_q8(*c.args(), 4, dtype=torch.float32)):
        got = got.view(4, 4, 32)
        bad = torch.zeros(4, 4, dtype=torch.bool, device="cuda")
        bad[(1, 1) if x is k else (2, 0)] = True
        if x is k and not math.isfinite(value):
            bad[1, 0] = True  # value 8, which is turned with value 40, by 0: NaN
        q, d = quantized(x.view(4, 4, 32))
        assert torch.equal(got[~bad].to(F64), values(q, d)[~bad])
        if math.isfinite(value) and value < 1e6:
            assert torch.equal(got[bad].to(F64), values(q, d)[bad])
        elif math.isfinite(value):  # a scale of infinity: quants of zero are NaN, others infinite
            assert not torch.isfinite(got[bad]).any()
        else:
            assert torch.isnan(got[bad]).all()


@pytest.mark.parametrize("dtype", [torch.float32, *TYPES])
@pytest.mark.parametrize("dim,page,layout,scales", [(128, 16, "token", "token"), (64, 128, "head", "last"), (128, 8, "slot", "head")])
def test_read(dim, page, layout, scales, dtype):
    """The last tokens of each sequence, all of them, none; rows of no sequence and tokens before the first are zero."""
    for new, n in [((1, 5, 0, 40), (300, 5, 7, 40)), ((300, 5, 7, 40), (300, 5, 7, 40)), ((4, 3, 2, 1), (2, 3, 0, 9))]:
        c = Cache8(list(zip(new, n)), 3, dim, page, layout, scales)
        k, v = binding.cache_read_q8(*c.args(), c.total + 3, dtype=dtype)
        assert k.shape == (c.total + 3, 3, dim) and k.dtype == dtype
        at = 0
        for (dk, dv), m, length in zip(c.dense, new, n):
            before = max(0, m - length)
            for got, want in ((k, dk), (v, dv)):
                assert (got[at:at + before] == 0).all()
                assert torch.equal(got[at + before:at + m], want[length - m + before:].to(torch.float32).to(dtype))
            at += m
        assert (k[at:] == 0).all() and (v[at:] == 0).all()
        binding.device_status()


def test_read_into_given_tensors_on_a_stream_and_bad_pages():
    c = Cache8([(50, 50), (3, 20)], 2, 64, 16)
    want = [t.half() for t in binding.cache_read_q8(*c.args(), 53, dtype=torch.float32)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    k = torch.full((53, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    got = binding.cache_read_q8(*c.args(), 53, k_out=k, v_out=v, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert got[0] is not None and got[0].data_ptr() == k.data_ptr() and torch.equal(k, want[0]) and torch.equal(v, want[1])
    c.table[0, 1] = 1 << 28
    binding.device_status()
    bad, _ = binding.cache_read_q8(*c.args(), 53, dtype=torch.float16)
    assert binding.device_status() == 2
    assert (bad[16:32] == 0).all() and torch.equal(bad[:16], want[0][:16]) and torch.equal(bad[32:], want[0][32:])


def test_what_the_binding_refuses():
    c = Cache8([(1, 20)], 1, 64, 16)
    x, table = normal(1, 1, 64), rope_table(20, 64)
    with pytest.raises(TypeError, match="bfloat16, float16"):
        binding.rope_append_q8(x, x, x, table, *c.args(), dtype=torch.float32)
    with pytest.raises(TypeError, match="q_out has dtype"):
        binding.rope_append_q8(x, x, x, table, *c.args(), q_out=torch.empty(1, 1, 64, device="cuda"))
    for i, text in ((0, "cache_k has dtype"), (1, "cache_v has dtype"), (2, "scale_k has dtype"), (3, "scale_v has dtype")):
        bad = list(c.args())
        bad[i] = bad[i].to(torch.float32)
        with pytest.raises(TypeError, match=text):
            binding.cache_read_q8(*bad, 1)
    bad = list(c.args())
    bad[3] = torch.empty(*bad[3].shape[:3], 3, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="scale_v has shape"):
        binding.cache_read_q8(*bad, 1)
    bad[3] = torch.empty(*c.vs.shape[:3], 4, dtype=torch.float16, device="cuda")[..., :2]
    with pytest.raises(ValueError, match="same strides"):
        binding.cache_read_q8(*bad, 1)
    with pytest.raises(ValueError, match="positive"):
        binding.cache_read_q8(*c.args(), 0)
    q = normal(2, 1, 2, 64, dtype=torch.float16)
    with pytest.raises(binding.Q1Error, match="workspace holds"):
        binding.paged_attention_q8(q, *c.args(), max_new=1, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="q has dim 128, the cache 64"):
        binding.paged_attention_q8(q.view(1, 1, 128), *c.args(), max_new=1)
    with pytest.raises(TypeError, match="q has dtype"):
        binding.paged_attention_q8(q.float(), *c.args(), max_new=1)
    assert binding.device_status() == 0


# -------------------------------------------------------------- attention --
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 2), (4, 4), (7, 1), (32, 2), (12, 1)])
@pytest.mark.parametrize("length", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000])
def test_attend_one_token(length, heads, kv_heads, dim, dtype):
    check_attend(Cache8([(1, length)], kv_heads, dim, 16), heads, dtype, many=False)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (16, 1), (32, 8), (36, 12)])
@pytest.mark.parametrize("width", [4, 8, 17, 40, 110, 200])
def test_attend_whatever_the_table_holds(width, heads, kv_heads, dim):
    most = width * 16
    seqs = [(1, most), (1, 1), (1, max(1, most // 2 - 3)), (0, most), (2, min(most, 70)), (1, most - 1)]
    check_attend(Cache8(seqs, kv_heads, dim, 16, width=width), heads, torch.bfloat16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 128), (2, 2, 64), (5, 1, 128), (8, 1, 64), (3, 1, 64)])
@pytest.mark.parametrize("new,length", [(2, 2), (3, 50), (8, 300), (15, 200), (64, 64), (65, 700), (127, 129), (128, 128), (129, 1025), (257, 300)])
def test_attend_chunk(new, length, heads, kv_heads, dim, dtype):
    check_attend(Cache8([(new, length)], kv_heads, dim, 16), heads, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,layout,scales", [(8, "token", "head"), (64, "head", "token"), (256, "slot", "last"), (128, "last", "slot")])
def test_attend_ragged_batch(page, layout, scales, dim, dtype):
    seqs = [(1, 700), (0, 40), (33, 33), (1, 1), (140, 500), (4, 70), (2, 2000), (17, 300)]
    check_attend(Cache8(seqs, 2, dim, page, layout, scales), 8, dtype)


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 16, 16), (128, 8, 2), (64, 5, 1)])
def test_attend_many_items_a_cta(dim, heads, kv_heads):
    rng = np.random.default_rng(5)
    seqs = [(int(n), int(n + rng.integers(0, 300))) for n in np.exp(rng.uniform(0, np.log(300), 40))]
    for dtype in TYPES:
        check_attend(Cache8(seqs, kv_heads, dim, 32), heads, dtype)


@pytest.mark.parametrize("new,length", [(1, 0), (4, 2), (40, 10), (300, 1), (130, 129)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_attend_rows_that_see_nothing(new, length, dim, dtype):
    c = Cache8([(2, 9), (new, length), (1, 30)], 2, dim, 16, width=2 if length < 33 else None)
    q, got = check_attend(c, 4, dtype)
    empty = got[2:2 + new - length]
    assert empty.shape[0] == new - length and (empty == 0).all()


@pytest.mark.parametrize("width", [None, 500])
@pytest.mark.parametrize("max_new", [1, 7, 40, 4096, 1 << 30])
def test_attend_max_new_is_only_a_hint(max_new, width):
    check_attend(Cache8([(1, 100), (40, 333), (7, 50)], 2, 64, 16, width=width), 8, torch.float16, max_new=max_new)


@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("dtype", TYPES)
def test_attend_strides(new, dtype):
    """Strided q and out, rows of no sequence left alone."""
    c = Cache8([(new, 500), (1, 33)], 2, 128, 64)
    wide = normal(71, c.total + 3, 8 + 2, 128 + 8, dtype=dtype)
    q = wide[:, 1:-1, 8:]
    buf = torch.full((c.total + 3, 8, 128 + 16), 9.0, dtype=dtype, device="cuda")
    got = binding.paged_attention_q8(q, *c.args(), max_new=new, out=buf[..., 8:-8])
    want = attend_reference(c, q[:c.total].contiguous(), 128 ** -0.5)
    within(got[:c.total], want[0], attend_tol(c, q[:c.total], *want))
    assert (buf[..., :8] == 9).all() and (buf[..., -8:] == 9).all() and (buf[c.total:] == 9).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("scale", [0.3, -0.3, 0.0])
def test_attend_sharp_and_growing_scores(scale, new, dtype):
    """Large scores of both signs: one key takes all weight, and the maximum grows along the keys."""
    c = Cache8([(new, 900)], 1, 128, 16)
    q = normal(72, c.total, 4, 128, dtype=dtype)
    one = q[0, 0].float() / q[0, 0].float().norm()
    ramp = one * torch.linspace(-20, 20, 900, device="cuda")[:, None]
    c.put(0, normal(1, 900, 1, 128) * 0.1 + ramp[:, None], normal(2, 900, 1, 128))
    got = binding.paged_attention_q8(q, *c.args(), max_new=new, scale=scale)
    want = attend_reference(c, q, scale)
    within(got, want[0], attend_tol(c, q, *want, many=new > 1))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 5, 90])
@pytest.mark.parametrize("kstd,vstd,qstd", [(1e6, 1e6, 1e-6), (1e-4, 1e-4, 100.0), (30.0, 2e5, 0.03), (1.0, 1e-5, 1.0)])
def test_attend_any_size_of_values(kstd, vstd, qstd, new, dtype):
    """Keys and values far outside f16, and near its least ones; the sizes of q, k and v are each other's inverse."""
    if dtype == torch.float16 and vstd > 1e4:
        vstd = 1e3  # the output is f16
    c = Cache8([(new, 400), (new, 90)], 2, 64, 16)
    for i, n in enumerate(c.len):
        k, v = normal(8 + i, n, 2, 64, std=kstd), normal(18 + i, n, 2, 64, std=vstd)
        if kstd > 1e5:  # (within what a scale holds)
            k, v = k.clamp(-6e6, 6e6), v.clamp(-6e6, 6e6)
        c.put(i, k, v)
    q = normal(73, c.total, 4, 64, std=qstd, dtype=dtype)
    got = binding.paged_attention_q8(q, *c.args(), max_new=new, scale=0.1)
    want = attend_reference(c, q, 0.1)
    within(got, want[0], attend_tol(c, q, *want))


@pytest.mark.parametrize("most", [1, 12])
def test_attend_many_sequences(most):
    rng = np.random.default_rng(most)
    seqs = []
    for _ in range(300):
        n = int(rng.integers(0, most + 1))
        seqs.append((n, int(n + rng.integers(0, 90))))
    check_attend(Cache8(seqs, 2, 64, 16), 8, torch.float16, max_new=most)


@pytest.mark.parametrize("max_new", [1, 100])
def test_attend_nothing_new(max_new):
    c = Cache8([(0, 40), (0, 0)], 2, 64, 16)
    q = normal(76, 3, 4, 64, dtype=torch.float16)
    out = torch.full_like(q, 3.0)
    binding.paged_attention_q8(q, *c.args(), max_new=max_new, out=out)
    assert (out == 3).all() and binding.device_status() == 0


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("new", [1, 5, 40])
@pytest.mark.parametrize("dtype", TYPES)
def test_attend_no_number_in_a_row_stays_there(new, dtype, value):
    c = Cache8([(new, 600), (1, 77)], 2, 128, 16)
    q = normal(77, c.total, 4, 128, dtype=dtype)
    want = binding.paged_attention_q8(q, *c.args(), max_new=new)
    q[0, 1, 5] = value
    got = binding.paged_attention_q8(q, *c.args(), max_new=new)
    assert torch.isnan(got[0, 1]).all()
    keep = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
    keep[0, 1] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("new", [1, 6, 16, 100])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("which", ["k", "v"])
def test_attend_no_number_in_the_cache(which, dtype, new, value):
    """A block of the key or value of a new token without a number: no other rows than those that see it are touched."""
    c = Cache8([(new, 300), (2, 50)], 2, 128, 16)
    q = normal(78, c.total, 6, 128, dtype=dtype)
    want = binding.paged_attention_q8(q, *c.args(), max_new=new)
    hit = 300 - new // 2 - 1
    at = c.where(0, torch.tensor(hit, device="cuda"))
    (c.ks if which == "k" else c.vs)[at[0], at[1], 1, 2] = value  # key head 1, values 64..95
    got = binding.paged_attention_q8(q, *c.args(), max_new=new)
    first = hit - (300 - new)  # the first row that sees it
    touched = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
    touched[first:new, 3:] = True
    if which == "v":
        touched[..., :64] = touched[..., 96:] = False
        assert not torch.isfinite(got[touched]).any()
    else:  # of a NaN all, of an infinite key scale all rows with a score that is none
        assert torch.isnan(got[touched]).all()
    # The others are as without the value, to the bit where the powers of two that weights and copies are
    # relative to (of the largest finite scales) are the same, and within the bound in any case.
    ref = attend_reference(c, q, 128 ** -0.5)
    within(got[~touched], ref[0][~touched], attend_tol(c, q, *ref)[~touched])
    within(want, ref[0], attend_tol(c, q, *ref))
    binding.device_status()


@pytest.mark.parametrize("new,max_new", [(1, 1), (200, 200)])
def test_attend_repeats_bit_for_bit_and_on_another_stream(new, max_new):
    c = Cache8([(new, 3000), (1, 500)], 2, 128, 16)
    q = normal(73, c.total, 8, 128, dtype=torch.bfloat16)
    want = binding.paged_attention_q8(q, *c.args(), max_new=max_new)
    assert torch.equal(want, binding.paged_attention_q8(q, *c.args(), max_new=max_new))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(q) for _ in range(4)]
    for o in outs:
        binding.paged_attention_q8(q, *c.args(), max_new=max_new, out=o, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for o in outs:
        assert torch.equal(want, o)


@pytest.mark.parametrize("dtype", TYPES)
def test_attend_workspaces_of_any_number_of_sequences(dtype):
    """Copies of one sequence at a time, of two, of all: other shares of the CTAs, so other last bits."""
    c = Cache8([(60, 900), (1, 40), (100, 100), (0, 30), (5, 700), (80, 1300)], 2, 64, 16, width=90)
    q = normal(74, c.total, 8, 64, dtype=dtype)
    size = [binding.paged_attention_q8_workspace(100, 8, 2, 64, 90 * 16, n, dtype) for n in (1, 2, 6)]
    outs = [binding.paged_attention_q8(q, *c.args(), max_new=100, workspace=torch.full((n,), 255, dtype=torch.uint8, device="cuda"))
            for n in size]
    assert size[0] < size[1] < size[2]
    want = attend_reference(c, q, 64 ** -0.5)
    for o in outs:
        within(o, want[0], attend_tol(c, q, *want))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_attend_mixed_calls_one_after_another(dim, dtype):
    """Calls of short and long sequences back to back on one workspace, in a graph."""
    heads, calls = 16, 8
    cs = [Cache8([(200, 1500), (1, 900), (3, 2500), (130, 131), (16, 40)], 4, dim, 32, seed=90 + i, width=250) for i in range(3)]
    qs = [normal(95 + i, cs[0].total, heads, dim, dtype=dtype) for i in range(3)]
    size = binding.paged_attention_q8_workspace(200, heads, 4, dim, 250 * 32, 3, dtype)  # of three of the five at once
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    want = [binding.paged_attention_q8(q, *c.args(), max_new=200, workspace=torch.empty_like(ws)) for q, c in zip(qs, cs)]
    for q, c, w in zip(qs, cs, want):
        ref = attend_reference(c, q, dim ** -0.5)
        within(w, ref[0], attend_tol(c, q, *ref))
    outs = [torch.empty_like(qs[0]) for _ in range(calls)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(calls):
            binding.paged_attention_q8(qs[i % 3], *cs[i % 3].args(), max_new=200, out=outs[i], workspace=ws)
    for _ in range(5):
        for o in outs:
            o.fill_(7.0)
        g.replay()
        for i, o in enumerate(outs):
            assert torch.equal(o, want[i % 3])
    assert binding.device_status() == 0


def test_attend_in_a_graph_with_changing_lengths():
    """Lengths live on the device: a captured call follows them."""
    c = Cache8([(1, 700), (1, 90)], 2, 64, 16)
    q = normal(74, 2, 8, 64, dtype=torch.float16)
    out = torch.empty_like(q)
    ws = torch.empty(binding.paged_attention_q8_workspace(1, 8, 2, 64, 700), dtype=torch.uint8, device="cuda")
    call = lambda: binding.paged_attention_q8(q, *c.args(), max_new=1, out=out, workspace=ws)  # noqa: E731
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


@pytest.mark.parametrize("max_new", [1, 64])
def test_attend_bad_pages_are_not_followed(max_new):
    c = Cache8([(1, 100), (1, 100)], 2, 64, 16)
    q = normal(75, 2, 4, 64, dtype=torch.bfloat16)
    want = binding.paged_attention_q8(q, *c.args(), max_new=max_new)
    assert binding.device_status() == 0
    c.table[1, 3] = 1 << 28
    got = binding.paged_attention_q8(q, *c.args(), max_new=max_new)
    assert binding.device_status() == 2 and torch.equal(got[0], want[0]) and torch.isfinite(got).all()


def test_pages_past_32_bit_offsets():
    """A cache of more than 2^32 values: pages at its far end, appended to, attended to and read."""
    page, kv_heads, dim = 256, 8, 128
    pages = (1 << 32) // (page * kv_heads * dim) + 8
    c = Cache8([(1, 600), (20, 500)], kv_heads, dim, page, spare=0)
    used = c.k.shape[0]
    for name in ("k", "v", "ks", "vs"):
        small = getattr(c, name)
        big = torch.empty(pages, kv_heads, page, small.shape[-1], dtype=small.dtype, device="cuda").transpose(1, 2)
        big[pages - used:] = small
        setattr(c, name, big)
    c.table = torch.where((c.table >= 0) & (c.table < used), c.table + (pages - used), c.table)
    check_attend(c, 16, torch.bfloat16)
    check_attend(c, 16, torch.bfloat16, max_new=1)
    k, v = binding.cache_read_q8(*c.args(), 21, dtype=torch.float32)
    assert torch.equal(k[1:].to(F64), c.dense[1][0][-20:]) and torch.equal(v[:1].to(F64), c.dense[0][1][-1:])
    x = normal(9, 21, kv_heads * dim)
    binding.rope_append_q8(x, x, x, rope_table(600, dim), *c.args())
    _, v = binding.cache_read_q8(*c.args(), 21, dtype=torch.float32)
    assert torch.equal(v.to(F64), values(*quantized(x.view(21, kv_heads, dim)))) and binding.device_status() == 0


def test_new_keys_then_attention():
    """The cache as rope_append_q8 leaves it is what cache_read_q8 gives and paged_attention_q8 reads."""
    heads, kv_heads, dim = 8, 2, 128
    c = Cache8([(1, 50), (30, 200)], kv_heads, dim, 16)
    q, k, v = normal(52, 31, heads * dim), normal(53, 31, kv_heads * dim), normal(54, 31, kv_heads * dim)
    turned = binding.rope_append_q8(q, k, v, rope_table(200, dim), *c.args())
    got = binding.paged_attention_q8(turned, *c.args(), max_new=30)
    whole = torch.tensor([0, 50, 250], dtype=torch.int32, device="cuda")
    k, v = binding.cache_read_q8(*c.args()[:-1], whole, 250, dtype=torch.float32)
    c.dense = [(k[:50].to(F64), v[:50].to(F64)), (k[50:].to(F64), v[50:].to(F64))]
    want = attend_reference(c, turned, dim ** -0.5)
    within(got, want[0], attend_tol(c, turned, *want))


LONG_TABLE = [(test_attend_chunk, (new, length, *heads, dtype))
              for new, length in [(15, 200), (64, 64), (65, 700), (128, 128), (129, 1025), (257, 300)]
              for heads in [(4, 1, 128), (2, 2, 64), (5, 1, 128)] for dtype in TYPES]
LONG_TABLE += [(test_attend_one_token, (length, *heads, dim, dtype)) for length in [1, 16, 65, 129, 1000]
               for heads in [(8, 2), (12, 1)] for dim in [64, 128] for dtype in TYPES]
LONG_TABLE += [(test_attend_rows_that_see_nothing, (*seq, dim, torch.bfloat16))
               for seq in [(1, 0), (4, 2), (40, 10), (300, 1), (130, 129)] for dim in [64, 128]]
LONG_TABLE += [(test_attend_ragged_batch, (64, "head", "token", dim, dtype)) for dim in [64, 128] for dtype in TYPES]
LONG_TABLE += [(test_attend_strides, (n, torch.bfloat16)) for n in [1, 100]]
LONG_TABLE += [(test_attend_sharp_and_growing_scores, (s, n, dtype)) for n in [1, 64] for s in [0.3, -0.3, 0.0] for dtype in TYPES]
LONG_TABLE += [(test_attend_nothing_new, (n,)) for n in [1, 100]]
LONG_TABLE += [(test_attend_no_number_in_a_row_stays_there, (n, dtype, math.inf)) for n in [1, 5, 40] for dtype in TYPES]
LONG_TABLE += [(test_attend_no_number_in_the_cache, (which, dtype, n, v)) for n in [1, 6, 16, 100] for which in "kv" for dtype in TYPES
               for v in (math.nan, math.inf)]
LONG_TABLE += [(test_attend_any_size_of_values, (1e6, 1e6, 1e-6, n, torch.bfloat16)) for n in [1, 5, 90]]
LONG_TABLE += [(test_attend_in_a_graph_with_changing_lengths, ())]
LONG_TABLE += [(test_attend_bad_pages_are_not_followed, (n,)) for n in [1, 64]]


@pytest.mark.parametrize("case", range(len(LONG_TABLE)))
def test_attend_in_a_long_table(case, monkeypatch):
    """A table for more tokens than clusters take: the same calls by shares of the keys or on the tensor cores."""
    monkeypatch.setattr(Cache8, "least_tokens", 7300)
    test, args = LONG_TABLE[case]
    test(*args)
