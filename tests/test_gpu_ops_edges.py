"""The operators between the products where inputs are not ordinary: values that
are no numbers, streams of the caller's, rows and axes of one entry, long sums,
caches past 32-bit offsets in every form of the attention.  Plain forms and
tolerances are those of test_gpu_ops.py where nothing else is said."""
import math

import pytest
import torch

from decode_q1_gemv_gb300 import binding
from tests.test_gpu_ops import Cache, U, check_attend, lora_reference, lora_tol, normal, rope_table, within

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]
# The NaN that the GPU's arithmetic gives, the host's, and the largest patterns of both signs.
NANS = [0x7FFFFFFF, 0x7FC00000, 0x7F800001, -1, -0x400000]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    binding.device_status()


def only_these(got, clean, bad, nan=True):
    """NaN (or an infinity) where `bad` is, elsewhere the bits of the call with numbers."""
    assert torch.isnan(got[bad]).all() if nan else not torch.isfinite(got[bad]).any()
    assert torch.equal(got[~bad], clean[~bad])


# ------------------------------------------------------------------- lora --
def lora_inputs(dtype, nvec, rank=24, n=264, rows=70, adapters=3):
    x, base = normal(1, nvec, n), normal(2, nvec, rows)
    a, b = normal(3, adapters, rank, n, std=0.05, dtype=dtype), normal(4, adapters, rows, rank, dtype=dtype)
    index = torch.arange(nvec, dtype=torch.int32, device="cuda") * 3 % (adapters + 1) - 1
    return x, a, b, index, base


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nvec", [4, 40, 200])  # a cluster a vector, buckets of eight, of sixteen
@pytest.mark.parametrize("bits", NANS)
def test_lora_nan_in_x(bits, nvec, dtype):
    x, a, b, index, base = lora_inputs(dtype, nvec)
    clean = binding.lora_add(x, a, b, index, base=base)
    hit = (index == 1).nonzero()[-1, 0]
    x.view(torch.int32)[hit, 77] = bits
    got = binding.lora_add(x, a, b, index, base=base)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[hit] = True
    only_these(got, clean, bad)
    x.view(torch.int32)[(index < 0).nonzero()[0, 0], 3] = bits  # a vector without an adapter: base
    assert torch.equal(binding.lora_add(x, a, b, index, base=base)[~bad], clean[~bad])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nvec", [4, 40, 200])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_lora_no_numbers_in_weights(value, nvec, dtype):
    """Within the rank: in A the adapter's vectors, in B one output of them.  (An infinite weight of B
    may give NaN: the parts of a rank value may be zero or of both signs.)"""
    x, a, b, index, base = lora_inputs(dtype, nvec)
    ranks = torch.tensor([24, 17, 8], dtype=torch.int32, device="cuda")
    clean = binding.lora_add(x, a, b, index, ranks=ranks, base=base)
    mine = index == 1
    a1, b1 = a.clone(), b.clone()
    a1[1, 16, 263] = value
    bad = torch.zeros_like(clean, dtype=torch.bool)
    bad[mine] = True
    only_these(binding.lora_add(x, a1, b, index, ranks=ranks, base=base), clean, bad)
    b1[1, 33, 16] = value
    bad[:] = False
    bad[mine, 33] = True
    only_these(binding.lora_add(x, a, b1, index, ranks=ranks, base=base), clean, bad, math.isnan(value))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_lora_infinity_in_x_and_scale(value, dtype):
    x, a, b, index, base = lora_inputs(dtype, 40)
    clean = binding.lora_add(x, a, b, index, base=base)
    scale = torch.tensor([1.0, 1.0, value], device="cuda")
    got = binding.lora_add(x, a, b, index, scale, base=base)
    assert not torch.isfinite(got[index == 2]).any()
    assert torch.equal(got[index != 2], clean[index != 2])
    x[0, 0] = value
    index[0] = 0
    clean = binding.lora_add(normal(1, 40, 264), a, b, index, base=base)
    got = binding.lora_add(x, a, b, index, base=base)
    assert not torch.isfinite(got[0]).any() and torch.equal(got[1:], clean[1:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("adapters", [200, 9])  # in the pool, whatever is used: buckets of eight, of sixteen too
@pytest.mark.parametrize("nvec,used", [(15, 3), (17, 17), (35, 35), (37, 5), (37, 37), (72, 36), (72, 72), (73, 73), (130, 2),
                                       (130, 130), (300, 3), (511, 100), (513, 7), (1025, 150)])
def test_lora_buckets_around_what_runs_at_once(nvec, used, adapters, dtype):
    """The device counts the buckets: clusters whole, in halves, several rounds of either, and vectors without an
    adapter among them, alone in a half or all of them."""
    used = min(used, adapters)
    g = torch.Generator().manual_seed(nvec)
    of = (torch.randperm(nvec, generator=g) % used).to(torch.int32) + adapters - used
    of[torch.randperm(nvec, generator=g)[:nvec // 7]] = -1
    x, base = normal(5, nvec, 136), normal(6, nvec, 50)
    a, b = normal(7, adapters, 16, 136, std=0.1, dtype=dtype), normal(8, adapters, 50, 16, dtype=dtype)
    ranks = (torch.arange(adapters, dtype=torch.int32) * 7 % 17).cuda()
    for index in (of.cuda(), torch.full((nvec,), -1, dtype=torch.int32, device="cuda")):
        got = binding.lora_add(x, a, b, index, ranks=ranks, base=base)
        want, mag = lora_reference(x, a, b, index, None, ranks, base)
        within(got, want, lora_tol(136, mag))
        assert torch.equal(got[index < 0], base[index < 0])
        assert torch.equal(got, binding.lora_add(x, a, b, index, ranks=ranks, base=base))
    assert binding.device_status() == 0


# ------------------------------------------------------------------- norm --
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [96, 4096, 24608])
def test_norm_of_a_row_with_nan(n, dtype):
    """NaN in residual_out there, in y and the q8_0 scales of the row, as the quantize call gives them of y;
    the other rows as they were."""
    x, r, w = normal(60, 3, n, dtype=dtype), normal(61, 3, n, dtype=dtype), 1 + normal(62, n, std=0.1)
    clean = binding.add_rms_norm(x, w, residual=r, out="both")
    x[1, n // 3] = math.nan
    got = binding.add_rms_norm(x, w, residual=r, out="both")
    bad = torch.zeros(3, n, dtype=torch.bool, device="cuda")
    bad[1, n // 3] = True
    only_these(got.residual, clean.residual, bad)
    bad[1] = True
    only_these(got.y, clean.y, bad)
    q, d = binding.quantize(got.y[1].float())
    assert torch.isnan(got.d[1].view(torch.float16)).all() and torch.equal(q, got.q[1]) and torch.equal(d, got.d[1])
    assert torch.equal(got.q[~bad], clean.q[~bad]) and torch.equal(got.d[::2], clean.d[::2])


# ---------------------------------------------------------------- streams --
def stream_calls():
    """Each operator, and the first tensor that it allocates."""
    x, w, r = normal(10, 512, 4096), 1 + normal(11, 4096, std=0.1), normal(12, 512, 4096)
    a, b = normal(13, 2, 16, 4096, std=0.02, dtype=torch.bfloat16), normal(14, 2, 4096, 16, dtype=torch.bfloat16)
    index = torch.arange(512, dtype=torch.int32, device="cuda") % 3 - 1
    c = Cache([(700, 900), (1, 8000), (5, 300)], 32, 8, 128, 64, torch.bfloat16)
    q, kv = normal(15, c.total, 32 * 128), normal(16, c.total, 8 * 128)
    heads = normal(17, c.total, 32, 128, dtype=torch.bfloat16)
    cs = rope_table(8000, 128)
    ws = binding.paged_attention_workspace(700, 32, 8, 128)
    return dict(
        norm=(lambda **k: binding.add_rms_norm(x, w, residual=r, out="both", **k), 512 * 4096 * 4),
        lora=(lambda **k: [binding.lora_add(x, a, b, index, base=r, **k)], 512 * 4096 * 4),
        rope=(lambda **k: [binding.rope_append(q, kv, kv, cs, *c.args(), **k)], c.total * 32 * 128 * 2),
        attention=(lambda **k: [binding.paged_attention(heads, *c.args(), max_new=700, **k)], c.total * 32 * 128 * 2),
        workspace=(lambda **k: [binding.paged_attention(heads, *c.args(), max_new=700, **k)], ws))


@pytest.mark.parametrize("name", ["norm", "lora", "rope", "attention", "workspace"])
def test_another_stream_leaves_pending_work_alone(name):
    """A call on another stream allocates its outputs: not from memory that was given back while work
    pending on the current stream still reads it."""
    call, size = stream_calls()[name]
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    block = torch.full((size // 4,), 7, dtype=torch.int32, device="cuda")
    keep = torch.empty_like(block)
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(100_000_000)
    keep.copy_(block)
    del block
    got = call(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert (keep == 7).all()


def test_the_current_stream_is_the_default():
    call, _ = stream_calls()["lora"]
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])


# ------------------------------------------------------ axes of one entry --
def one_row(x):
    """x [1, ...] with a stride of its first axis that no kernel would take, 16-byte aligned."""
    return x.as_strided(x.shape, (x[0].numel() + 3,) + x.stride()[1:])


def test_one_row_may_have_any_stride():
    x, w, base = normal(20, 1, 4096), 1 + normal(21, 4096, std=0.1), normal(22, 1, 300)
    want = binding.add_rms_norm(x, w, residual=x, out="both")
    got = binding.add_rms_norm(one_row(x), w, residual=one_row(x), out="both", y=one_row(torch.empty_like(x)))
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    a, b = normal(23, 2, 16, 4096, std=0.02, dtype=torch.bfloat16), normal(24, 2, 300, 16, dtype=torch.bfloat16)
    index = torch.ones(1, dtype=torch.int32, device="cuda")
    want = binding.lora_add(x, a, b, index, base=base)
    assert torch.equal(binding.lora_add(one_row(x), a, b, index, base=one_row(base), out=one_row(torch.empty_like(base))), want)
    inplace = one_row(base.clone())
    assert torch.equal(binding.lora_add(x, a, b, index, out=inplace), want)


@pytest.mark.parametrize("kv_heads,page", [(1, 16), (2, 512)])
def test_axes_of_one_entry_may_have_any_stride(kv_heads, page):
    """One token, one head of keys, one page, one sequence: their strides are not looked at."""
    c = Cache([(1, 300)], 4, kv_heads, 64, page, torch.bfloat16, spare=0)
    q, kv = normal(25, 1, 256), normal(26, 1, kv_heads * 64)
    cs = rope_table(300, 64)
    turned = binding.rope_append(q, kv, kv, cs, *c.args())
    want = binding.paged_attention(turned, *c.args(), max_new=1)
    odd = lambda t, off: t.as_strided(t.shape, [s if n > 1 else s + off for n, s in zip(t.shape, t.stride())])  # noqa: E731
    args = [odd(c.k, 3), odd(c.v, 5), odd(c.table, -1), c.kv_len, c.new_start]
    got = binding.rope_append(one_row(q), one_row(kv), one_row(kv), cs, *args)
    assert torch.equal(got, turned)
    assert torch.equal(binding.paged_attention(odd(turned, 1), *args, max_new=1, out=odd(torch.empty_like(turned), 7)), want)
    pkv = binding.paged_kv(*args, 1)
    assert pkv.table_stride == c.table.shape[1] and pkv.head_stride == 64


# -------------------------------------------- attention: what is no number --
# (new, length) of the sequences and the table's least tokens: which form takes the call.
FORMS = dict(cluster=([(20, 300), (1, 40)], 0), shares=([(6, 3000), (2, 2)], 7300), one=([(7, 5000)], 7300),
             tensor=([(300, 1500), (1, 700), (70, 90)], 7300), split=([(100, 9000)], 7300))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_attend_values_that_earlier_tokens_do_not_see(form, dim, dtype, value, monkeypatch):
    """A value of a new token that is no number: its column of the rows from that token on, no other bit."""
    seqs, least = FORMS[form]
    monkeypatch.setattr(Cache, "least_tokens", least)
    c = Cache(seqs, 8, 2, dim, 32, dtype)
    q = normal(30, c.total, 8, dim, dtype=dtype)
    clean = binding.paged_attention(q, *c.args(), max_new=max(c.new))
    new, n = seqs[0]
    bad = torch.zeros_like(clean, dtype=torch.bool)
    for token, head, col in ((new - 1, 0, 3), (new // 2, 1, dim - 1), (1, 1, 17)):
        pos = n - new + token
        c.v[c.table[0, pos // 32], pos % 32, head, col] = value
        bad[token:new, head * 4:head * 4 + 4, col] = True
        got = binding.paged_attention(q, *c.args(), max_new=max(c.new))
        only_these(got, clean, bad, math.isnan(value))
        if math.isinf(value):
            assert (got[bad] == value).all()
    old = n - new - 1  # and one that all rows see
    c.v[c.table[0, old // 32], old % 32, 0, 5] = value
    bad[:new, :4, 5] = True
    only_these(binding.paged_attention(q, *c.args(), max_new=max(c.new)), clean, bad, math.isnan(value))
    assert binding.device_status() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("form", FORMS)
def test_attend_keys_that_earlier_tokens_do_not_see(form, dim, monkeypatch):
    seqs, least = FORMS[form]
    monkeypatch.setattr(Cache, "least_tokens", least)
    c = Cache(seqs, 8, 2, dim, 32, torch.bfloat16)
    q = normal(31, c.total, 8, dim, dtype=torch.bfloat16)
    clean = binding.paged_attention(q, *c.args(), max_new=max(c.new))
    new, n = seqs[0]
    token = new // 3
    pos = n - new + token
    c.k[c.table[0, pos // 32], pos % 32, 1, 9] = math.nan
    bad = torch.zeros_like(clean, dtype=torch.bool)
    bad[token:new, 4:] = True
    only_these(binding.paged_attention(q, *c.args(), max_new=max(c.new)), clean, bad)


@pytest.mark.parametrize("form", [*FORMS, "first"])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_all_scores_minus_infinity(dim, form, monkeypatch):
    """A row whose visible scores are all -inf has no weights to divide by: NaN, not the zeros of a row
    that sees no key."""
    seqs, least = ([(3, 2)], 0) if form == "first" else FORMS[form]
    monkeypatch.setattr(Cache, "least_tokens", least)
    c = Cache(seqs, 8, 2, dim, 32, torch.bfloat16)
    for i, n in enumerate(c.len):
        pos = torch.arange(n, device="cuda")
        c.k[c.table[i, pos // 32].long(), pos % 32, :, 0] = 1
    q = normal(32, c.total, 8, dim, dtype=torch.bfloat16)
    clean = binding.paged_attention(q, *c.args(), max_new=max(c.new))
    bad = torch.zeros_like(clean, dtype=torch.bool)
    for token in {seqs[0][0] - 1, 1}:
        q[token, 2, 0] = -math.inf
        bad[token, 2] = True
    only_these(binding.paged_attention(q, *c.args(), max_new=max(c.new)), clean, bad)
    if form == "first":
        assert (clean[0] == 0).all()


@pytest.mark.parametrize("spread", [0.0, 0.3, 2.0])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch,new", [(1, 2048), (64, 1)])  # the tensor cores, whole items; the streaming kernel
def test_attend_long_sums_of_one_sign(batch, new, dim, dtype, spread):
    """Positive values, the same for all of 16384 keys, are their own mean: what the MMAs cut from a sum does
    not average out here.  Each of 1024 cuts at most an ulp (2^-23) of the sum, 2^-13 together; a weight is off
    by U for its product with v, and the result by U."""
    length, page = 16384, 64
    k = normal(40, batch * length // page, page, 8, dim, dtype=dtype)
    column = (0.5 + torch.rand(dim, generator=torch.Generator().manual_seed(41))).to(dtype).cuda()
    v = column.expand_as(k).contiguous()
    table = torch.arange(batch * length // page, dtype=torch.int32, device="cuda").view(batch, -1)
    kv_len = torch.full((batch,), length, dtype=torch.int32, device="cuda")
    starts = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * new
    q = normal(42, batch * new, 32, dim, std=spread, dtype=dtype)
    got = binding.paged_attention(q, k, v, table, kv_len, starts, max_new=new)
    want = column.to(torch.float64).expand(got.shape)
    within(got, want, (2 * U[dtype] + 2.0 ** -13) * want)


# ------------------------------------------------- caches past 32 bits --
@pytest.mark.parametrize("least", [0, 7300])
def test_far_pages_in_every_form(least, monkeypatch):
    """Pages at the end of a cache of more than 2^32 elements: rotary append by bits, then attention by clusters
    (the short table), and by shares of the keys and on the tensor cores (the long one: few rows, many)."""
    monkeypatch.setattr(Cache, "least_tokens", least)
    page, kv_heads, dim, heads = 256, 8, 128, 16
    pages = (1 << 32) // (page * kv_heads * dim) + 8
    big = [torch.empty(pages, page, kv_heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for seqs in ([(1, 600), (20, 500)], [(40, 900), (3, 300)]):
        c = Cache(seqs, heads, kv_heads, dim, page, torch.bfloat16, spare=0)
        used = c.k.shape[0]
        far = torch.where((c.table >= 0) & (c.table < used), c.table + (pages - used), c.table)
        for b, near in zip(big, (c.k, c.v)):
            b[pages - used:] = near
        q, kv = normal(50, c.total, heads * dim), normal(51, c.total, kv_heads * dim)
        cs = rope_table(900, dim)
        turned = binding.rope_append(q, kv, kv, cs, *c.args())
        assert torch.equal(binding.rope_append(q, kv, kv, cs, *big, far, c.kv_len, c.new_start), turned)
        for b, near in zip(big, (c.k, c.v)):
            assert torch.equal(b[pages - used:].view(torch.int16), near.view(torch.int16))
        for i, n in enumerate(c.len):
            pos = torch.arange(n, device="cuda")
            at = c.table[i, pos // page].long(), pos % page
            c.dense[i] = c.k[at], c.v[at]
        c.k, c.v, c.table = *big, far
        for max_new in {1, max(c.new)}:
            check_attend(c, heads, torch.bfloat16, dim, max_new=max_new)
