"""Attention over a q8_0 cache, row by row with what the row's own keys allow: scales of very different sizes, and the
bounds of the kernel for few rows wherever that one runs."""
import math

import pytest
import torch

from decode_q1_gemv_gb300 import binding
from tests.test_gpu_cache8 import TYPES, Cache8, attend_reference
from tests.test_gpu_ops import F64, TINY, U, U32, normal, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    binding.device_status()


def few_rows(c, heads, max_new):
    """Tokens that certainly go to the kernel for few rows, whose keys and values are exact: all tokens of a call with at
    most 64 rows a key head (32 with one sequence), else those of sequences of at most 16 among several."""
    group = heads // c.kv_heads
    batch = len(c.new)
    whole = min(max_new, c.total) <= (32 if batch == 1 else 64) // group
    return torch.tensor([whole or (batch > 1 and n * group <= 16) for n in c.new for _ in range(n)], device="cuda")


def heaviest(c, q, scale):
    """Of each row: the largest product of a visible key's weight (of all of them 1) and its largest value, and of a weight alone."""
    out, top = (torch.zeros(q.shape[:2], dtype=F64, device="cuda") for _ in range(2))
    group, at = q.shape[1] // c.kv_heads, 0
    for (k, v), new, n in zip(c.dense, c.new, c.len):
        if new and n:
            hidden = torch.arange(n, device="cuda") > torch.arange(n - new, n, device="cuda")[:, None]
            s = torch.einsum("rhd,khd->rhk", q[at:at + new].to(F64), k.repeat_interleave(group, 1)) * scale
            w = torch.softmax(s.masked_fill(hidden[:, None], -math.inf), -1).nan_to_num(0.0)
            out[at:at + new] = (w * v.abs().amax(-1).repeat_interleave(group, 1).T).amax(-1)
            top[at:at + new] = w.amax(-1)
        at += new
    return out, top


# Few rows: a weight times its key's scale is rounded once to f16, off by 2^-11 of itself; below f16's normal numbers by
# 2^-25 of the largest such product of the keys that the row sees (which, times a quant of 127, is a weight times a
# key's largest value), or of 2^-40 of the largest weight where all scales are smaller.  Keys and values are exact, q is
# but for elements below 2^-17 of a row's largest (2^-22 covers them).
# Many rows: as attend_tol; values are off by 2^-39 of the sequence's largest where they are 2^-28 of it and less.
def row_tol(c, q, scale, max_new, want):
    out, mag, total, seen, size = want
    dtype, dim = q.dtype, q.shape[2]
    few = few_rows(c, q.shape[1], max_new)[:, None]
    bf = dtype == torch.bfloat16
    exact = torch.full((), 2.0 ** -22, dtype=F64, device="cuda")
    key = torch.where(few, exact, 2.0 ** -11 if bf else 2.0 ** -22)
    heavy, top = heaviest(c, q, scale)
    most = max((v.abs().max().item() for _, v in c.dense if v.numel()), default=0.0)
    small = torch.where(few, 2.0 ** -25 * seen[:, None] * (heavy + 127 * 2.0 ** -40 * top),
                        2.0 ** -25 * seen[:, None] / total * heavy.new_tensor(most) + 2.0 ** -39 * most)
    part = (2.0 ** -11 + key + 1e-6) + (2 * key + 2 * dim * U32) * size
    return part[..., None] * mag + small[..., None] + U[dtype] * out.abs() + TINY[dtype]


def check_rows(c, heads, dtype, max_new=None, scale=None, seed=70, q=None):
    max_new, scale = max_new or max(c.new), c.dim ** -0.5 if scale is None else scale
    if q is None:
        q = normal(seed, max(1, c.total), heads, c.dim, dtype=dtype)[:c.total]
    got = binding.paged_attention_q8(q, *c.args(), max_new=max_new, scale=scale)
    want = attend_reference(c, q, scale)
    within(got, want[0], row_tol(c, q, scale, max_new, want))
    assert binding.device_status() == 0
    return got


@pytest.mark.parametrize("width", [None, 500])  # clusters, shares of the keys
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [2, 5, 16])
@pytest.mark.parametrize("dtype,std,factor", [(torch.bfloat16, 1.0, 2.0 ** 13), (torch.bfloat16, 2.0 ** -10, 2.0 ** 28), (torch.float16, 1.0, 2.0 ** 13)])
def test_a_later_tokens_scale_is_not_an_earlier_rows(dtype, std, factor, new, dim, width):
    """The last new token's values are far larger: only the row that sees them may lose bits to them."""
    c = Cache8([(new, 300), (1, 70)], 2, dim, 16, width=width)
    k, v = normal(1, 300, 2, dim), normal(2, 300, 2, dim, std=std)
    v[-1] = v[-1].clamp(-2 * std, 2 * std) * factor
    c.put(0, k, v)
    check_rows(c, 4, dtype)


@pytest.mark.parametrize("width", [None, 500])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 4])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_scale_that_hardly_weighs(dtype, new, dim, width):
    """A key early on with a weight below 2^-50 of the others' and values 2^22 times theirs."""
    c = Cache8([(new, 400), (1, 70)], 1, dim, 16, width=width)
    q = normal(70, c.total, 4, dim, dtype=dtype).abs() + 0.5
    k, v = normal(1, 400, 1, dim) * 0.1, normal(2, 400, 1, dim, std=2.0 ** -8)
    k[7] = -2.0
    v[7] = 2.0 ** 14
    c.put(0, k, v)
    check_rows(c, 4, dtype, q=q, scale=0.6)


@pytest.mark.parametrize("width", [None, 500])
@pytest.mark.parametrize("new", [1, 3, 16, 90])
@pytest.mark.parametrize("dtype", TYPES)
def test_zeros_and_small_scales_among_the_values(dtype, new, width):
    """Tokens of zeros (scales of zero), of values near f16's least scales, and usual ones, in runs longer than a chunk."""
    for sizes in ([0.0, 1.0], [2.0 ** -24, 0.0, 2.0 ** -12], [0.0, 2.0 ** -20], [0.0]):
        c = Cache8([(new, 330), (new, 50)], 2, 64, 16, width=width)
        for i, n in enumerate(c.len):
            v = normal(18 + i, n, 2, 64)
            run = torch.arange(n, device="cuda") // 40 % len(sizes)
            c.put(i, normal(8 + i, n, 2, 64), v * torch.tensor(sizes, device="cuda")[run][:, None, None])
        check_rows(c, 4, dtype)


@pytest.mark.parametrize("width", [None, 500])
@pytest.mark.parametrize("new", [1, 5, 16, 90])
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_scales_below_zero(which, new, width):
    """Quants and scales of the other sign are the same values."""
    c = Cache8([(new, 300), (1, 70)], 2, 128, 16, width=width)
    q = normal(70, c.total, 4, 128, dtype=torch.bfloat16)
    for name in ("k", "v"):
        if which in (name, "both"):
            quants, scales = getattr(c, name), getattr(c, name + "s")
            quants.copy_(-quants)
            scales.copy_(-scales)
    check_rows(c, 4, torch.bfloat16, q=q)


@pytest.mark.parametrize("width", [None, 500])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 128), (2, 2, 64), (5, 1, 128), (8, 1, 64), (3, 1, 64)])
@pytest.mark.parametrize("new,length", [(2, 2), (3, 50), (8, 300), (15, 200), (32, 1500), (64, 64)])
def test_chunks_within_each_kernels_bounds(new, length, heads, kv_heads, dim, dtype, width):
    check_rows(Cache8([(new, length)], kv_heads, dim, 16, width=width), heads, dtype)


@pytest.mark.parametrize("width", [None, 500])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("max_new", [None, 1, 4096])
def test_batches_within_each_kernels_bounds(max_new, dim, dtype, width):
    seqs = [(1, 700), (0, 40), (33, 33), (1, 1), (140, 500), (4, 70), (2, 2000), (17, 300)]
    check_rows(Cache8(seqs, 2, dim, 16, width=width), 8, dtype, max_new=max_new)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("new", [1, 5])
@pytest.mark.parametrize("kstd,vstd,qstd", [(1e4, 1e4, 1e-4), (1e-4, 1e-4, 100.0), (30.0, 100.0, 0.03), (1.0, 1e-5, 1.0)])
def test_any_size_of_values_within_the_bounds_of_few_rows(kstd, vstd, qstd, new, dtype):
    if dtype == torch.float16 and (vstd > 1e3 or qstd < 1e-3):
        pytest.skip("beyond f16")
    c = Cache8([(new, 400), (new, 90)], 2, 64, 16)
    for i, n in enumerate(c.len):
        c.put(i, normal(8 + i, n, 2, 64, std=kstd), normal(18 + i, n, 2, 64, std=vstd))
    check_rows(c, 4, dtype, scale=0.1, q=normal(73, c.total, 4, 64, std=qstd, dtype=dtype))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("seqs,max_new", [([(1, 700), (1, 90), (1, 1)], 1), ([(90, 400), (1, 700), (3, 90), (2, 2)], 90), ([(70, 300)], 70)])
def test_appended_over_and_over_between_calls(seqs, max_new, dtype, dim):
    """The new tokens' slots are written again before every call of a graph: each call sees what was written last, in
    the launches that do not wait for the one before them too."""
    heads, kv_heads, calls = 8, 2, 6
    c = Cache8(seqs, kv_heads, dim, 16, width=70)
    rows = [normal(60 + i, c.total, (heads + 2 * kv_heads) * dim) for i in range(calls)]
    cs = torch.zeros(700, dim, device="cuda")
    cs[:, :dim // 2] = 1  # no turn
    ws = torch.empty(binding.paged_attention_q8_workspace(max_new, heads, kv_heads, dim, 70 * 16, 4, dtype), dtype=torch.uint8, device="cuda")

    def step(i):
        q, k, v = rows[i].split([heads * dim, kv_heads * dim, kv_heads * dim], 1)
        turned = binding.rope_append_q8(q, k, v, cs, *c.args(), dtype=dtype)
        return binding.paged_attention_q8(turned, *c.args(), max_new=max_new, workspace=ws)

    want = []
    for i in range(calls):
        want.append(step(i))
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [step(i) for i in range(calls)]
    for _ in range(20):
        for o in outs:
            o.fill_(7.0)
        g.replay()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    for _ in range(20):
        for o, w in zip([step(i) for i in range(calls)], want):
            assert torch.equal(o, w)
    assert binding.device_status() == 0
