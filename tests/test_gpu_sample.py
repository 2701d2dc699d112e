"""Sampling against its definition in 64 bits: whole numbers, equal or not."""
import math

import numpy as np
import pytest
import torch

from decode_q1_gemv_gb300 import binding

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
BELOW_ONE = 1 - 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def expected(logits, uniform, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row after the other: sorted, cut, drawn in the vocabulary's order."""
    x = logits.double().cpu().numpy()
    u = uniform.double().cpu().numpy()

    def each(v, kind):
        return v.cpu().numpy() if isinstance(v, torch.Tensor) else np.full(x.shape[0], v, dtype=kind)

    settings = zip(each(temperature, np.float32), each(top_k, np.int64), each(top_p, np.float32), each(min_p, np.float32))
    out = []
    for row, draw, (t, k, p, m) in zip(x, u, settings):
        t, p, m = float(t), float(p), float(m)
        if np.isnan(row).any() or row.max() in (math.inf, -math.inf) or any(map(math.isnan, (t, p, m, draw))):
            out.append(-1)
            continue
        best = int(row.argmax())
        if t <= 0:
            out.append(best)
            continue
        tokens = np.argsort(-row, kind="stable")
        tokens = tokens[row[tokens] > -math.inf]
        if k > 0:
            tokens = tokens[:k]
        w = np.exp((row[tokens] - row[best]) / t)
        if p < 1:
            count = max(1, int(np.searchsorted(np.cumsum(w), p * w.sum(), side="left")) + 1)
            tokens, w = tokens[:count], w[:count]
        stay = w >= min(m, 1.0)
        stay[0] = True
        tokens, w = tokens[stay], w[stay]
        order = np.argsort(tokens)
        sums = np.cumsum(w[order])
        at = int(np.searchsorted(sums, min(max(draw, 0.0), BELOW_ONE) * sums[-1], side="right"))
        out.append(int(tokens[order][min(at, len(tokens) - 1)]))
    return out


def inputs(seed, rows, vocab, dtype=torch.float32, std=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * std
    return x.to(dtype), torch.rand(rows, generator=g, device="cuda")


def check(x, u, **settings):
    got = binding.sample(x, u, **settings)
    assert got.dtype == torch.int32 and got.tolist() == expected(x, u, **settings)
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 100, 511, 512, 513, 1023, 2049, 4097, 32000, 128256, 151937])
@pytest.mark.parametrize("settings", [dict(), dict(temperature=0.0), dict(temperature=0.7, top_k=50, top_p=0.95), dict(top_p=0.9),
                                      dict(top_k=1), dict(top_k=3, min_p=0.3), dict(min_p=0.05), dict(temperature=3.0, top_k=600),
                                      dict(temperature=5.0, top_k=3000, top_p=0.8, min_p=0.01)])
def test_sizes_and_settings(settings, vocab, dtype):
    for rows in (1, 5):
        check(*inputs(vocab + rows, rows, vocab, dtype), **settings)


@pytest.mark.parametrize("rows", [1, 2, 3, 9, 10, 19, 20, 38, 39, 76, 77, 152, 153, 304, 305, 700])
def test_rows_do_not_depend_on_each_other(rows):
    """Clusters of every size, and rows past what runs at once."""
    x, u = inputs(rows, rows, 20001)
    some = dict(temperature=1.5, top_k=300, top_p=0.97)
    got = check(x, u, **some)
    for r in {0, rows // 2, rows - 1}:
        assert binding.sample(x[r:r + 1], u[r:r + 1], **some).tolist() == [got[r].item()]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 60000), (40, 3001), (3, 128256)])
def test_settings_of_each_row(rows, vocab, dtype):
    x, u = inputs(3, rows, vocab, dtype)
    rng = np.random.default_rng(rows)
    t = torch.tensor(rng.choice([0.0, 0.2, 0.7, 1.0, 4.0, -1.0, math.inf], rows), dtype=torch.float32, device="cuda")
    k = torch.tensor(rng.choice([0, -3, 1, 2, 40, 511, 513, 2000, vocab, vocab + 7], rows), dtype=torch.int32, device="cuda")
    p = torch.tensor(rng.choice([1.0, 2.0, 0.0, -1.0, 0.1, 0.9, 0.999], rows), dtype=torch.float32, device="cuda")
    m = torch.tensor(rng.choice([0.0, -1.0, 0.01, 0.5, 1.0, 7.0], rows), dtype=torch.float32, device="cuda")
    check(x, u, temperature=t, top_k=k, top_p=p, min_p=m)
    check(x, u, temperature=0.9, top_k=k, top_p=0.9, min_p=m)


@pytest.mark.parametrize("vocab", [5, 640, 4000, 100000])
@pytest.mark.parametrize("draw", [0.0, 0.25, 0.5, 0.75, BELOW_ONE, 1.0, 2.0, -1.0])
def test_equal_logits_and_borders(draw, vocab):
    """All weights are one: sums are whole, and a draw on a border takes the next token."""
    x, u = torch.full((2, vocab), -3.25, device="cuda"), torch.full((2,), draw, device="cuda")
    for settings in (dict(), dict(top_k=vocab // 5 * 4), dict(top_p=0.5), dict(top_k=vocab // 5 * 4, top_p=0.25), dict(min_p=1.0),
                     dict(temperature=0.0), dict(temperature=math.inf), dict(temperature=1e-30)):
        check(x, u, **settings)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("values", [2, 7, 100])
@pytest.mark.parametrize("settings", [dict(top_k=700), dict(top_p=0.6), dict(top_k=5000, top_p=0.6), dict(top_k=20000, top_p=0.99, min_p=0.2)])
def test_ties_across_the_threshold(settings, values, dtype):
    """Few different values, so that the threshold lies within equal ones, which stay by index; zeros of both signs are equal."""
    g = torch.Generator(device="cuda")
    g.manual_seed(values)
    x = (torch.randint(values, (6, 50000), generator=g, device="cuda") - values // 2).to(dtype) / 4
    x[:, ::3] = torch.where(x[:, ::3] == 0, -x[:, ::3].abs(), x[:, ::3])
    check(x, torch.rand(6, generator=g, device="cuda"), **settings)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("settings", [dict(), dict(top_k=100), dict(top_p=0.9), dict(temperature=0.0), dict(top_k=4000, top_p=0.95)])
def test_masked_tokens(settings, dtype):
    x, u = inputs(8, 5, 30000, dtype)
    x[torch.rand(x.shape, device="cuda") < 0.9] = -math.inf
    x[1] = -math.inf
    x[1, 12345] = -5.0
    x[2] = torch.finfo(dtype).min  # a mask of the type's lowest value
    x[2, [77, 29999]] = 1.0
    x[3, :29990] = -math.inf
    x[3, 29990:] = 0.5
    got = check(x, u, **settings)
    assert got[1] == 12345 and got[2] in (77, 29999)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("settings", [dict(), dict(temperature=0.0), dict(top_k=20, top_p=0.5)])
def test_rows_without_a_distribution(settings, dtype):
    x, u = inputs(9, 6, 5000, dtype)
    x[0] = -math.inf
    x[1, 4999] = math.nan
    x[2, 17] = math.inf
    x[3, 1] = -math.nan
    got = check(x, u, **settings)
    assert got[:4].tolist() == [-1] * 4 and (got[4:] >= 0).all()
    one = binding.sample(x[4:, :1], u[4:], **settings)
    assert one.tolist() == [0, 0]


def test_settings_that_are_nan():
    x, u = inputs(10, 6, 700)
    nan = lambda i, v: torch.tensor([math.nan if j == i else v for j in range(6)], dtype=torch.float32, device="cuda")  # noqa: E731
    u[4] = math.nan
    check(x, u, temperature=nan(0, 0.8), top_p=nan(1, 0.9), min_p=nan(2, 0.1), top_k=9)


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows_at_any_alignment(dtype):
    x, u = inputs(11, 7, 9000, dtype)
    for first, last in [(0, 9000), (1, 9000), (3, 8998), (5, 6), (7, 8000), (8, 8001)]:
        part = x[::2, first:last]
        for settings in (dict(), dict(top_k=30), dict(top_k=1000, top_p=0.9), dict(temperature=0.0)):
            check(part, u[::2].contiguous(), **settings)


@pytest.mark.parametrize("std", [0.01, 30.0, 1e4, 1e30])
def test_flat_and_sharp_logits(std):
    x, u = inputs(12, 8, 40000, std=std)
    for settings in (dict(), dict(top_k=700), dict(top_p=0.9), dict(top_k=900, top_p=0.5), dict(temperature=0.01), dict(temperature=1e4, top_p=0.3)):
        check(x, u, **settings)


@pytest.mark.parametrize("rows", [1, 3])
def test_largest_vocabulary(rows):
    x, u = inputs(13, rows, 1 << 19)
    for settings in (dict(), dict(temperature=2.0, top_p=0.95), dict(top_k=100), dict(temperature=0.0), dict(temperature=9.0, top_k=300000)):
        check(x, u, **settings)


@pytest.mark.parametrize("settings", [dict(temperature=1.0), dict(temperature=2.0, top_p=0.97), dict(temperature=0.8, top_k=40)])
def test_many_draws(settings):
    """2048 draws from rows of a real vocabulary's size: one that falls to the neighbouring token would be seen."""
    x, _ = inputs(14, 1, 32003)
    g = torch.Generator(device="cuda")
    g.manual_seed(15)
    u = torch.rand(2048, generator=g, device="cuda")
    check(x.expand(2048, -1), u, **settings)


def test_captured_on_another_stream_and_into_a_given_tensor():
    x, u = inputs(16, 20, 50001, torch.bfloat16)
    t = torch.full((20,), 0.9, device="cuda")
    out = torch.full((20,), -7, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert binding.sample(x, u, t, 40, out=out, stream=s).data_ptr() == out.data_ptr()
    torch.cuda.current_stream().wait_stream(s)
    assert out.tolist() == expected(x, u, t, 40)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        binding.sample(x, u, t, 40, out=out)
        binding.sample(x, u, t, 0, 0.9, out=out)
    for seed in (17, 18):
        x2, u2 = inputs(seed, 20, 50001, torch.bfloat16)
        x.copy_(x2), u.copy_(u2), t.fill_(0.1 * seed)
        g.replay()
        assert out.tolist() == expected(x, u, t, 0, 0.9)
