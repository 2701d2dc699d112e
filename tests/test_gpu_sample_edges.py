"""Sampling where its blocks and clusters pass what they found from one step to the next: every combination of cuts,
again and again, with the device full."""
import pytest
import torch

from decode_q1_gemv_gb300 import binding
from tests.test_gpu_sample import TYPES, expected, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 128256), (19, 32000), (76, 9001), (200, 3001)])
@pytest.mark.parametrize("settings", [dict(top_k=401), dict(top_k=600), dict(top_k=2500), dict(top_k=600, min_p=0.02),
                                      dict(top_k=600, top_p=0.8), dict(top_p=0.8), dict(temperature=8.0, top_k=2500),
                                      dict(temperature=8.0, top_k=2500, top_p=0.6)])
def test_cuts_again_and_again(settings, rows, vocab, dtype):
    """Top-k with and without top-p: the bin that top-k reaches into is counted while the bins to look at are found."""
    x, u = inputs(rows, rows, vocab, dtype)
    want = expected(x, u, **settings)
    outs = [binding.sample(x, u, **settings) for _ in range(40)]
    for o in outs:
        assert o.tolist() == want


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [2, 150])
@pytest.mark.parametrize("settings", [dict(top_k=40), dict(top_k=400, min_p=0.5), dict(top_k=40, top_p=0.5)])
def test_small_top_k_among_many_equal_tokens(settings, rows, dtype):
    """More tokens reach the threads' value than a list holds, so that counts decide."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    x = torch.randint(3, (rows, 20000), generator=g, device="cuda").to(dtype)
    u = torch.rand(rows, generator=g, device="cuda")
    want = expected(x, u, **settings)
    outs = [binding.sample(x, u, **settings) for _ in range(40)]
    for o in outs:
        assert o.tolist() == want


@pytest.mark.parametrize("rest,kept", [(-20.0, 2), (-30.0, 2), (-31.0, 1), (-50.0, 1)])
def test_two_equal_maxima_and_half_of_the_sum(rest, kept):
    """top_p 0.5 of two equal maxima is the first one alone, unless others weigh something: e^-30 is 2^-43.3, e^-31 2^-44.7,
    which is below the last bit of the weights."""
    x = torch.full((2, 100), -torch.inf, device="cuda")
    x[:, [40, 70]] = 3.0
    x[:, 90] = 3.0 + rest
    u = torch.tensor([0.25, 0.75], device="cuda")
    assert binding.sample(x, u, top_p=0.5).tolist() == [40, 70 if kept == 2 else 40]
