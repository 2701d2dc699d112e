"""The decoder layer over tables of every length: what a prompt at once gives and what
its tokens give one by one, with the attention by clusters (a short table), on the
tensor cores and by shares of the keys (a table too long for clusters)."""
import math

import pytest
import torch

from decode_q1_gemv_gb300 import binding, layer
from tests.test_gpu_layer import make
from tests.test_gpu_ops import lora_reference, lora_tol, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    binding.device_status()


@pytest.mark.parametrize("whole_tokens,step_tokens", [(64, 64), (8192, 64), (8192, 8192)])
def test_prompt_at_once_and_token_by_token_agree(whole_tokens, step_tokens):
    """80 rows a key head: the tensor-core kernel where the table is long.  The bound is that of
    test_gpu_layer.py: four quantizations, each a step off at most where the runs differ."""
    m = make()
    tokens, seqs = 40, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn(seqs, tokens, 256, generator=g, device="cuda")
    index = torch.tensor([-1, 0, 1], dtype=torch.int32, device="cuda")
    whole = layer.PagedCache(seqs, 20, 16, 2, 128, whole_tokens)
    whole.extend([tokens] * seqs)
    out, _ = m(x.view(-1, 256), None, whole, index.repeat_interleave(tokens))
    out = out.view(seqs, tokens, 256)
    steps = layer.PagedCache(seqs, 20, 16, 2, 128, step_tokens)
    for t in range(tokens):
        steps.extend([1] * seqs)
        one, _ = m(x[:, t].contiguous(), None, steps, index)
        off = (one - out[:, t]).norm() / out[:, t].norm()
        assert off < 0.05, (t, off.item())
    assert binding.device_status() == 0


def test_more_tokens_than_one_adapter_call_takes():
    m = make(adapters=2)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    tokens = 65535 + 40
    x = torch.randn(tokens, 256, generator=g, device="cuda")
    index = (torch.arange(tokens, device="cuda") % 3 - 1).to(torch.int32)
    out = m._adapt("v", x, torch.zeros(tokens, 256, device="cuda"), index)
    a, b, scale = m.adapters["v"]
    for part in (slice(0, 100), slice(65500, 65535), slice(65535, tokens)):
        want, mag = lora_reference(x[part], a, b, index[part], scale, None, torch.zeros_like(out[part]))
        within(out[part], want, lora_tol(256, mag))


def test_adapters_of_different_ranks():
    """(a, b, scale, ranks): what lies past a rank is not used."""
    m, plain = make(adapters=2), make(adapters=2)
    x = torch.randn(9, 256, device="cuda")
    index = torch.arange(9, dtype=torch.int32, device="cuda") % 3 - 1
    ranks = torch.tensor([3, 8], dtype=torch.int32, device="cuda")
    for name, (a, b, scale) in m.adapters.items():
        plain.adapters[name] = (a.clone(), b.clone(), scale)
        plain.adapters[name][0][0, 3:] = 0
        a[0, 3:] = math.nan
        m.adapters[name] = (a, b, scale, ranks)
    outs = []
    for layer_ in (m, plain):
        c = layer.PagedCache(1, 2, 16, 2, 128, 32)
        c.extend([9])
        outs.append(layer_(x, None, c, index))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
