"""The decoder layer that runs the operators and the products together: a
prompt at once and the same tokens one by one take different kernels (batched
and single products, the tensor-core and the streaming attention) and must
agree; and each stage is the binding's own call, bit for bit."""
import pytest
import torch

from decode_q1_gemv_gb300 import binding, layer

pytestmark = pytest.mark.gpu

SHAPES = (("q", 512, 256), ("k", 256, 256), ("v", 256, 256), ("o", 256, 512), ("gate", 640, 256), ("up", 640, 256),
          ("down", 256, 640))


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    binding.device_status()


def make(adapters=2):
    return layer.synthetic_layer(SHAPES, dim=128, positions=256, adapters=adapters, rank=8, seed=9)


def test_prompt_at_once_and_token_by_token_agree():
    """Two runs may round a quant either way at each of the layer's four
    quantizations: a step of amax/127, at most 3.5 % of a block's root mean
    square where its largest value is 4.5 times that, half a step (uniform:
    0.3 of it, 1 %) on average and only where the runs differ at all; 5 % of the
    output's norm bounds their sum."""
    m = make()
    tokens, seqs = 40, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(seqs, tokens, 256, generator=g, device="cuda")
    index = torch.tensor([-1, 0, 1], dtype=torch.int32, device="cuda")
    whole = layer.PagedCache(seqs, 20, 16, 2, 128, 64)
    whole.extend([tokens] * seqs)
    out, res = m(x.view(-1, 256), None, whole, index.repeat_interleave(tokens))
    out = out.view(seqs, tokens, 256)
    steps = layer.PagedCache(seqs, 20, 16, 2, 128, 64)
    for t in range(tokens):
        steps.extend([1] * seqs)
        one, _ = m(x[:, t].contiguous(), None, steps, index)
        off = (one - out[:, t]).norm() / out[:, t].norm()
        assert off < 0.05, (t, off.item())
    assert binding.device_status() == 0


@pytest.mark.parametrize("tokens", [1, 5, 70])
def test_the_layer_is_its_calls(tokens):
    """The attention half of the layer, call by call."""
    m = make(adapters=0)
    x = torch.randn(tokens, 256, device="cuda")
    r = torch.randn(tokens, 256, device="cuda")
    caches = []
    for _ in range(2):
        c = layer.PagedCache(1, 6, 16, 2, 128, 96)
        c.extend([tokens])
        caches.append(c)
    out, residual = m(x, r, caches[0])
    n = binding.add_rms_norm(x, m.norms[0], residual=r)
    q, k, v = (torch.cat([binding.gemm_small(m.packed[p], *m.shape[p], n.q[t:t + 64], n.d[t:t + 64])
                          for t in range(0, tokens, 64)]) for p in "qkv")
    c = caches[1]
    a = binding.paged_attention(binding.rope_append(q, k, v, m.cos_sin, *c.args()), *c.args(), max_new=tokens)
    qa, da = binding.quantize(a.view(tokens, -1).float())
    o = torch.cat([binding.gemm_small(m.packed["o"], *m.shape["o"], qa[t:t + 64], da[t:t + 64]) for t in range(0, tokens, 64)])
    want = binding.add_rms_norm(o, m.norms[1], residual=n.residual).residual
    assert torch.equal(residual, want) and torch.isfinite(out).all()
    used = -(-tokens // 16)
    for a, b in ((caches[0].k, c.k), (caches[0].v, c.v)):
        pages = c.table[0, :used].long()
        filled = torch.arange(used * 16, device="cuda") < tokens
        assert torch.equal(a[pages].flatten(0, 1)[filled], b[pages].flatten(0, 1)[filled])


def test_the_cache_refuses_what_it_cannot_hold():
    c = layer.PagedCache(2, 3, 16, 1, 64, 32)
    with pytest.raises(ValueError, match="no free pages"):
        c.extend([20, 20])
    with pytest.raises(ValueError, match="outgrows"):
        c.extend([33, 1])
    with pytest.raises(ValueError, match="one count"):
        c.extend([1])
    c.extend([16, 1])
    c.extend([1, 0])
    with pytest.raises(ValueError, match="no free pages"):
        c.extend([0, 16])
    assert c.lengths == [17, 1] and c.kv_len.tolist() == [17, 1] and c.new_start.tolist() == [0, 1, 1]
