"""The decoder layer over a q8_0 cache, and the head: a prompt at once and token by token,
the stages call by call, and the next tokens."""
import pytest
import torch

from decode_q1_gemv_gb300 import binding, layer, synth
from tests.test_gpu_layer import make
from tests.test_gpu_sample import expected

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()
    binding.device_status()


def cache(seqs=1, tokens=96, pages=20):
    return layer.PagedCache(seqs, pages, 16, 2, 128, tokens, torch.int8)


@pytest.mark.parametrize("whole_tokens,step_tokens", [(64, 64), (8192, 64), (8192, 8192)])
def test_prompt_at_once_and_token_by_token_agree(whole_tokens, step_tokens):
    """80 rows a key head: the tensor-core kernel over a copy where the table is long.  The bound is that of
    test_gpu_layer.py (four quantizations, each a step off at most where the runs differ); keys and
    values are quantized from the same products in both runs."""
    m = make()
    tokens, seqs = 40, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn(seqs, tokens, 256, generator=g, device="cuda")
    index = torch.tensor([-1, 0, 1], dtype=torch.int32, device="cuda")
    whole = cache(seqs, whole_tokens)
    whole.extend([tokens] * seqs)
    out, _ = m(x.view(-1, 256), None, whole, index.repeat_interleave(tokens))
    out = out.view(seqs, tokens, 256)
    steps = cache(seqs, step_tokens)
    for t in range(tokens):
        steps.extend([1] * seqs)
        one, _ = m(x[:, t].contiguous(), None, steps, index)
        off = (one - out[:, t]).norm() / out[:, t].norm()
        assert off < 0.05, (t, off.item())
    assert binding.device_status() == 0


def test_a_quantized_cache_is_near_a_16_bit_one():
    """A value of the cache is off by half a quant of its block, 1 / 254 of the block's largest; with the four
    quantizations that both runs have, 10 % of the output's norm bounds what they differ by."""
    m = make(adapters=0)
    x = torch.randn(60, 256, device="cuda")
    outs = []
    for dtype in (torch.bfloat16, torch.int8):
        c = layer.PagedCache(1, 6, 16, 2, 128, 96, dtype)
        c.extend([60])
        outs.append(m(x, None, c)[0])
    assert (outs[0] - outs[1]).norm() < 0.1 * outs[0].norm()


@pytest.mark.parametrize("tokens", [1, 5, 70])
def test_the_layer_is_its_calls(tokens):
    m = make(adapters=0)
    x, r = torch.randn(tokens, 256, device="cuda"), torch.randn(tokens, 256, device="cuda")
    caches = [cache() for _ in range(2)]
    for c in caches:
        c.extend([tokens])
    out, residual = m(x, r, caches[0])
    n = binding.add_rms_norm(x, m.norms[0], residual=r)

    def product(p, q, d):
        return torch.cat([binding.gemm_small(m.packed[p], *m.shape[p], q[t:t + 64], d[t:t + 64]) for t in range(0, tokens, 64)])

    q, k, v = (product(p, n.q, n.d) for p in "qkv")
    c = caches[1]
    a = binding.paged_attention_q8(binding.rope_append_q8(q, k, v, m.cos_sin, *c.args()), *c.args(), max_new=tokens)
    n = binding.add_rms_norm(product("o", *binding.quantize(a.view(tokens, -1).float())), m.norms[1], residual=n.residual)
    gate, up = product("gate", n.q, n.d), product("up", n.q, n.d)
    h = torch.nn.functional.silu(gate) * up  # gated_act gives its q8_0 form
    want = product("down", *binding.quantize(h))
    assert torch.equal(residual, n.residual) and torch.equal(out, want)
    for got, ref in zip(caches[0].read(0), c.read(0)):
        assert got.shape == (tokens, 2, 128) and torch.equal(got, ref)
    kq, kd = binding.quantize(v.view(tokens, 2, 128).reshape(-1, 128))
    values = (kq.view(-1, 4, 32).float() * kd.view(torch.float16).float()[:, :, None]).view(tokens, 2, 128)
    assert torch.equal(c.read(0)[1], values)


def test_reading_either_cache():
    m = make(adapters=0)
    x = torch.randn(20, 256, device="cuda")
    for dtype in (torch.bfloat16, torch.int8):
        c = layer.PagedCache(3, 6, 16, 2, 128, 32, dtype)
        c.extend([3, 0, 17])
        m(x, None, c)
        k, v = c.read(2)
        assert k.shape == v.shape == (17, 2, 128) and torch.isfinite(k).all() and (k != 0).any()
        assert c.read(1)[0].shape == (0, 2, 128) and c.read(0, torch.float16)[0].dtype == torch.float16


@pytest.mark.parametrize("tokens", [1, 3, 70])
def test_head(tokens):
    head = layer.synthetic_head(1000, 256)
    x, r = torch.randn(tokens, 256, device="cuda"), torch.randn(tokens, 256, device="cuda")
    u = torch.rand(tokens, device="cuda")
    logits = head.logits(x, r)
    n = binding.add_rms_norm(x, head.norm, residual=r)
    assert torch.equal(logits[tokens - 1], binding.gemv(head.packed, 1000, 256, n.q[-1], n.d[-1]))
    for settings in (dict(), dict(temperature=0.0), dict(temperature=0.7, top_k=40, top_p=0.9)):
        assert head(x, r, u, **settings).tolist() == expected(logits, u, **settings)


def test_decoding_in_a_graph():
    """A step of the layer over a q8_0 cache and the next token, captured once and replayed as lengths grow."""
    m, head = make(adapters=0), layer.synthetic_head(512, 256)
    caches = [cache(2, 64, 8) for _ in range(2)]
    x, u = torch.empty(2, 256, device="cuda"), torch.empty(2, device="cuda")

    def step(c):
        out, residual = m(x, None, c)
        return head(out, residual, u, temperature=0.9, top_p=0.9)

    g = torch.cuda.CUDAGraph()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    drawn = None
    for t in range(6):
        x.normal_(generator=gen), u.uniform_(generator=gen)
        for c in caches:
            c.extend([1, 1])
        want = step(caches[0])
        if t == 0:
            step(caches[1])
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                drawn = step(caches[1])
        g.replay()
        assert drawn.tolist() == want.tolist()


def test_the_command(capsys, monkeypatch):
    for kind in ("bf16", "q8_0"):
        monkeypatch.setattr("sys.argv", ["layer", "--prompt", "9", "--sequences", "2", "--steps", "2", "--cache", kind, "--vocab", "2000"])
        layer.main()
        assert "next [" in capsys.readouterr().out
