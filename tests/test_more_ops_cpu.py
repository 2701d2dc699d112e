"""What the q8_0 cache's calls, the gated activation and sampling refuse, before any device is touched,
and the quantized cache's book-keeping.  No GPU needed."""
import ctypes
import math

import pytest
import torch

from decode_q1_gemv_gb300 import binding, layer

A = 1 << 20  # an aligned address that is never followed
ARG = binding.Q1_ERR_ARG


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def refused(rc, text):
    assert rc == ARG
    assert text in binding.last_error(), binding.last_error()


def cache(**change):
    v = dict(k=A, v=A, k_scale=A, v_scale=A, page_stride=8 * 16 * 64, slot_stride=64, head_stride=16 * 64, scale_page_stride=256,
             scale_slot_stride=2, scale_head_stride=32, table=A, table_width=4, table_stride=4, kv_len=A, new_start=A, pages=10,
             page_size=16, kv_heads=8, dim=64, batch=2, total_new=5)
    v.update(change)
    return binding.PagedQ8(**v)


CACHE = [(dict(pages=0), "bad shape"), (dict(kv_heads=0), "bad shape"), (dict(batch=0), "bad shape"), (dict(total_new=0), "bad shape"),
         (dict(table_width=0), "bad shape"), (dict(page_size=24), "page_size"), (dict(page_size=4), "page_size"),
         (dict(page_size=8192), "page_size"), (dict(dim=96), "dim"), (dict(dim=32), "dim"), (dict(k=None), "null"), (dict(v=None), "null"),
         (dict(k_scale=None), "null"), (dict(v_scale=None), "null"), (dict(table=None), "null"), (dict(kv_len=None), "null"),
         (dict(new_start=None), "null"), (dict(k=A + 8), "aligned"), (dict(v=A + 8), "aligned"), (dict(k_scale=A + 4), "aligned"),
         (dict(v_scale=A + 8), "aligned"), (dict(table=A + 2), "aligned"), (dict(slot_stride=72), "multiples of 16"),
         (dict(head_stride=1032), "multiples of 16"), (dict(page_stride=-64), "strides"), (dict(slot_stride=32), "strides"),
         (dict(scale_slot_stride=1), "scales' strides"), (dict(scale_head_stride=33), "scales' strides"),
         (dict(scale_page_stride=0), "scales' strides"), (dict(scale_page_stride=-2), "scales' strides"),
         (dict(dim=128, slot_stride=128, head_stride=2048, page_stride=16384, scale_slot_stride=2), "scales' strides"),
         (dict(table_stride=3), "table_stride")]


def rope(lib, kv=None, q=A, ldq=512, k=A, ldk=512, v=A, ldv=512, cs=A, positions=100, rot=64, inter=0, heads=8, out=A, dtype=1):
    kv = cache() if kv is None else kv
    return lib.q1_rope_append_q8(q, ldq, k, ldk, v, ldv, cs, positions, rot, inter, heads, out, dtype, ctypes.byref(kv), None)


@pytest.mark.parametrize("change,text", [
    (dict(q=None), "null"), (dict(k=None), "null"), (dict(v=None), "null"), (dict(cs=None), "null"), (dict(out=None), "null"),
    (dict(rot=4), "rot"), (dict(rot=72), "rot"), (dict(rot=20), "rot"), (dict(positions=0), "rot"), (dict(heads=0), "heads"),
    (dict(heads=4097), "heads"), (dict(ldq=511), "aligned"), (dict(q=A + 4), "aligned"), (dict(out=A + 8), "aligned"),
    (dict(ldk=508), "row stride"), (dict(heads=9), "row stride"), (dict(dtype=0), "bad type"), (dict(dtype=3), "bad type")])
def test_append_refusals(lib, change, text):
    refused(rope(lib, **change), text)


def read(lib, kv=None, dtype=0, k=A, v=A):
    kv = cache() if kv is None else kv
    return lib.q1_cache_read_q8(ctypes.byref(kv), dtype, k, v, None)


@pytest.mark.parametrize("change,text", [(dict(dtype=3), "bad type"), (dict(dtype=-1), "bad type"), (dict(k=None, v=None), "null"),
                                         (dict(k=A + 8), "aligned"), (dict(v=A + 4), "aligned")])
def test_read_refusals(lib, change, text):
    refused(read(lib, **change), text)


def attend(lib, kv=None, q=A, qt=512, qh=64, heads=8, scale=0.125, dtype=1, max_new=1, out=A, ot=512, oh=64, ws=A, wb=1 << 40):
    kv = cache() if kv is None else kv
    return lib.q1_paged_attention_q8(q, qt, qh, heads, scale, dtype, ctypes.byref(kv), max_new, out, ot, oh, ws, wb, None)


@pytest.mark.parametrize("change,text", [
    (dict(q=None), "null"), (dict(out=None), "null"), (dict(ws=None), "null"), (dict(heads=12), "heads"), (dict(heads=0), "heads"),
    (dict(qt=508), "strides"), (dict(oh=60), "strides"), (dict(qh=56), "stride is less"), (dict(scale=math.inf), "scale"),
    (dict(scale=math.nan), "scale"), (dict(scale=3e38), "scale"), (dict(max_new=0), "max_new"), (dict(wb=64), "workspace"),
    (dict(q=A + 2), "aligned"), (dict(ws=A + 8), "aligned"), (dict(dtype=0), "bad type")])
def test_attend_refusals(lib, change, text):
    refused(attend(lib, **change), text)


def test_attend_refuses_a_workspace_without_a_copy(lib):
    """Many rows need one sequence's copy beside what few rows need."""
    few = binding.paged_attention_q8_workspace(1, 8, 8, 64, 64)
    refused(attend(lib, max_new=2000, wb=few), "workspace")


@pytest.mark.parametrize("change,text", CACHE)
def test_cache_refusals(lib, change, text):
    for call in (rope, read, attend):
        refused(call(lib, cache(**change)), text)


def test_null_descriptors(lib):
    refused(lib.q1_rope_append_q8(A, 512, A, 512, A, 512, A, 9, 64, 0, 8, A, 1, None, None), "null descriptor")
    refused(lib.q1_cache_read_q8(None, 0, A, A, None), "null descriptor")
    refused(lib.q1_paged_attention_q8(A, 512, 64, 8, 0.1, 1, None, 1, A, 512, 64, A, 1 << 40, None), "null descriptor")


@pytest.mark.parametrize("args", [(0, 8, 8, 64, 100, 1), (1, 8, 3, 64, 100, 1), (1, 8, 8, 80, 100, 1), (1, 0, 1, 64, 100, 1),
                                  (1, 8, 8, 64, 0, 1), (1, 8, 8, 64, 100, 0), (1 << 20, 8, 8, 64, 1 << 43, 1)])
def test_workspace_refusals(lib, args):
    with pytest.raises(binding.Q1Error, match="bad shape"):
        binding.paged_attention_q8_workspace(*args)
    with pytest.raises(TypeError, match="int32"):
        binding.paged_attention_q8_workspace(1, 8, 8, 64, 100, dtype=torch.int32)
    with pytest.raises(binding.Q1Error, match="bad type"):
        binding.paged_attention_q8_workspace(1, 8, 8, 64, 100, dtype=torch.float32)


def test_workspace_sizes(lib):
    size = binding.paged_attention_q8_workspace
    assert size(1, 8, 8, 128, 1000) > size(1, 8, 8, 64, 1000) > 0
    assert size(1, 8, 8, 64, 1000, 9) == size(1, 8, 8, 64, 5, 1)  # few rows: no copies
    one, two = size(500, 8, 2, 64, 1000), size(500, 8, 2, 64, 1000, 2)
    assert two - one >= 2 * 1024 * 2 * 64 * 2 and size(500, 8, 2, 64, 1000, 1, torch.float16) > one  # keys and values of 8 pages of 128


def gate(lib, gate=A, ldg=64, up=A, ldu=64, nvec=2, n=64, dtype=0, act=0, y=A, ldy=64, q=A, d=A):
    return lib.q8_gated_act(gate, ldg, up, ldu, nvec, n, dtype, act, y, ldy, q, d, None)


@pytest.mark.parametrize("change,text", [
    (dict(nvec=0), "bad shape"), (dict(n=0), "bad shape"), (dict(n=1 << 25, ldg=1 << 25), "bad shape"), (dict(nvec=(1 << 24) + 1), "bad shape"),
    (dict(dtype=3), "bad type"), (dict(act=2), "bad activation"), (dict(act=-1), "bad activation"), (dict(gate=None), "null"),
    (dict(up=None), "null"), (dict(q=None), "null"), (dict(d=None), "null"), (dict(q=None, d=None, y=None), "null"),
    (dict(n=48), "multiple of 32"), (dict(ldg=63), "row stride"), (dict(ldu=63), "row stride"), (dict(ldy=63), "row stride"),
    (dict(q=A + 4), "misaligned"), (dict(d=A + 2), "misaligned"), (dict(gate=A + 2), "misaligned"), (dict(dtype=1, up=A + 1), "misaligned")])
def test_gate_refusals(lib, change, text):
    refused(gate(lib, **change), text)


def sample(lib, logits=A, ld=100, rows=2, vocab=100, dtype=0, uniform=A, out=A, **settings):
    s = dict(temperature=None, top_k=None, top_p=None, min_p=None, temperature_all=1.0, top_k_all=0, top_p_all=1.0, min_p_all=0.0)
    s.update(settings)
    return lib.q1_sample(logits, ld, rows, vocab, dtype, uniform, ctypes.byref(binding.Sampling(**s)), out, None)


@pytest.mark.parametrize("change,text", [
    (dict(rows=0), "bad shape"), (dict(rows=65536), "bad shape"), (dict(vocab=0), "bad shape"), (dict(vocab=(1 << 19) + 1, ld=1 << 20), "bad shape"),
    (dict(dtype=3), "bad type"), (dict(logits=None), "null"), (dict(uniform=None), "null"), (dict(out=None), "null"), (dict(ld=99), "row stride"),
    (dict(ld=-100), "row stride"), (dict(logits=A + 2), "misaligned"), (dict(dtype=1, logits=A + 1), "misaligned"), (dict(uniform=A + 2), "misaligned"),
    (dict(out=A + 2), "misaligned"), (dict(temperature=A + 1), "misaligned"), (dict(top_k=A + 2), "misaligned"), (dict(top_p=A + 2), "misaligned"),
    (dict(min_p=A + 2), "misaligned"), (dict(temperature_all=math.nan), "NaN"), (dict(top_p_all=math.nan), "NaN"), (dict(min_p_all=math.nan), "NaN")])
def test_sample_refusals(lib, change, text):
    refused(sample(lib, **change), text)


def test_sample_wants_its_settings(lib):
    refused(lib.q1_sample(A, 100, 2, 100, 0, A, None, A, None), "null")


# ---------------------------------------------------------------- binding --
def test_binding_wants_cuda_tensors():
    x, u = torch.zeros(2, 64), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        binding.gated_act(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        binding.sample(x, u)
    k, d = torch.zeros(2, 16, 1, 64, dtype=torch.int8), torch.zeros(2, 16, 1, 2, dtype=torch.float16)
    t, n, s = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.paged_attention_q8(torch.zeros(1, 2, 64, dtype=torch.float16), k, k, d, d, t, n, s, max_new=1)
    with pytest.raises(ValueError, match="CUDA"):
        binding.rope_append_q8(torch.zeros(1, 128), torch.zeros(1, 64), torch.zeros(1, 64), torch.zeros(9, 64), k, k, d, d, t, n, s)
    with pytest.raises(ValueError, match="CUDA"):
        binding.cache_read_q8(k, k, d, d, t, n, s, 1)


def test_binding_names_what_is_wrong():
    x = torch.zeros(2, 48)
    with pytest.raises(ValueError, match="multiple of 32"):
        binding.gated_act(x, x)
    with pytest.raises(ValueError, match="out must be"):
        binding.gated_act(x, x, out="int8")
    with pytest.raises(ValueError, match="activation must be"):
        binding.gated_act(x, x, "relu")
    with pytest.raises(TypeError, match="dtype"):
        binding.gated_act(x.double(), x.double(), out="y")
    with pytest.raises(ValueError, match=r"\[nvec, n\]"):
        binding.gated_act(x[0], x[0], out="y")
    with pytest.raises(ValueError, match=r"\[rows, vocab\]"):
        binding.sample(x[0], x[0])
    with pytest.raises(ValueError, match="heads, dim"):
        binding.paged_attention_q8(x, x, x, x, x, x, x, x, max_new=1)
    with pytest.raises(ValueError, match="pages, page_size"):
        binding.paged_q8(x, x, x, x, x, x, x, 1)
    with pytest.raises(TypeError, match="int8"):
        binding.cache_read_q8(x, x, x, x, x, x, x, 1, dtype=torch.int8)


def test_quantized_cache_on_the_cpu():
    c = layer.PagedCache(2, 4, 16, 3, 64, 64, torch.int8, device="cpu")
    c.extend([20, 3])
    k, v, ks, vs, table, kv_len, new_start = c.args()
    assert k.shape == v.shape == (4, 16, 3, 64) and ks.shape == vs.shape == (4, 16, 3, 2)
    assert k.dtype == torch.int8 and ks.dtype == torch.float16 and k.stride() == (3072, 64, 1024, 1) and ks.stride() == (96, 2, 32, 1)
    assert kv_len.tolist() == [20, 3] and new_start.tolist() == [0, 20, 23] and c.max_new == 20
    with pytest.raises(ValueError, match="multiple of 32"):
        layer.PagedCache(1, 1, 16, 1, 48, 16, torch.int8, device="cpu")
    c = layer.PagedCache(2, 4, 16, 3, 64, 64, device="cpu")
    assert not c.quantized and len(c.args()) == 5 and c.read(0)[0].shape == (0, 3, 64)
