"""What the operators between the products refuse, before any device is
touched: the C ABI's own checks with made-up addresses (nothing is launched),
and the binding's checks of tensors.  No GPU needed."""
import ctypes

import pytest
import torch

from decode_q1_gemv_gb300 import binding

A = 1 << 20  # an aligned address that is never followed
ARG = binding.Q1_ERR_ARG


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def refused(rc, text):
    assert rc == ARG
    assert text in binding.last_error(), binding.last_error()


def norm(lib, x=A, ldx=64, res=A, ldr=64, w=A, eps=1e-5, nvec=2, n=64, dtype=0, ro=A, ldo=64, y=A, ldy=64, q=A, d=A):
    return lib.q8_add_rms_norm(x, ldx, res, ldr, w, eps, nvec, n, dtype, ro, ldo, y, ldy, q, d, None)


@pytest.mark.parametrize("change,text", [
    (dict(nvec=0), "bad shape"), (dict(n=0), "bad shape"), (dict(n=1 << 25, ldx=1 << 25), "bad shape"),
    (dict(nvec=(1 << 24) + 1), "bad shape"), (dict(dtype=3), "bad type"), (dict(dtype=-1), "bad type"),
    (dict(x=None), "null"), (dict(w=None), "null"), (dict(q=None), "null"), (dict(d=None), "null"),
    (dict(q=None, d=None, y=None, ro=None), "null"), (dict(n=48), "multiple of 32"), (dict(eps=-1e-6), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(ldx=63), "row stride"), (dict(ldr=63), "row stride"),
    (dict(ldo=63), "row stride"), (dict(ldy=63), "row stride"), (dict(q=A + 4), "misaligned"),
    (dict(d=A + 2), "misaligned"), (dict(x=A + 2), "misaligned"), (dict(w=A + 2), "misaligned"),
    (dict(dtype=1, res=A + 1), "misaligned")])
def test_norm_refusals(lib, change, text):
    refused(norm(lib, **change), text)


def lora(lib, x=A, ldx=64, nvec=2, n=64, rows=32, a=A, b=A, dtype=1, adapters=2, rank=16, index=A, ranks=A, scale=A,
         base=A, ldb=32, out=A, ldo=32):
    return lib.q1_lora_add(x, ldx, nvec, n, rows, a, b, dtype, adapters, rank, index, ranks, scale, base, ldb, out, ldo,
                           None)


@pytest.mark.parametrize("change,text", [
    (dict(nvec=0), "bad shape"), (dict(nvec=65536), "bad shape"), (dict(n=60), "bad shape"), (dict(n=0), "bad shape"),
    (dict(rows=0), "bad shape"), (dict(adapters=0), "bad shape"), (dict(rank=0), "bad shape"),
    (dict(rank=12), "bad shape"), (dict(rank=136), "bad shape"), (dict(dtype=0), "bad weight type"),
    (dict(x=None), "null"), (dict(a=None), "null"), (dict(b=None), "null"), (dict(index=None), "null"),
    (dict(base=None), "null"), (dict(out=None), "null"), (dict(x=A + 4), "aligned"), (dict(a=A + 8), "aligned"),
    (dict(b=A + 2), "aligned"), (dict(ldx=66), "aligned"), (dict(out=A + 2), "aligned"), (dict(ldx=60), "row stride"),
    (dict(ldb=31), "row stride"), (dict(ldo=31), "row stride"), (dict(ldb=36), "same stride")])
def test_lora_refusals(lib, change, text):
    refused(lora(lib, **change), text)


def cache(**change):
    v = dict(k=A, v=A, page_stride=8 * 16 * 64, slot_stride=8 * 64, head_stride=64, table=A, table_width=4,
             table_stride=4, kv_len=A, new_start=A, pages=10, page_size=16, kv_heads=8, dim=64, batch=2, total_new=5,
             dtype=1)
    v.update(change)
    return binding.PagedKV(**v)


CACHE = [(dict(dtype=0), "bad cache type"), (dict(pages=0), "bad shape"), (dict(kv_heads=0), "bad shape"),
         (dict(batch=0), "bad shape"), (dict(total_new=0), "bad shape"), (dict(table_width=0), "bad shape"),
         (dict(page_size=24), "page_size"), (dict(page_size=4), "page_size"), (dict(page_size=8192), "page_size"),
         (dict(dim=96), "dim"), (dict(k=None), "null"), (dict(v=None), "null"), (dict(table=None), "null"),
         (dict(kv_len=None), "null"), (dict(new_start=None), "null"), (dict(k=A + 8), "aligned"),
         (dict(slot_stride=516), "strides"), (dict(head_stride=56), "strides"), (dict(page_stride=-64), "strides"),
         (dict(table_stride=3), "table_stride")]


def rope(lib, kv=None, q=A, ldq=512, k=A, ldk=512, v=A, ldv=512, cs=A, positions=100, rot=64, inter=0, heads=8, out=A):
    kv = cache() if kv is None else kv
    return lib.q1_rope_append(q, ldq, k, ldk, v, ldv, cs, positions, rot, inter, heads, out, ctypes.byref(kv), None)


@pytest.mark.parametrize("change,text", [
    (dict(q=None), "null"), (dict(k=None), "null"), (dict(v=None), "null"), (dict(cs=None), "null"),
    (dict(out=None), "null"), (dict(rot=4), "rot"), (dict(rot=72), "rot"), (dict(rot=20), "rot"),
    (dict(positions=0), "rot"), (dict(heads=0), "heads"), (dict(ldq=511), "aligned"), (dict(q=A + 4), "aligned"),
    (dict(ldk=508), "row stride"), (dict(heads=9), "row stride")])
def test_rope_refusals(lib, change, text):
    refused(rope(lib, **change), text)


def attend(lib, kv=None, q=A, qt=512, qh=64, heads=8, scale=0.125, max_new=1, out=A, ot=512, oh=64, ws=A, wb=1 << 40):
    kv = cache() if kv is None else kv
    return lib.q1_paged_attention(q, qt, qh, heads, scale, ctypes.byref(kv), max_new, out, ot, oh, ws, wb, None)


@pytest.mark.parametrize("change,text", [
    (dict(q=None), "null"), (dict(out=None), "null"), (dict(ws=None), "null"), (dict(heads=12), "heads"),
    (dict(heads=0), "heads"), (dict(qt=508), "strides"), (dict(oh=60), "strides"), (dict(qh=56), "stride is less"),
    (dict(scale=float("inf")), "scale"), (dict(max_new=0), "max_new"), (dict(wb=64), "workspace"),
    (dict(q=A + 2), "aligned"), (dict(ws=A + 8), "aligned")])
def test_attend_refusals(lib, change, text):
    refused(attend(lib, **change), text)


@pytest.mark.parametrize("change,text", CACHE)
def test_cache_refusals(lib, change, text):
    refused(rope(lib, cache(**change)), text)
    refused(attend(lib, cache(**change)), text)
    refused(lib.q1_paged_attention(A, 512, 64, 8, 0.1, None, 1, A, 512, 64, A, 1 << 40, None), "null descriptor")


@pytest.mark.parametrize("args", [(0, 8, 8, 64), (1, 8, 3, 64), (1, 8, 8, 80), (1, 0, 1, 64)])
def test_workspace_refusals(lib, args):
    with pytest.raises(binding.Q1Error, match="bad shape"):
        binding.paged_attention_workspace(*args)


def test_workspace_grows_with_nothing_but_shape(lib):
    assert binding.paged_attention_workspace(1, 8, 8, 128) > binding.paged_attention_workspace(1, 8, 8, 64) > 0


# ---------------------------------------------------------------- binding --
def test_binding_wants_cuda_tensors():
    x, w = torch.zeros(2, 64), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.add_rms_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        binding.lora_add(x, torch.zeros(1, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 8, dtype=torch.bfloat16),
                         torch.zeros(2, dtype=torch.int32), base=torch.zeros(2, 4))
    k = torch.zeros(2, 16, 1, 64, dtype=torch.float16)
    t, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    s = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.paged_attention(torch.zeros(1, 2, 64, dtype=torch.float16), k, k, t, n, s, max_new=1)
    with pytest.raises(ValueError, match="CUDA"):
        binding.rope_append(torch.zeros(1, 128), torch.zeros(1, 64), torch.zeros(1, 64), torch.zeros(9, 64), k, k, t, n, s)


def test_binding_names_what_is_wrong():
    x, w = torch.zeros(2, 48), torch.ones(48)
    with pytest.raises(ValueError, match="multiple of 32"):
        binding.add_rms_norm(x, w)
    with pytest.raises(ValueError, match="out must be"):
        binding.add_rms_norm(x, w, out="int8")
    with pytest.raises(TypeError, match="dtype"):
        binding.add_rms_norm(x.double(), w, out="y")
    with pytest.raises(ValueError, match=r"\[nvec, n\]"):
        binding.add_rms_norm(x[0], w, out="y")
    with pytest.raises(ValueError, match="base, out or both"):
        binding.lora_add(x, torch.zeros(1, 8, 48), torch.zeros(1, 4, 8), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="heads, dim"):
        binding.paged_attention(x, x, x, x, x, x, max_new=1)
    with pytest.raises(ValueError, match="pages, page_size"):
        binding.paged_kv(x, x, x, x, x, 1)
