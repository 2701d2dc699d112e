"""The gated activation against its formula in 64 bits, and its q8_0 form by bits."""
import math

import pytest
import torch

from decode_q1_gemv_gb300 import binding
from tests.test_gpu_ops import F64, TINY, U, U32, normal, within

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    binding.load()


def reference(gate, up, act):
    """The value, and the exponent's argument."""
    x = gate.to(F64)
    if act == "silu":
        return x * torch.sigmoid(x) * up.to(F64), x
    arg = 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    return x * torch.sigmoid(arg) * up.to(F64), arg


# The argument is off by five roundings, which the exponential turns into as many
# of its size; the exponential by 2 of its last places; then four roundings (sum, quotient,
# product, and the type's own).  Below 2^-126 the quotient may be cut to zero: e^89 is infinite.
def tol(want, arg, up, dtype):
    return (5 * arg.abs() + 10) * U32 * want.abs() + U[dtype] * want.abs() + TINY[dtype] + 1e-36 * up.to(F64).abs() + 1e-38


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("nvec,n", [(1, 1), (3, 7), (2, 32), (5, 33), (1, 8192), (7, 4128), (64, 1000), (1, 100003), (300, 96)])
def test_values(nvec, n, act, dtype):
    gate, up = normal(1, nvec, n, std=3.0, dtype=dtype), normal(2, nvec, n, dtype=dtype)
    r = binding.gated_act(gate, up, act, out="y")
    assert r.q is None and r.d is None and r.y.dtype == dtype
    want, arg = reference(gate, up, act)
    within(r.y, want, tol(want, arg, up, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("nvec,n", [(1, 32), (2, 64), (1, 14336), (9, 1056), (33, 4096), (5, 96)])
@pytest.mark.parametrize("skew", [0, 1])
def test_q8_form(skew, nvec, n, act, dtype):
    """As quantize gives it of the same y in f32, whether or not rows are aligned."""
    wide_gate, wide_up = normal(3, nvec, n + 8, std=3.0, dtype=dtype), normal(4, nvec, n + 8, dtype=dtype)
    gate, up = wide_gate[:, skew:skew + n], wide_up[:, skew:skew + n]
    y = binding.gated_act(gate.float(), up.float(), act, out="y").y
    q, d = binding.quantize(y)
    for out in ("q8", "both"):
        r = binding.gated_act(gate, up, act, out=out)
        assert torch.equal(r.q, q) and torch.equal(r.d, d)
        if out == "both":
            assert torch.equal(r.y, y.to(dtype))


def test_in_place_halves_of_one_tensor_and_given_outputs():
    x = normal(5, 11, 2 * 192)
    gate, up = x.split(192, 1)
    want = binding.gated_act(gate, up, out="both")
    q, d = torch.zeros(11, 192, dtype=torch.int8, device="cuda"), torch.zeros(11, 6, dtype=torch.float16, device="cuda")
    r = binding.gated_act(gate, up, out="both", y=gate, q=q, d=d)
    assert torch.equal(gate, want.y) and torch.equal(q, want.q) and torch.equal(d.view(torch.int16), want.d)
    assert r.q.data_ptr() == q.data_ptr() and torch.equal(up, normal(5, 11, 2 * 192)[:, 192:])


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", TYPES)
def test_no_numbers_stay_in_their_block(value, dtype):
    gate, up = normal(6, 3, 96, dtype=dtype), normal(7, 3, 96, dtype=dtype)
    clean = binding.gated_act(gate, up, out="both")
    gate[1, 40], up[2, 95] = value, value
    got = binding.gated_act(gate, up, out="both")
    bad = torch.zeros(3, 96, dtype=torch.bool, device="cuda")
    bad[1, 40] = bad[2, 95] = True
    assert not torch.isfinite(got.y[bad]).any() and torch.equal(got.y[~bad], clean.y[~bad])
    blocks = bad.view(3, 3, 32).any(-1)
    assert torch.isnan(got.d.view(torch.float16)[blocks]).all() and torch.equal(got.d[~blocks], clean.d[~blocks])
    keep = ~blocks.repeat_interleave(32, 1)
    assert torch.equal(got.q[keep], clean.q[keep])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_extremes(act):
    """Far from zero: x for the one sign, zero for the other; zeros and least numbers."""
    x = torch.tensor([[0.0, -0.0, 1e-40, -1e-40, 80.0, -80.0, 100.0, -100.0, 1e4, -1e4, 1e20, -1e20, 3e38, -3e38]], device="cuda")
    up = torch.ones_like(x)
    got = binding.gated_act(x, up, act, out="y").y
    want, arg = reference(x, up, act)
    want = torch.where(x.to(F64) < -50, torch.zeros_like(want), want)
    within(got, want, tol(want, arg.abs().clamp(max=1e3), up, torch.float32) + 1e-30)


def test_on_another_stream_and_captured():
    gate, up = normal(8, 40, 640), normal(9, 40, 640)
    want = binding.gated_act(gate, up)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = binding.gated_act(gate, up, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(r.q, want.q) and torch.equal(r.d, want.d)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        r = binding.gated_act(gate, up, "gelu")
    gate.copy_(normal(10, 40, 640))
    g.replay()
    want = binding.gated_act(gate, up, "gelu")
    assert torch.equal(r.q, want.q) and torch.equal(r.d, want.d)
