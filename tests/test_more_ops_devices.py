"""The q8_0 cache's, the gated activation's and sampling's tensors are on one device: fake tensors
have a device and no memory, so the refusal is seen without any GPU; nothing is launched."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from decode_q1_gemv_gb300 import binding


class Calls:
    """Each operator's tensors by name, on cuda:0 but for one."""

    def __init__(self, other=None):
        def make(name, *shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda:1" if name == other else "cuda:0")

        i8, i32, half = torch.int8, torch.int32, torch.float16
        with FakeTensorMode():
            t = {n: make(n, 2, 64) for n in ("gate", "up", "y", "x", "k", "v", "logits")}
            t.update(q8=make("q8", 2, 64, dtype=i8), d=make("d", 2, 2, dtype=torch.int16), cs=make("cs", 9, 64),
                     cache_k=make("cache_k", 2, 16, 1, 64, dtype=i8), cache_v=make("cache_v", 2, 16, 1, 64, dtype=i8),
                     scale_k=make("scale_k", 2, 16, 1, 2, dtype=half), scale_v=make("scale_v", 2, 16, 1, 2, dtype=half),
                     table=make("table", 1, 2, dtype=i32), kv_len=make("kv_len", 1, dtype=i32), new_start=make("new_start", 2, dtype=i32),
                     heads=make("heads", 2, 1, 64, dtype=half), turned=make("turned", 2, 1, 64, dtype=half),
                     workspace=make("workspace", 1 << 20, dtype=torch.uint8), k_out=make("k_out", 2, 1, 64), v_out=make("v_out", 2, 1, 64),
                     out=make("out", 2, dtype=i32), top_k=make("top_k", 2, dtype=i32),
                     **{n: make(n, 2) for n in ("uniform", "temperature", "top_p", "min_p")})
        self.t = t
        self.cache = [t[n] for n in CACHE]

    def gated(self):
        t = self.t
        binding.gated_act(t["gate"], t["up"], out="both", y=t["y"], q=t["q8"], d=t["d"])

    def append(self):
        t = self.t
        binding.rope_append_q8(t["x"], t["k"], t["v"], t["cs"], *self.cache, q_out=t["turned"])

    def read(self):
        binding.cache_read_q8(*self.cache, 2, k_out=self.t["k_out"], v_out=self.t["v_out"])

    def attend(self):
        t = self.t
        binding.paged_attention_q8(t["heads"], *self.cache, max_new=2, out=t["turned"], workspace=t["workspace"])

    def descriptor(self):
        binding.paged_q8(*self.cache, 2)

    def sample(self):
        t = self.t
        binding.sample(t["logits"], t["uniform"], t["temperature"], t["top_k"], t["top_p"], t["min_p"], out=t["out"])


CACHE = ["cache_k", "cache_v", "scale_k", "scale_v", "table", "kv_len", "new_start"]
NAMES = dict(gated=["gate", "up", "y", "q8", "d"], append=["x", "k", "v", "cs", *CACHE, "turned"], read=[*CACHE, "k_out", "v_out"],
             attend=["heads", *CACHE, "turned", "workspace"], descriptor=CACHE,
             sample=["logits", "uniform", "temperature", "top_k", "top_p", "min_p", "out"])


@pytest.fixture(autouse=True)
def _no_device(monkeypatch):
    """The current stream of a fake tensor's device: none here."""
    binding.load()
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)


@pytest.mark.parametrize("call,other", [(c, n) for c in NAMES for n in NAMES[c]])
def test_a_tensor_of_another_device_is_refused(call, other):
    with pytest.raises(ValueError, match="different devices: cuda:[01] and cuda:[01]"):
        getattr(Calls(other), call)()


class OtherStream:
    device = torch.device("cuda:1")
    cuda_stream = 0


@pytest.mark.parametrize("call", ["gated_act", "sample"])
def test_a_stream_of_another_device_is_refused(call):
    t = Calls().t
    with pytest.raises(ValueError, match="stream is of cuda:1, the tensors of cuda:0"):
        getattr(binding, call)(t["gate"], t["up"] if call == "gated_act" else t["uniform"], stream=OtherStream())
