"""The operators' tensors are on one device.  Fake tensors have a device and no
memory, so the refusal is seen without any GPU; nothing is launched."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from decode_q1_gemv_gb300 import binding


class Calls:
    """Each operator's tensors by name, on cuda:0 but for one."""

    def __init__(self, other=None):
        def make(name, *shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda:1" if name == other else "cuda:0")

        i32, bf = torch.int32, torch.bfloat16
        with FakeTensorMode():
            t = {n: make(n, 2, 64) for n in ("x", "residual", "residual_out", "y", "base", "out")}
            t.update(weight=make("weight", 64), q8=make("q8", 2, 64, dtype=torch.int8), d=make("d", 2, 2, dtype=torch.int16),
                     a=make("a", 3, 8, 64, dtype=bf), b=make("b", 3, 64, 8, dtype=bf), index=make("index", 2, dtype=i32),
                     scale=make("scale", 3), ranks=make("ranks", 3, dtype=i32), cs=make("cs", 9, 64),
                     k=make("k", 2, 64), v=make("v", 2, 64), cache_k=make("cache_k", 2, 16, 1, 64, dtype=bf),
                     cache_v=make("cache_v", 2, 16, 1, 64, dtype=bf), table=make("table", 1, 2, dtype=i32),
                     kv_len=make("kv_len", 1, dtype=i32), new_start=make("new_start", 2, dtype=i32),
                     heads=make("heads", 2, 1, 64, dtype=bf), turned=make("turned", 2, 1, 64, dtype=bf),
                     workspace=make("workspace", 1 << 20, dtype=torch.uint8))
        self.t = t
        self.cache = [t[n] for n in ("cache_k", "cache_v", "table", "kv_len", "new_start")]

    def norm(self):
        t = self.t
        binding.add_rms_norm(t["x"], t["weight"], residual=t["residual"], residual_out=t["residual_out"], out="both", y=t["y"],
                             q=t["q8"], d=t["d"])

    def lora(self):
        t = self.t
        binding.lora_add(t["x"], t["a"], t["b"], t["index"], t["scale"], t["ranks"], t["base"], t["out"])

    def rope(self):
        t = self.t
        binding.rope_append(t["x"], t["k"], t["v"], t["cs"], *self.cache, q_out=t["turned"])

    def attend(self):
        t = self.t
        binding.paged_attention(t["heads"], *self.cache, max_new=2, out=t["turned"], workspace=t["workspace"])

    def descriptor(self):
        binding.paged_kv(*self.cache, 2)


NAMES = dict(norm=["x", "weight", "residual", "residual_out", "y", "q8", "d"],
             lora=["x", "a", "b", "index", "scale", "ranks", "base", "out"],
             rope=["x", "k", "v", "cs", "cache_k", "cache_v", "table", "kv_len", "new_start", "turned"],
             attend=["heads", "cache_k", "cache_v", "table", "kv_len", "new_start", "turned", "workspace"],
             descriptor=["cache_k", "cache_v", "table", "kv_len", "new_start"])


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


def test_a_stream_of_another_device_is_refused():
    t = Calls().t
    with pytest.raises(ValueError, match="stream is of cuda:1, the tensors of cuda:0"):
        binding.add_rms_norm(t["x"], t["weight"], stream=OtherStream())
