"""Refusals of the paged cache's calls at sizes that their own arithmetic would divide by.  No GPU needed."""
import pytest
import torch

from decode_q1_gemv_gb300 import binding


@pytest.mark.parametrize("heads", [0, 2])
def test_a_cache_of_no_dims(heads):
    """An empty last axis is refused before anything is divided by it (or looked at as a device's)."""
    k, d = torch.zeros(2, 16, 1, 0, dtype=torch.int8), torch.zeros(2, 16, 1, 0, dtype=torch.float16)
    k16 = torch.zeros(2, 16, 1, 0, dtype=torch.bfloat16)
    t, n, s = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q, x, cs = torch.zeros(1, heads * 64), torch.zeros(1, 0), torch.zeros(9, 64)
    with pytest.raises(ValueError, match="dim is 0"):
        binding.rope_append_q8(q, x, x, cs, k, k, d, d, t, n, s)
    with pytest.raises(ValueError, match="dim is 0"):
        binding.rope_append(q, x, x, cs, k16, k16, t, n, s)
    with pytest.raises(ValueError, match="dim is 0"):
        binding.cache_read_q8(k, k, d, d, t, n, s, 1)
    with pytest.raises(ValueError, match="dim is 0"):
        binding.paged_attention_q8(torch.zeros(1, 2, 0, dtype=torch.float16), k, k, d, d, t, n, s, max_new=1)
    with pytest.raises(ValueError, match="dim is 0"):
        binding.paged_attention(torch.zeros(1, 2, 0, dtype=torch.bfloat16), k16, k16, t, n, s, max_new=1)
    with pytest.raises(ValueError, match="dim is 0"):
        binding.paged_q8(k, k, d, d, t, n, s, 1)
    with pytest.raises(ValueError, match="dim is 0"):
        binding.paged_kv(k16, k16, t, n, s, 1)
