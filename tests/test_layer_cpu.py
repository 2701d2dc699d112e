"""The paged cache's book-keeping, on the CPU."""
import pytest

from decode_q1_gemv_gb300 import layer


def cache(sequences=2, pages=4):
    return layer.PagedCache(sequences, pages, 16, 1, 64, 64, device="cpu")


def test_counts_below_zero_are_refused():
    c = cache()
    c.extend([20, 3])
    for new in ([-1, 2], [1, -3]):
        with pytest.raises(ValueError, match="below zero"):
            c.extend(new)
    assert c.lengths == [20, 3] and c.kv_len.tolist() == [20, 3] and c.new_start.tolist() == [0, 20, 23] and len(c.free) == 1
