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


def test_released_pages_are_handed_out_again():
    c = cache()
    c.extend([40, 16])
    assert not c.free
    with pytest.raises(ValueError, match="no free pages"):
        c.extend([0, 1])
    c.release(0)
    assert len(c.free) == 3 and c.lengths == [0, 16] and c.kv_len.tolist() == [0, 16]
    assert c.new_start.tolist() == [0, 0, 0] and c.max_new == 0
    c.extend([17, 15])
    used = c.table[0, :2].tolist() + c.table[1, :2].tolist()
    assert sorted(used) == [0, 1, 2, 3] and c.kv_len.tolist() == [17, 31] and c.new_start.tolist() == [0, 17, 32]
    c.release(0)
    c.release(0)
    assert len(c.free) == 2
