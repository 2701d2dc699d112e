"""Refusals of the operators' C ABI beside those of test_ops_cpu.py; nothing is launched."""
import pytest

from tests.test_ops_cpu import A, attend, cache, lib, lora, refused, rope  # noqa: F401  (lib is a fixture)


@pytest.mark.parametrize("scale", [3e38, -3e38, float("nan"), float("-inf")])
def test_attention_scale_in_log2_units_is_finite(lib, scale):  # noqa: F811
    """Scores are taken in units of log2(e): a scale that overflows there would make zero scores NaN."""
    refused(attend(lib, scale=scale), "scale")


@pytest.mark.parametrize("change", [dict(table=A + 2), dict(kv_len=A + 1), dict(new_start=A + 2)])
def test_misaligned_index_arrays_of_the_cache(lib, change):  # noqa: F811
    refused(rope(lib, cache(**change)), "4-byte aligned")
    refused(attend(lib, cache(**change)), "4-byte aligned")


@pytest.mark.parametrize("change", [dict(index=A + 2), dict(ranks=A + 1), dict(scale=A + 2)])
def test_misaligned_arrays_of_the_adapters(lib, change):  # noqa: F811
    refused(lora(lib, **change), "4-byte aligned")


def test_rows_of_a_key_head_are_counted_in_31_bits(lib):  # noqa: F811
    """2^24 new tokens of 128 heads over one key head: row numbers would wrap."""
    kv = cache(kv_heads=1, slot_stride=64, total_new=1 << 24)
    refused(attend(lib, kv, heads=128, qt=128 * 64, ot=128 * 64), "2^31 rows")
