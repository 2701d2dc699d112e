"""Refusals of the operators' C ABI beside those of test_ops_cpu.py; nothing is launched."""
import pytest

from tests.test_ops_cpu import attend, lib, refused  # noqa: F401  (lib is a fixture)


@pytest.mark.parametrize("scale", [3e38, -3e38, float("nan"), float("-inf")])
def test_attention_scale_in_log2_units_is_finite(lib, scale):  # noqa: F811
    """Scores are taken in units of log2(e): a scale that overflows there would make zero scores NaN."""
    refused(attend(lib, scale=scale), "scale")
