"""Scales that the kernels cannot use are refused (fake addresses; nothing is launched)."""
import pytest

from test_attn_checks import SHAPE, decode, lib, prefill  # noqa: F401


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38])
def test_scales_past_the_range_of_exp2(lib, scale):  # noqa: F811
    """Times log2 e they are infinite: every score, and a score of zero first, would be NaN."""
    assert prefill(lib, scale=scale) == SHAPE
    assert decode(lib, scale=scale) == SHAPE
