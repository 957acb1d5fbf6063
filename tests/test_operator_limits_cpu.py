"""Limits of the operators around verification, refused on the host before anything is launched."""
import pytest

from speculative_decoding_verification_verify_gb300 import binding
from test_operators_cpu import attention, lib  # noqa: F401


@pytest.mark.parametrize("scale", [2.31e38, 2.4e38, 3e38, 3.4e38])
def test_scales_whose_exponent_overflows(lib, scale):  # noqa: F811
    assert attention(lib, scale=scale) == binding.EINVAL


def test_release_builds_keep_their_limit_of_waits(lib):  # noqa: F811
    assert lib.spec_verify_debug_wait_clocks(5) == binding.EINVAL
