"""Limits of the operators around verification, refused on the host before anything is launched."""
import pytest
import torch

from speculative_decoding_verification_verify_gb300 import binding
from test_operators_cpu import append, attention, lib  # noqa: F401


@pytest.mark.parametrize("scale", [2.31e38, 2.4e38, 3e38, 3.4e38])
def test_scales_whose_exponent_overflows(lib, scale):  # noqa: F811
    assert attention(lib, scale=scale) == binding.EINVAL


def test_release_builds_keep_their_limit_of_waits(lib):  # noqa: F811
    assert lib.spec_verify_debug_wait_clocks(5) == binding.EINVAL


@pytest.mark.parametrize("B,N,stride", [(2, 8, 48 * 128), (1, 1, 32 * 128), (3, 1, 40 * 128)])
def test_rotated_queries_over_their_own(lib, B, N, stride):  # noqa: F811
    """From the byte range of q's rows on either side; the calls that pass the check go on to the device, which
    is not there."""
    q, width = 1 << 30, 32 * 128 * 2
    first, end = q - B * N * width, q + ((B * N - 1) * stride + 32 * 128) * 2
    for at in (first + 16, q, q + 16, end - 16):
        assert append(lib, q=q, q_out=at, B=B, N=N, qs=stride) == binding.EINVAL
    if not torch.cuda.is_available():
        for at in (first, end):
            assert append(lib, q=q, q_out=at, B=B, N=N, qs=stride) == binding.ECUDA
