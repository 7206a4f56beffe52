"""gem_logprobs' host-side refusals at the ends of its ranges, without a GPU."""
import pytest

from test_fp8_cpu import D, INVALID, OK, lib  # noqa: F401


@pytest.mark.parametrize("scale,want", [(2.0 ** -100, OK), (2.0 ** 100, OK), (2.0 ** -101, INVALID), (2.0 ** 100.5, INVALID), (1e-40, INVALID),
                                        (3e38, INVALID), (0.0, INVALID), (-1.0, INVALID), (float("nan"), INVALID), (float("inf"), INVALID)])
def test_scale(lib, scale, want):  # noqa: F811
    assert lib.gem_logprobs(D, 1000, 0, 1000, scale, D, D, D, D, 5, D, D, None, None) == want
