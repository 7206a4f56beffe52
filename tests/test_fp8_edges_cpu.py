"""The 8-bit floating-point path's oracle at the ends of its ranges, without a GPU."""
import numpy as np
import pytest

from oracle import fp8
from test_fp8_cpu import D, INVALID, OK, lib  # noqa: F401


@pytest.mark.parametrize("act", [0, 1])
def test_gate_of_what_is_not_finite(act):
    """A product with an infinity or a NaN is never finite; a gate below its end is 0 for finite x alone."""
    x = np.array([[np.inf, -np.inf, np.nan, 1, 1, -np.inf, -200, 0, -200, 0]], np.float32)
    up = np.array([[1, 1, 1, np.inf, np.nan, 0, np.inf, -np.inf, 5, 5]], np.float32)
    y = fp8.gated(x, up, act)
    assert not np.isfinite(y[0, :8]).any() and np.array_equal(y[0, 8:], [0, 0])


def test_scales_end_with_the_largest_number():
    y = np.zeros((2, 256))
    y[0, 3], y[1, 3] = np.finfo(np.float32).max, -2.0 ** 128
    codes, scales = fp8.quantise(y)
    assert scales[0, 0] == 2.0 ** 120 and np.isnan(scales[1, 0]) and not codes[1].any() and not scales[:, 1].any()


@pytest.mark.parametrize("eps,want", [(0.0, OK), (1e-45, OK), (2.0 ** 127, OK), (2.0 ** 127.1, INVALID), (3.4e38, INVALID), (-1e-45, INVALID)])
def test_eps(lib, eps, want):  # noqa: F811
    assert lib.gem_rmsnorm_fp8(D, 256, None, 0, None, 0, 0, 256, None, eps, D, 256, D, 2, None) == want
