"""The 8-bit floating-point path's oracle at the ends of its ranges, without a GPU."""
import numpy as np
import pytest

from oracle import fp8


@pytest.mark.parametrize("act", [0, 1])
def test_gate_of_what_is_not_finite(act):
    """A product with an infinity or a NaN is never finite; a gate below its end is 0 for finite x alone."""
    x = np.array([[np.inf, -np.inf, np.nan, 1, 1, -np.inf, -200, 0, -200, 0]], np.float32)
    up = np.array([[1, 1, 1, np.inf, np.nan, 0, np.inf, -np.inf, 5, 5]], np.float32)
    y = fp8.gated(x, up, act)
    assert not np.isfinite(y[0, :8]).any() and np.array_equal(y[0, 8:], [0, 0])
