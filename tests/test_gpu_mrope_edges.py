"""Multi-axis RoPE where a head holds values that are not finite: the dims past the rotated ones are a copy
(after the norm), each of itself alone."""
import numpy as np
import pytest

from test_gpu_kv4 import _cu, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 80, 128, 256, 512])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
def test_kept_dims_keep_values_that_are_not_finite_to_themselves(env, d, norm):
    g, t = env
    r = np.random.RandomState(d)
    R, n_q, n_kv, T = d // 2, 3, 2, 5
    x = r.randn(T, n_q + n_kv, d).astype(np.float32)
    x[0, 1, R] = np.inf                       # the first of the kept dims
    x[1, 3, d - 1] = -np.inf
    x[2, 0, R + 5] = np.nan
    x[3, 2, R + (d - R) // 2] = -0.0
    x[4, 4, R:] = np.where(np.arange(d - R) % 2, np.inf, 3.0)
    gamma = (1 + 0.1 * r.randn(d)).astype(np.float32)
    out = t.zeros((T, (n_q + n_kv) * d), device="cuda")
    dg = _cu(t, gamma) if norm else None
    g.qknorm_mrope(_cu(t, x.reshape(T, -1)), n_q, n_kv, d, dg, dg, 1e-6, _cu(t, np.arange(T, dtype=np.int32)[None]), [R // 2],
                   1e4, out)
    got = out.cpu().numpy().reshape(x.shape)[..., R:]
    if not norm:
        assert np.array_equal(got.view(np.uint32), x[..., R:].view(np.uint32)), "kept dims are not a copy"
        return
    # under the norm an infinity makes the others 0 and itself NaN; a NaN makes all of its head NaN
    with np.errstate(invalid="ignore"):
        x64 = x.astype(np.float64)
        want = (x64 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + 1e-6) * gamma)[..., R:]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    # the factor, two roundings and the reciprocal root: 5 * 2^-24 and 2 * 2^-23
    assert np.all(np.abs(got[ok] - want[ok]) <= 9 * 2.0 ** -24 * np.abs(want[ok]))
