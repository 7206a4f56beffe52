"""Paged 4-bit attention: what is left where a wait runs out, the stream of its scratch, and every form of the
kernel at the row counts that choose it."""
import numpy as np
import pytest

from parity import assert_close
from test_gpu_kv4 import _attn_case, _attn_run, _attn_want, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 1, 128), (8, 4, 64), (4, 2, 256), (8, 1, 256), (4, 2, 512), (8, 1, 512)],
                         ids=str)
def test_units_that_a_failed_wait_cuts_short_are_not_written(env, heads):
    """The first warp waits for 16 bytes that no copy brings (the wait runs out after the limit set here): the units
    that it and its neighbours had parts of stay as they were, all others are right."""
    g, t = env
    n_q, n_kv, d = heads
    kv_len, page = [900] * 24, 32
    r = np.random.RandomState(d + n_q)
    pool, table, cu, q = _attn_case(r, t, kv_len, [1] * 24, n_q, n_kv, d, page)
    args = (pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, d ** -0.5)
    want = _attn_want(*args)
    # an earlier call leaves parts of other values in the workspace
    ws = t.empty(g.kv4_attn_workspace(24, 24, n_q, n_kv, d), dtype=t.uint8, device="cuda")
    _attn_run(g, t, pool, table, cu, -q, *args[4:], workspace=ws)
    status = t.zeros(1, dtype=t.int32, device="cuda")
    t.cuda.synchronize()
    g.set_wait_limit(1_000_000)
    g.set_test_injection(g.INJECT_RING_SHORTFALL)
    try:
        got = _attn_run(g, t, *args, status=status, workspace=ws)
    finally:
        g.set_test_injection(0)
        g.set_wait_limit(0)
    assert g.status_from_flags(int(status)) == 6
    units, ref = (x.reshape(24 * n_kv, -1) for x in (got, want))
    left = np.all(units == 4.0, axis=1)
    assert left[0] and not left.all() and np.count_nonzero(left) <= 24 * n_kv // 2
    assert_close(units[~left], ref[~left], "the other units")
    status.zero_()
    assert_close(_attn_run(g, t, *args, status=status, workspace=ws), want, "the call after")
    assert int(status) == 0
