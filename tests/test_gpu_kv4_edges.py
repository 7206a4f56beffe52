"""Paged 4-bit cache: what is left where a wait runs out, every form of the attention kernel at the row counts that
choose it, and offsets past 32 bits."""
import numpy as np
import pytest

from oracle import kv4
from parity import assert_close
from test_gpu_kv4 import ATTN, _attn_case, _attn_run, _attn_want, env  # noqa: F401

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


def _form(T, B, G, d):
    """The rule by which the library chooses a kernel: 0 up to 4 query rows a request on average, 1 up to 8
    (any more at d 256 and 512), 2 beyond.  T counts the rows of q, those behind the last request too."""
    rows = max(1, -(-T // B)) * G
    return 0 if rows <= 4 else 1 if rows <= 8 or d >= 256 else 2


# (kv lengths, new tokens, n_q, n_kv, d, page, window): single tokens at every number of query heads to a KV head,
# windows among them, and several tokens that leave rows of a unit empty
ROWS_OF_A_UNIT = [
    ([1, 700, 63], [1] * 3, G * 2, 2, d, 16, w) for G in (1, 2, 3, 4, 5, 6, 7, 8) for d in (64, 128) for w in (0, 100)
] + [
    ([400, 33], [1] * 2, G, 1, d, 32, w) for G in (1, 3, 4, 5, 8) for d in (256, 512) for w in (0, 45)
] + [
    ([150, 40, 500], [2, 1, 3], 6, 2, 64, 16, 0), ([150, 40, 500], [2, 1, 1], 2, 2, 128, 32, 60),
    ([90, 200], [3, 2], 3, 1, 128, 16, 0), ([90, 200], [7, 3], 5, 1, 128, 16, 33), ([77], [4], 7, 1, 64, 32, 0),
    ([77, 300], [5, 4], 3, 1, 256, 16, 20), ([200], [3], 5, 1, 512, 64, 0), ([45] * 34, [1] * 34, 3, 1, 128, 16, 0),
]
EXACT = [c for c in ATTN if sum(c[1])] + ROWS_OF_A_UNIT


def test_every_form_of_the_kernel_is_among_the_cases():
    seen = {(c[4], _form(sum(c[1]), len(c[1]), c[2] // c[3], c[4])) for c in EXACT}
    assert seen == {(d, f) for d in (64, 128, 256, 512) for f in range(3 if d < 256 else 2)}
    windows = {(c[4], _form(sum(c[1]), len(c[1]), c[2] // c[3], c[4])) for c in EXACT if c[6]}
    assert windows == seen


@pytest.mark.parametrize("spare", [0, 40], ids=["exact", "spare_rows"])
@pytest.mark.parametrize("case", EXACT, ids=lambda c: "kv%d_new%d_G%d_d%d_p%d_w%d_B%d" % (
    max(c[0]), max(c[1]), c[2] // c[3], c[4], c[5], c[6], len(c[0])))
def test_attention_with_rows_for_the_tokens_alone_and_with_room_to_spare(env, case, spare):
    """The rows of q choose the kernel, so both a call that has as many rows as tokens and one of a step that was
    captured with room for more are compared; rows behind the last request stay as they were."""
    g, t = env
    kv_len, fresh, n_q, n_kv, d, page, window = case
    r = np.random.RandomState(sum(kv_len) + d + n_q)
    pool, table, cu, q = _attn_case(r, t, kv_len, fresh, n_q, n_kv, d, page, spare_rows=spare)
    args = (pool, table, cu, q, kv_len, n_q, n_kv, d, page, window, d ** -0.5)
    got = _attn_run(g, t, *args)
    assert np.all(got[cu[-1]:] == 4.0), "rows behind the last request were written"
    assert_close(got[:cu[-1]], _attn_want(*args), "attention")
    assert g.device_status(reset=True) == 0


def test_offsets_past_32_bits(env):
    """A pool of more than 4 GiB and rows of more than 2^31 values: the last pages and rows are the ones in use."""
    g, t = env
    n_q, n_kv, d, page, n = 8, 2, 128, 64, 70
    size = g.kv4_page_bytes(n_kv, d, page)
    n_pages = (5 << 30) // size
    pool = t.empty((n_pages, size), dtype=t.uint8, device="cuda")
    cols = (n_q + 2 * n_kv) * d
    T = (1 << 31) // cols + 5000
    qkv = t.empty((T, cols), device="cuda")
    r = np.random.RandomState(90)
    x = r.randn(n, cols).astype(np.float32)
    qkv[T - n:] = t.from_numpy(x).cuda()
    i32 = dict(dtype=t.int32, device="cuda")
    pos, slot = t.full((1, T), -1, **i32), t.full((T,), -1, **i32)
    pages = [n_pages - 1, n_pages - 3]
    where = np.array([pages[j // page] * page + j % page for j in range(n)], np.int32)
    pos[0, T - n:] = t.arange(n, **i32)
    slot[T - n:] = t.from_numpy(where).cuda()
    g.qknorm_mrope(qkv, n_q, n_kv, d, None, None, 1e-6, pos, [d // 2], 1e4, qkv)
    rows = qkv[T - n:].cpu().numpy()
    want = kv4.qknorm_mrope(x, n_q, n_kv, d, None, None, 1e-6, np.arange(n)[None], [d // 2], 1e4)
    assert_close(rows[:, :want.shape[1]], want, "rope", max_abs=2e-6 * np.abs(want).max(), rel_l2=1e-6)
    k, v = qkv[:, n_q * d:(n_q + n_kv) * d], qkv[:, (n_q + n_kv) * d:]
    g.kv4_append(k, v, n_kv, d, slot, pool, page)
    K, V = (kv4.values(*kv4.quantise(rows[:, at:at + n_kv * d].reshape(n, n_kv, d))).reshape(n, -1)
            for at in (n_q * d, (n_q + n_kv) * d))
    out = t.zeros((2, T, n_kv * d), device="cuda")
    g.kv4_gather(pool, page, n_kv, d, slot, out[0], out[1])
    assert np.array_equal(out[:, T - n:].cpu().numpy(), np.stack([K, V]).astype(np.float32))
    del out
    att = t.zeros((T, n_q * d), device="cuda")
    g.kv4_attn(qkv, n_q, n_kv, d, t.tensor([T - n, T], **i32), t.tensor([n], **i32), t.tensor([pages], **i32), pool, page, 0,
               d ** -0.5, att)
    ref = kv4.attention(rows[:, :n_q * d].reshape(n, n_q, d), K.reshape(n, n_kv, d), V.reshape(n, n_kv, d), n, 0, d ** -0.5)
    assert_close(att[T - n:].cpu().numpy(), ref.reshape(n, -1), "attention")
    assert g.device_status(reset=True) == 0


def test_a_workspace_is_asked_for_wherever_there_is_work(env):
    g, _ = env
    for d in (64, 128, 256, 512):
        for G in range(1, 9):
            for T, B in ((1, 1), (4, 4), (64, 3), (4096, 4096)):
                assert g.kv4_attn_workspace(T, B, 2 * G, 2, d) > 0
