"""The paged 4-bit KV cache on the GPU against the oracle's numpy arithmetic in 64 bits.

Tolerances, from the arithmetic:
  - tables, codes and scales, and the values read back, are equal: the maps are integers, the codes
    are decided exactly, and (code - 8) * scale is exact in fp32 (at most 15 significant bits);
  - rope: a value passes the norm's factor (a reciprocal square root within 2 units in the last
    place of 2^-23, three roundings of 2^-24), a sine and a cosine (2 units, and an angle that is off
    by at most pi * 2^-25 after reduction) and two products with one sum: below 16 * 2^-24 of the
    pair's length, so 1e-6 in the 2-norm and 2e-6 of the largest value element by element;
  - attention: tests/parity.py's tolerances of the library's attention (relative L2 1e-5,
    max-abs 2e-3).
"""
import numpy as np
import pytest

from oracle import kv4
from parity import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import q4_gemv_gqa_gb300 as g
    g.device_status(reset=True)
    return g, torch


def _cu(t, a, dtype=None):
    a = np.ascontiguousarray(a if dtype is None else np.asarray(a, dtype))
    return t.from_numpy(a).cuda()


# ---- append and gather -------------------------------------------------------------------------

ROWS = [
    # (T, n_kv, d, page, extra columns between the rows' ends)
    (1, 1, 64, 16, 0), (8, 8, 128, 16, 0), (9, 2, 64, 32, 3), (33, 3, 128, 64, 1), (5, 16, 256, 128, 4),
    (17, 4, 512, 256, 8), (130, 2, 128, 16, 0), (301, 1, 64, 32, 5),
]


@pytest.mark.parametrize("case", ROWS, ids=str)
def test_append_matches_the_oracle_bit_for_bit_and_touches_nothing_else(env, case):
    g, t = env
    T, n_kv, d, page, extra = case
    r = np.random.RandomState(T + d)
    n = n_kv * d
    x = (r.randn(T, 2 * n + extra) * np.exp(r.randn(2 * n + extra))).astype(np.float32)
    n_pages = -(-T // page) + 2
    slots = r.permutation(n_pages * page)[:T].astype(np.int32)
    if T > 4:
        slots[2] = -1
    ref = kv4.Pool(n_pages, page, n_kv, d)
    ref.bytes[:] = r.randint(0, 256, ref.bytes.shape)
    pool = _cu(t, ref.bytes.copy())
    ref.append(x[:, :n], x[:, n:2 * n], slots)
    dx = _cu(t, x)
    g.kv4_append(dx[:, :n], dx[:, n:2 * n], n_kv, d, _cu(t, slots), pool, page)
    assert np.array_equal(pool.cpu().numpy(), ref.bytes)
    # and back, with a repeated slot and a row left as it was
    at = np.concatenate([slots, slots[:1]])
    out = t.full((2, T + 1, n + extra), 7.0, device="cuda")
    g.kv4_gather(pool, page, n_kv, d, _cu(t, at), out[0][:, :n], out[1][:, :n])
    got = out.cpu().numpy()
    for which in range(2):
        want = np.full((T + 1, n + extra), 7.0)
        real = at >= 0
        want[real, :n] = ref.rows(at[real], which)
        assert np.array_equal(got[which], want.astype(np.float32))
    assert g.device_status(reset=True) == 0


def test_append_borders_zeros_huge_and_not_finite(env):
    g, t = env
    d, page = 64, 16
    r = np.random.RandomState(5)
    rows = []
    for s in (1.0, 0.37, 2.0 ** -14, 2.0 ** -24, 3 * 2.0 ** -24, 1000.0, 65504.0):
        s = float(np.float16(s))
        for sign in (1, -1):      # every border of every code, and one unit in the last place on either side
            b = np.float32(sign * s) * (np.arange(-8, 8, dtype=np.float32) + np.float32(0.5))
            b[0] = np.float32(-8 * sign * s)
            rows.append(np.concatenate([b, np.nextafter(b, np.float32(np.inf))]))
            rows.append(np.concatenate([b, np.nextafter(b, np.float32(-np.inf))]))
    rows += [np.zeros(32), np.full(32, 1e38), np.full(32, -3e38), np.full(32, 1e-45), r.randn(32) * 1e-8,
             np.where(np.arange(32) == 3, np.nan, 1.0), np.where(np.arange(32) == 30, np.inf, 1.0),
             np.where(np.arange(32) == 17, -np.inf, 1.0), np.where(np.arange(32) % 2, 5.0, -5.0),
             np.where(np.arange(32) % 2, -5.0, 5.0)]
    if len(rows) % 2:
        rows.append(np.ones(32))
    x = np.stack(rows).astype(np.float32).reshape(-1, d)
    T = len(x)
    ref = kv4.Pool(-(-T // page), page, 1, d)
    pool = _cu(t, ref.bytes.copy())
    slots = np.arange(T, dtype=np.int32)
    ref.append(x, x[::-1], slots)
    g.kv4_append(_cu(t, x), _cu(t, x[::-1]), 1, d, _cu(t, slots), pool, page)
    for which in range(2):
        out = t.zeros((T, d), device="cuda")
        g.kv4_gather(pool, page, 1, d, _cu(t, slots), *((out, None) if which == 0 else (None, out)))
        assert np.array_equal(out.cpu().numpy(), ref.rows(slots, which).astype(np.float32), equal_nan=True)


def test_append_and_gather_flag_bad_slots_and_leave_the_rest(env):
    g, t = env
    n_kv, d, page, n_pages = 2, 64, 16, 2
    r = np.random.RandomState(6)
    x = r.randn(5, n_kv * d).astype(np.float32)
    slots = np.array([3, 32, -2, 31, 2 ** 31 - 1], np.int32)
    ref = kv4.Pool(n_pages, page, n_kv, d, fill=0x55)
    pool = _cu(t, ref.bytes.copy())
    status = t.zeros(1, dtype=t.int32, device="cuda")
    g.kv4_append(_cu(t, x), _cu(t, x), n_kv, d, _cu(t, slots), pool, page, status=status)
    ref.append(x, x, slots)
    assert np.array_equal(pool.cpu().numpy(), ref.bytes)
    assert int(status) == g.DEVFLAG_PAGE_RANGE
    out = t.full((5, n_kv * d), 3.0, device="cuda")
    g.kv4_gather(pool, page, n_kv, d, _cu(t, slots), out, None)
    assert g.status_from_flags(g.device_status(reset=True)) == 5
    got = out.cpu().numpy()
    assert np.all(got[[1, 2, 4]] == 3.0) and np.array_equal(got[[0, 3]], ref.rows(slots[[0, 3]], 0).astype(np.float32))


# ---- rope --------------------------------------------------------------------------------------

ROPE = [
    # (T, n_q, n_kv, d, sections, interleaved, norm, in place, extra columns)
    (1, 16, 8, 128, [64], False, True, False, 0),
    (8, 32, 8, 128, [64], False, True, True, 1024),
    (5, 4, 2, 64, [16, 8, 8], False, True, False, 3),
    (7, 4, 2, 64, [12, 10, 10], True, False, True, 0),
    (33, 32, 4, 512, [64], False, True, False, 0),             # the first 128 dims rotate
    (6, 32, 16, 256, [24, 20, 20], True, True, False, 7),      # 128 of 256 dims
    (3, 3, 1, 80, [17], False, True, False, 2),                # sizes of no layout of its own
    (4, 1, 1, 2, [1], False, True, False, 0),
    (300, 6, 2, 128, [16, 16, 16, 16], True, True, False, 4),
    (2, 2, 1, 512, [100, 56, 100], False, False, False, 0),
    (9, 0, 2, 128, [30, 2], False, True, False, 0),
    (50, 2, 0, 256, [1], False, True, True, 0),
]


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_mrope_matches_the_oracle(env, case):
    g, t = env
    T, n_q, n_kv, d, sections, inter, norm, in_place, extra = case
    r = np.random.RandomState(d + T)
    cols = (n_q + n_kv) * d
    x = r.randn(T, cols + extra).astype(np.float32) * np.float32(3)
    pos = r.randint(0, 200000, (len(sections), T)).astype(np.int32)
    pos[:, 0] = 0
    if T > 3:
        pos[0, 1] = -1                         # a row of padding
        pos[:, 2] = 2 ** 31 - 1
    gq, gk = (1 + 0.2 * r.randn(2, d)).astype(np.float32) if norm else (None, None)
    want = kv4.qknorm_mrope(x[:, :cols], n_q, n_kv, d, gq, gk, 1e-6, pos, sections, 1e6, inter)
    dx = _cu(t, x)
    out = dx if in_place else t.full((T, cols + extra), 9.0, device="cuda")
    g.qknorm_mrope(dx, n_q, n_kv, d, *(None if a is None else _cu(t, a) for a in (gq, gk)), 1e-6, _cu(t, pos), sections,
                   1e6, out, interleaved=inter)
    got = out.cpu().numpy()
    assert np.array_equal(got[:, cols:], x[:, cols:] if in_place else np.full((T, extra), 9.0))
    real = pos[0] >= 0
    assert np.array_equal(got[~real], x[~real] if in_place else np.full(((~real).sum(), cols + extra), 9.0))
    got, want = got[real, :cols], want[real]
    far = np.arange(T)[real] == 2
    # at the last position 64-bit angles of the oracle are themselves off by 2^31 * 2^-52 (and the
    # frequencies by 2^-53 of theirs): 5e-7 of the pair's length
    assert_close(got[~far], want[~far], "rope", max_abs=2e-6 * np.abs(want).max(), rel_l2=1e-6)
    if far.any():
        assert_close(got[far], want[far], "rope at the last position", max_abs=4e-6 * np.abs(want).max(), rel_l2=2.5e-6)
    assert g.device_status(reset=True) == 0


def test_mrope_flags_negative_positions_and_skips_their_rows(env):
    g, t = env
    x = t.randn(4, 128, device="cuda")
    out = t.full((4, 128), 5.0, device="cuda")
    pos = t.tensor([[1, -2, 3, -1], [1, 1, -1, 7]], dtype=t.int32, device="cuda")
    status = t.zeros(1, dtype=t.int32, device="cuda")
    g.qknorm_mrope(x, 1, 1, 64, None, None, 1e-6, pos, [16, 16], 1e4, out, status=status)
    assert int(status) == g.DEVFLAG_POS_RANGE
    assert t.all(out[1:] == 5.0) and t.all(out[0] != 5.0)


# ---- tables ------------------------------------------------------------------------------------


def _table_case(r, B, page, most_cached, most_fresh, ends, short=0):
    cached = r.randint(0, most_cached + 1, B).astype(np.int32)
    fresh = r.randint(0, most_fresh + 1, B).astype(np.int32)
    fresh[r.rand(B) < ends] = -1
    held = -(-cached // page)
    need = np.where(fresh > 0, -(-(cached + np.maximum(fresh, 0)) // page) - held, 0)
    wide = int(max(1, (held + need).max(initial=1))) + 1
    n_pages = int(held.sum() + need.sum()) + 3 - short
    perm = r.permutation(n_pages).astype(np.int32)
    table = np.full((B, wide), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    head = int(r.randint(0, 5 * n_pages))
    ring = np.full(n_pages, -1, np.int32)
    ring[(head + np.arange(n_pages - at)) % n_pages] = perm[at:]
    return cached, fresh, table, ring, np.array([head, head + n_pages - at], np.int64)


def _run_tables(g, t, cached, fresh, page, table, ring, ring_in, T, status=None):
    B = len(cached)
    d = dict(table=_cu(t, table), ring=_cu(t, ring), ring_out=t.full((2,), -9, dtype=t.int64, device="cuda"))
    for k, n in (("kv_len", B), ("cu", B + 1), ("slot", T), ("pos", T), ("seq", T)):
        d[k] = t.full((n,), -9, dtype=t.int32, device="cuda")
    g.kv_block_tables(_cu(t, cached), _cu(t, fresh), page, d["table"], d["ring"], _cu(t, ring_in), d["ring_out"],
                      d["kv_len"], d["cu"], d["slot"], d["pos"], d["seq"], status=status)
    return {k: v.cpu().numpy() for k, v in d.items()}


TABLES = [
    # (B, page, most cached, most fresh, share ended, pages short, tokens short)
    (1, 16, 0, 1, 0.0, 0, 0), (1, 16, 100, 40, 0.0, 0, -5), (8, 16, 2048, 1, 0.0, 0, 0), (7, 32, 50, 90, 0.3, 0, -1),
    (33, 64, 300, 70, 0.2, 4, 0), (64, 128, 2000, 1, 0.1, 0, -64), (257, 256, 3000, 300, 0.2, 20, 100),
    (1025, 16, 60, 20, 0.25, 30, 500), (4096, 32, 100, 3, 0.3, 100, 0), (3, 16, 20, 100000, 0.0, 0, 0),
]


@pytest.mark.parametrize("case", TABLES, ids=str)
def test_tables_match_the_oracle(env, case):
    g, t = env
    B, page, most_cached, most_fresh, ends, short_pages, short_tokens = case
    r = np.random.RandomState(B + page)
    cached, fresh, table, ring, ring_in = _table_case(r, B, page, most_cached, most_fresh, ends, short_pages)
    if B > 30:
        cached[3], fresh[7] = -5, -2          # lengths that are refused
    T = max(0, int(np.maximum(fresh, 0).sum()) - short_tokens)
    status = t.zeros(1, dtype=t.int32, device="cuda")
    want = kv4.block_tables(cached, fresh, page, table, ring, ring_in, T)
    got = _run_tables(g, t, cached, fresh, page, table, ring, ring_in, T, status)
    for k in got:
        assert np.array_equal(got[k], want[k]), k
    assert int(status) == (g.DEVFLAG_NO_ROOM if want["refused"] else 0)


def test_tables_of_nothing_and_bad_rings(env):
    g, t = env
    empty = np.zeros(0, np.int32)
    got = _run_tables(g, t, empty, empty, 16, np.zeros((0, 3), np.int32), np.arange(4, dtype=np.int32),
                      np.array([2, 5], np.int64), 3)
    assert got["cu"].tolist() == [0] and got["slot"].tolist() == [-1] * 3 and got["ring_out"].tolist() == [2, 5]
    for ring_in in ([-1, 2], [5, 3], [0, 5], [2 ** 62, -2 ** 62]):
        status = t.zeros(1, dtype=t.int32, device="cuda")
        table = np.array([[3, -1], [2, -1]], np.int32)
        args = (np.array([1, 16], np.int32), np.array([1, 1], np.int32), 16, table, np.arange(4, dtype=np.int32),
                np.array(ring_in, np.int64), 8)
        want = kv4.block_tables(*args)
        got = _run_tables(g, t, *args, status=status)
        for k in got:
            assert np.array_equal(got[k], want[k]), (ring_in, k)
        assert want["bad_ring"] and int(status) == g.DEVFLAG_PAGE_RANGE | g.DEVFLAG_NO_ROOM


# ---- attention ---------------------------------------------------------------------------------


def _random_pool(r, t, n_pages, page, n_kv, d, amp=1.0):
    """A pool of random codes with scales of either sign; garbage is written where no token lies."""
    pool = kv4.Pool(n_pages, page, n_kv, d)
    tiles = pool.bytes.reshape(-1, 18 * d)
    tiles[:, :16 * d] = r.randint(0, 256, (len(tiles), 16 * d))
    s = (r.choice([-1, 1], (len(tiles), d)) * amp * np.exp(0.5 * r.randn(len(tiles), d)) / 5).astype(np.float16)
    tiles[:, 16 * d:] = s.view(np.uint8)
    return pool


def _unpack(pool, d):
    """Every row of a pool at once: [2][n_slots][n_kv][d] (the layout of oracle.kv4.Pool, checked against
    its read() in test_unpack_is_the_oracles)."""
    n_pages, page, n_kv = pool.bytes.shape[0], pool.page, pool.n_kv
    tiles = pool.bytes.reshape(n_pages, n_kv, page // 16, 18 * d)
    raw = tiles[..., :16 * d].reshape(n_pages, n_kv, page // 16, 2, d // 32, 16, 16)
    s = tiles[..., 16 * d:].copy().view(np.float16).reshape(n_pages, n_kv, page // 16, 2, d // 32, 16).astype(np.float64)
    x = (np.concatenate([raw & 15, raw >> 4], -1).astype(np.float64) - 8) * s[..., None]
    return x.transpose(3, 0, 2, 5, 1, 4, 6).reshape(2, n_pages * page, n_kv, d)


def test_unpack_is_the_oracles(env):
    r = np.random.RandomState(0)
    pool = _random_pool(r, None, 2, 32, 2, 64)
    x = _unpack(pool, 64)
    for which in range(2):
        assert np.array_equal(x[which].reshape(64, 128), pool.rows(range(64), which))


def _attn_case(r, t, kv_len, fresh, n_q, n_kv, d, page, spare_rows=0, amp=1.0, poison=True):
    """Tensors of a batch; every page holds garbage (NaN and infinite scales) behind its request's last token."""
    B = len(kv_len)
    held = [-(-L // page) for L in kv_len]
    n_pages = sum(held) + 2
    pool = _random_pool(r, t, n_pages, page, n_kv, d, amp)
    perm = r.permutation(n_pages)
    table = np.full((B, max(held + [1]) + 1), 10 ** 8, np.int32)    # entries behind a request are not read
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
        if poison:
            for s in range(kv_len[b], held[b] * page):
                slot = table[b, s // page] * page + s % page
                for h in range(n_kv):
                    for which in range(2):
                        bad = r.choice(np.array([0x7e00, 0xfe00, 0x7c00, 0xfc00], np.uint16), (d // 32,)).view(np.float16)
                        pool.write(slot, h, which, r.randint(0, 16, (d // 32, 32)).astype(np.uint8), bad)
    cu = np.concatenate([[0], np.cumsum(fresh)]).astype(np.int32)
    T = int(cu[-1]) + spare_rows
    q = (2 * r.randn(T, n_q * d)).astype(np.float32)
    return pool, table, cu, q


def _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, window, scale):
    out = np.zeros((cu[-1], n_q * d))
    x = _unpack(pool, d)
    for b, L in enumerate(kv_len):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        j = np.arange(L)
        slots = table[b, j // page] * page + j % page
        out[cu[b]:cu[b + 1]] = kv4.attention(q[cu[b]:cu[b + 1]].reshape(n, n_q, d), x[0, slots], x[1, slots], L, window,
                                             scale).reshape(n, -1)
    return out


def _attn_run(g, t, pool, table, cu, q, kv_len, n_q, n_kv, d, page, window, scale, status=None, workspace=None, fill=4.0):
    out = t.full(q.shape, fill, device="cuda")
    g.kv4_attn(_cu(t, q), n_q, n_kv, d, _cu(t, cu), _cu(t, kv_len, np.int32), _cu(t, table), _cu(t, pool.bytes), page,
               window, scale, out, workspace=workspace, status=status)
    return out.cpu().numpy()


ATTN = [
    # (kv lengths, new tokens, n_q, n_kv, d, page, window)
    ([1], [1], 4, 2, 64, 16, 0),
    ([2], [1], 2, 2, 128, 16, 0),
    ([15, 16, 17, 31, 32, 33], [1] * 6, 8, 4, 64, 16, 0),
    ([129], [1], 16, 8, 128, 16, 0),
    ([4097], [1], 16, 8, 128, 64, 0),
    ([1, 2049, 63, 700, 64, 65, 1500, 129], [1] * 8, 32, 8, 128, 32, 0),
    ([300, 5], [1, 1], 6, 2, 128, 16, 0),                     # three query heads to a KV head
    ([777], [1], 5, 1, 64, 256, 0),
    ([513, 40], [1, 1], 7, 1, 128, 32, 0),
    ([1000, 1], [1, 1], 8, 1, 128, 64, 0),
    ([2000], [1], 32, 16, 256, 64, 0),
    ([3001], [1], 32, 4, 512, 128, 0),
    ([100, 9], [1, 1], 4, 4, 512, 16, 0),
    ([3000, 100, 1024, 1025], [1] * 4, 32, 16, 256, 32, 1024),  # sliding windows
    ([50, 500], [1, 1], 4, 2, 64, 16, 1),
    ([50, 500, 7], [3, 5, 7], 4, 2, 64, 16, 9),
    ([40, 33, 5], [4, 0, 5], 16, 8, 128, 16, 0),              # chunks, an idle request, a whole prompt
    ([513, 2, 100], [8, 2, 1], 32, 8, 128, 32, 0),
    ([1111, 32, 300], [32, 32, 17], 32, 8, 128, 64, 0),
    ([600, 90], [33, 90], 8, 1, 128, 16, 70),
    ([256], [9], 32, 4, 512, 64, 0),
    ([700, 31], [20, 31], 32, 16, 256, 16, 100),
    ([0, 5, 0], [0, 1, 0], 4, 2, 64, 16, 0),                  # requests with nothing at all
    ([20000], [2], 2, 1, 128, 256, 0),
    ([90] * 40, [1] * 40, 4, 2, 64, 32, 0),
    ([33] * 5, [3, 1, 0, 2, 1], 3, 3, 64, 16, 0),
    ([1000], [1000], 4, 2, 64, 16, 0),                        # a whole prompt
    ([100, 61] * 18, [3, 1] * 18, 8, 2, 128, 16, 0),          # more than 32 requests, chunks among them
    ([130] * 40, [2] * 40, 8, 1, 128, 32, 50),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "kv%d_new%d_G%d_d%d_p%d_w%d_B%d" % (
    max(c[0]), max(c[1]), c[2] // c[3], c[4], c[5], c[6], len(c[0])))
def test_attention_matches_the_oracle(env, case):
    g, t = env
    kv_len, fresh, n_q, n_kv, d, page, window = case
    r = np.random.RandomState(sum(kv_len) + d)
    pool, table, cu, q = _attn_case(r, t, kv_len, fresh, n_q, n_kv, d, page, spare_rows=3)
    scale = d ** -0.5
    want = _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, window, scale)
    got = _attn_run(g, t, pool, table, cu, q, kv_len, n_q, n_kv, d, page, window, scale)
    assert np.all(got[cu[-1]:] == 4.0), "rows behind the last request were written"
    assert_close(got[:cu[-1]], want, "attention")
    again = _attn_run(g, t, pool, table, cu, q, kv_len, n_q, n_kv, d, page, window, scale)
    assert np.array_equal(got, again), "two runs differ"
    assert g.device_status(reset=True) == 0


@pytest.mark.parametrize("amp,qamp,scale", [(1e-4, 1.0, 0.125), (2000.0, 1e-3, 0.125), (1.0, 1e4, 1e-5), (1.0, 1e-6, 1e5),
                                            (1.0, 1.0, 0.0), (1.0, 0.3, -0.5), (0.02, 60.0, 0.125)], ids=str)
def test_attention_of_small_and_large_magnitudes(env, amp, qamp, scale):
    """Scales of the cache from 1e-4 / 8 up to thousands, and q far from one: the relative error of the
    output holds, since both enter the tensor cores under powers of two of their own."""
    g, t = env
    kv_len, fresh, n_q, n_kv, d, page = [300, 77], [1, 3], 8, 2, 128, 32
    r = np.random.RandomState(11)
    pool, table, cu, q = _attn_case(r, t, kv_len, fresh, n_q, n_kv, d, page, amp=amp)
    q = (q * np.float32(qamp)).astype(np.float32)
    want = _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, scale)
    got = _attn_run(g, t, pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, scale)
    assert_close(got, want, "attention", max_abs=2e-4 * np.abs(want).max(), rel_l2=1e-5)


def test_attention_of_scales_that_differ_a_lot_along_the_cache(env):
    g, t = env
    kv_len, n_q, n_kv, d, page = [900], 8, 2, 128, 32
    r = np.random.RandomState(12)
    pool, table, cu, q = _attn_case(r, t, kv_len, [1], n_q, n_kv, d, page)
    for j in range(0, 900, 7):          # some rows of V a thousand times larger, some a thousand times smaller
        slot = table[0, j // page] * page + j % page
        for h in range(n_kv):
            f = 10.0 ** r.uniform(-3, 3, d // 32)
            pool.write(slot, h, 1, r.randint(0, 16, (d // 32, 32)).astype(np.uint8), f.astype(np.float16))
    want = _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, d ** -0.5)
    got = _attn_run(g, t, pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, d ** -0.5)
    assert_close(got, want, "attention", max_abs=2e-4 * np.abs(want).max(), rel_l2=1e-5)


def test_attention_keeps_what_is_not_finite_to_its_row_and_head(env):
    g, t = env
    kv_len, fresh, n_q, n_kv, d, page = [100, 40], [2, 1], 4, 2, 64, 16
    r = np.random.RandomState(13)
    pool, table, cu, q = _attn_case(r, t, kv_len, fresh, n_q, n_kv, d, page)
    want = _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, 0.125)
    q[0, d + 3] = np.nan                                # row 0, head 1
    q[2, 3 * d] = np.inf                                # row 2, head 3
    got = _attn_run(g, t, pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, 0.125)
    bad = np.zeros(got.shape, bool)
    bad[0, d:2 * d] = bad[2, 3 * d:] = True
    assert np.all(np.isnan(got[bad])) and np.all(np.isfinite(got[~bad]))
    assert_close(got[~bad], want[~bad], "the other rows and heads")


def test_attention_device_checks(env):
    g, t = env
    kv_len, fresh, n_q, n_kv, d, page = [40, 40, 40, 40], [1, 1, 1, 1], 4, 2, 64, 16
    r = np.random.RandomState(14)
    pool, table, cu, q = _attn_case(r, t, kv_len, fresh, n_q, n_kv, d, page)
    want = _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, 0.125)
    status = t.zeros(1, dtype=t.int32, device="cuda")
    # request 1 claims more positions than its row of the table has, request 3 fewer than it has tokens
    long = [40, page * table.shape[1] + 1, 40, 0]
    got = _attn_run(g, t, pool, table, cu, q, long, n_q, n_kv, d, page, 0, 0.125, status=status)
    assert int(status) == g.DEVFLAG_POS_RANGE
    assert np.all(got[[1, 3]] == 4.0)
    assert_close(got[[0, 2]], want[[0, 2]], "the other requests")
    # pages outside the pool: their positions are left out; a request with no position left gives 0
    status.zero_()
    broken = table.copy()
    broken[0, 1], broken[2, :3] = pool.bytes.shape[0], (-1, 2 ** 31 - 1, -2 ** 31)
    got = _attn_run(g, t, pool, broken, cu, q, kv_len, n_q, n_kv, d, page, 0, 0.125, status=status)
    assert int(status) == g.DEVFLAG_PAGE_RANGE
    assert np.all(got[2] == 0.0)
    assert_close(got[[1, 3]], want[[1, 3]], "the other requests")
    keep = np.r_[0:16, 32:40]
    x = _unpack(pool, d)
    slots = table[0, keep // page] * page + keep % page
    part = kv4.attention(q[:1].reshape(1, n_q, d), x[0, slots], x[1, slots], len(keep), 0, 0.125)
    assert_close(got[0], part.reshape(-1), "the pages that are there")
    # cu_tokens out of order
    status.zero_()
    got = _attn_run(g, t, pool, table, np.array([0, 2, 1, 3, 99], np.int32), q, kv_len, n_q, n_kv, d, page, 0, 0.125, status=status)
    assert int(status) == g.DEVFLAG_POS_RANGE


def test_attention_refuses_a_short_workspace(env):
    g, t = env
    need = g.kv4_attn_workspace(4, 4, 8, 2, 64)
    if need == 0:
        return
    r = np.random.RandomState(15)
    pool, table, cu, q = _attn_case(r, t, [40] * 4, [1] * 4, 8, 2, 64, 16)
    with pytest.raises(g.GemError) as e:
        _attn_run(g, t, pool, table, cu, q, [40] * 4, 8, 2, 64, 16, 0, 0.1, workspace=t.empty(need - 1, dtype=t.uint8, device="cuda"))
    assert e.value.status == 7
    with pytest.raises(g.GemError) as e:
        _attn_run(g, t, pool, table, cu, q, [40] * 4, 8, 2, 64, 16, 0, 0.1,
                  workspace=t.empty(need + 256, dtype=t.uint8, device="cuda")[1:])
    assert e.value.status == 2


def test_binding_refuses_wrong_tensors(env):
    g, t = env
    pool = t.zeros((2, g.kv4_page_bytes(2, 64, 16)), dtype=t.uint8, device="cuda")
    x, slot = t.zeros((3, 128), device="cuda"), t.zeros(3, dtype=t.int32, device="cuda")
    with pytest.raises(ValueError):
        g.kv4_append(x, x.cpu(), 2, 64, slot, pool, 16)
    with pytest.raises(ValueError):
        g.kv4_append(x, x.half(), 2, 64, slot, pool, 16)
    with pytest.raises(ValueError):
        g.kv4_append(x, x, 2, 64, slot.long(), pool, 16)
    with pytest.raises(ValueError):
        g.kv4_append(x, x, 2, 64, slot, pool, 32)            # pages of another size
    with pytest.raises(ValueError):
        g.kv4_append(x, x[:, :100], 2, 64, slot, pool, 16)
    with pytest.raises(ValueError):
        g.kv4_append(x.t().contiguous().t(), x, 2, 64, slot, pool, 16)
    with pytest.raises(g.GemError):
        g.kv4_append(x[:1].expand(3, 128), x, 2, 64, slot, pool, 16)   # rows that overlap


# ---- the operators together --------------------------------------------------------------------


class _Server:
    """A serving loop's state for one layer: a pool, its tables and free pages."""

    def __init__(self, g, t, B, n_q, n_kv, d, page, n_pages, max_pages, T):
        self.g, self.t, self.page, self.heads = g, t, page, (n_q, n_kv, d)
        i32 = dict(dtype=t.int32, device="cuda")
        self.pool = t.zeros((n_pages, g.kv4_page_bytes(n_kv, d, page)), dtype=t.uint8, device="cuda")
        self.table = t.full((B, max_pages), -1, **i32)
        self.ring = t.arange(n_pages, **i32)
        self.counters = [t.tensor([0, n_pages], dtype=t.int64, device="cuda"), t.zeros(2, dtype=t.int64, device="cuda")]
        self.lens = [t.zeros(B, **i32), t.zeros(B, **i32)]
        self.fresh, self.cu = t.zeros(B, **i32), t.zeros(B + 1, **i32)
        self.slot, self.pos, self.seq = (t.zeros(T, **i32) for _ in range(3))
        self.gq, self.gk = (1 + 0.1 * t.randn(2, d, device="cuda")).unbind(0)
        self.qkv = t.zeros(T, (n_q + 2 * n_kv) * d, device="cuda")
        self.out = t.zeros(T, n_q * d, device="cuda")
        self.ws = t.empty(max(1, g.kv4_attn_workspace(T, B, n_q, n_kv, d)), dtype=t.uint8, device="cuda")
        self.status = t.zeros(1, **i32)

    def step(self, i):
        g, (n_q, n_kv, d), page = self.g, self.heads, self.page
        a, b = i % 2, 1 - i % 2
        g.kv_block_tables(self.lens[a], self.fresh, page, self.table, self.ring, self.counters[a], self.counters[b], self.lens[b],
                          self.cu, self.slot, self.pos, self.seq, status=self.status)
        g.qknorm_mrope(self.qkv, n_q, n_kv, d, self.gq, self.gk, 1e-6, self.pos[None], [d // 2], 1e6, self.qkv, status=self.status)
        g.kv4_append(self.qkv[:, n_q * d:(n_q + n_kv) * d], self.qkv[:, (n_q + n_kv) * d:], n_kv, d, self.slot, self.pool,
                     page, status=self.status)
        g.kv4_attn(self.qkv, n_q, n_kv, d, self.cu, self.lens[b], self.table, self.pool, page, 0, d ** -0.5, self.out,
                   workspace=self.ws, status=self.status)


# new tokens of each request step by step: prompts, decoding, ended requests and new ones in their place
STEPS = [[5, 40, 0], [1, 1, 17], [1, 1, 1], [-1, 3, 1], [33, 1, -1], [1, 0, 2], [1, 1, 1], [2, -1, 1]]


@pytest.mark.parametrize("graphs", [False, True], ids=["eager", "graph"])
def test_serving_steps_match_the_oracle(env, graphs):
    g, t = env
    n_q, n_kv, d, page, T = 8, 2, 64, 16, 64
    t.manual_seed(3)
    s = _Server(g, t, 3, n_q, n_kv, d, page, 9, 4, T)
    step = s.step
    if graphs:
        # one graph for each half of the ping-pong; captured before anything has run, replayed with other contents
        side, captured = t.cuda.Stream(), []
        saved = [x.clone() for x in s.counters]
        for i in range(2):
            side.wait_stream(t.cuda.current_stream())
            graph = t.cuda.CUDAGraph()
            with t.cuda.graph(graph, stream=side):
                s.step(i)
            captured.append(graph)
        for x, y in zip(s.counters, saved):
            x.copy_(y)
        step = lambda i: captured[i % 2].replay()  # noqa: E731
    r = np.random.RandomState(4)
    K, V = [np.zeros((0, n_kv, d))] * 3, [np.zeros((0, n_kv, d))] * 3
    gq, gk = s.gq.cpu().numpy(), s.gk.cpu().numpy()
    ring, counters, lens = np.arange(9, dtype=np.int32), [0, 9], [0, 0, 0]
    table = np.full((3, 4), -1, np.int32)
    for i, fresh in enumerate(STEPS):
        x = r.randn(T, (n_q + 2 * n_kv) * d).astype(np.float32)
        s.qkv.copy_(t.from_numpy(x))
        s.fresh.copy_(t.tensor(fresh, dtype=t.int32))
        s.out.fill_(6.0)
        step(i)
        maps = kv4.block_tables(lens, fresh, page, table, ring, counters, T)
        assert not maps["refused"]
        table, ring, counters, lens = maps["table"], maps["ring"], maps["ring_out"], maps["kv_len"]
        n = maps["cu"][-1]
        assert np.array_equal(s.table.cpu().numpy(), table) and np.array_equal(s.slot.cpu().numpy(), maps["slot"])
        rotated = kv4.qknorm_mrope(x[:n], n_q, n_kv, d, gq, gk, 1e-6, maps["pos"][None, :n], [d // 2], 1e6)
        qkv = s.qkv.cpu().numpy()
        assert_close(qkv[:n, :(n_q + n_kv) * d], rotated, "rope", max_abs=2e-6 * np.abs(rotated).max(), rel_l2=1e-6)
        # the cache holds the rows that the library itself rotated
        kk, vv = (kv4.values(*kv4.quantise(qkv[:n, lo:lo + n_kv * d].reshape(n, n_kv, d))).reshape(n, n_kv, d)
                  for lo in (n_q * d, (n_q + n_kv) * d))
        want = np.zeros((n, n_q * d))
        for b in range(3):
            a, z = maps["cu"][b], maps["cu"][b + 1]
            if fresh[b] < 0:
                K[b], V[b] = K[b][:0], V[b][:0]
            K[b], V[b] = np.concatenate([K[b], kk[a:z]]), np.concatenate([V[b], vv[a:z]])
            if z > a:
                want[a:z] = kv4.attention(qkv[a:z, :n_q * d].reshape(z - a, n_q, d), K[b], V[b], lens[b], 0, d ** -0.5).reshape(z - a, -1)
        got = s.out.cpu().numpy()
        assert_close(got[:n], want, "attention of step %d" % i)
        assert np.all(got[n:] == 6.0)
    assert int(s.status) == 0 and s.counters[0].tolist() == counters.tolist()


def test_attention_on_two_streams_with_a_workspace_each(env):
    g, t = env
    n_q, n_kv, d, page = 32, 8, 128, 32
    cases = []
    for k in range(2):
        r = np.random.RandomState(20 + k)
        kv_len = [2000 - 300 * k, 900]
        pool, table, cu, q = _attn_case(r, t, kv_len, [1, 1], n_q, n_kv, d, page)
        want = _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, d ** -0.5)
        ws = t.empty(max(1, g.kv4_attn_workspace(2, 2, n_q, n_kv, d)), dtype=t.uint8, device="cuda")
        cases.append(([_cu(t, a) for a in (q, cu, np.array(kv_len, np.int32), table, pool.bytes)], t.zeros(2, n_q * d, device="cuda"), ws, want))
    streams = [t.cuda.Stream() for _ in range(2)]
    t.cuda.synchronize()
    for _ in range(20):
        for (x, out, ws, _), s in zip(cases, streams):
            with t.cuda.stream(s):
                g.kv4_attn(x[0], n_q, n_kv, d, x[1], x[2], x[3], x[4], page, 0, d ** -0.5, out, workspace=ws)
    t.cuda.synchronize()
    for _, out, _, want in cases:
        assert_close(out.cpu().numpy(), want, "attention")


def test_attention_reports_a_copy_that_never_lands(env):
    """The first step of the first warp waits for 16 bytes more than its copies bring (nothing faults and
    nothing hangs: the wait runs out after the limit set here), and the next call is right again."""
    g, t = env
    for n_q, n_kv, d in ((8, 2, 128), (8, 1, 512)):
        r = np.random.RandomState(30)
        kv_len, page = [200], 32
        pool, table, cu, q = _attn_case(r, t, kv_len, [1], n_q, n_kv, d, page)
        args = (pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, d ** -0.5)
        status = t.zeros(1, dtype=t.int32, device="cuda")
        t.cuda.synchronize()
        g.set_wait_limit(1_000_000)
        g.set_test_injection(g.INJECT_RING_SHORTFALL)
        try:
            _attn_run(g, t, *args, status=status)
            t.cuda.synchronize()
        finally:
            g.set_test_injection(0)
            g.set_wait_limit(0)
        assert g.status_from_flags(int(status)) == 6
        status.zero_()
        got = _attn_run(g, t, *args, status=status)
        assert int(status) == 0
        assert_close(got, _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, d ** -0.5), "the call after")


# ---- what the documentation allows at its edges ---------------------------------------------------


def test_tables_pass_pages_that_are_none_on_as_slots_that_are_refused(env):
    g, t = env
    table = np.array([[9, -1, 2 ** 27 + 1], [1, 2, -5]], np.int32)
    ring = np.array([0, -7, 3, 2 ** 30], np.int32)
    args = (np.array([20, 33], np.int32), np.array([30, 2], np.int32), 16, table, ring, np.array([1, 4], np.int64), 40)
    want = kv4.block_tables(*args)
    status = t.zeros(1, dtype=t.int32, device="cuda")
    got = _run_tables(g, t, *args, status=status)
    for k in got:
        assert np.array_equal(got[k], want[k]), k
    # (request 0 is refused as well: its 50 tokens do not fit its row)
    assert (want["slot"] == -2 ** 31).any() and want["refused"] == [0]
    assert int(status) == g.DEVFLAG_PAGE_RANGE | g.DEVFLAG_NO_ROOM


@pytest.mark.parametrize("bits", [0x7e00, 0x7c00, 0xfc00])
@pytest.mark.parametrize("case", [([70, 40], [5, 1], 8, 2, 128, 16, 0), ([90, 64], [6, 3], 4, 2, 64, 32, 20),
                                  ([100], [9], 8, 1, 256, 16, 0), ([50], [2], 16, 2, 512, 16, 7)], ids=str)
def test_attention_keeps_scales_that_are_not_finite_to_the_rows_that_attend_them(env, case, bits):
    """A scale that is NaN or infinite at a position that some rows of a request attend and others mask
    (the newest tokens, and the oldest of a window): the others are as if it were not there."""
    g, t = env
    kv_len, fresh, n_q, n_kv, d, page, window = case
    r = np.random.RandomState(40 + d)
    pool, table, cu, q = _attn_case(r, t, kv_len, fresh, n_q, n_kv, d, page)
    want = _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, window, d ** -0.5)
    bad = np.zeros((len(q), n_q, d), bool)
    G = n_q // n_kv
    for b, L in enumerate(kv_len):
        n = fresh[b]
        spots = [L - 1 - n // 2] + ([L - window] if window else [])
        for j in spots:
            slot = table[b, j // page] * page + j % page
            for which in range(2):
                blk = int(r.randint(0, d // 32))
                p, c, at = pool._at(slot, n_kv - 1, which, blk)
                pool.bytes[p, at:at + 2] = np.array([bits], np.uint16).view(np.uint8)
                for i in range(n):
                    pos = L - n + i
                    if j <= pos and (not window or j > pos - window):
                        dims = slice(blk * 32, blk * 32 + 32) if which else slice(None)
                        bad[cu[b] + i, (n_kv - 1) * G:, dims] = True
    bad = bad.reshape(len(q), -1)
    got = _attn_run(g, t, pool, table, cu, q, kv_len, n_q, n_kv, d, page, window, d ** -0.5)
    assert not np.any(np.isfinite(got[bad])), "a row that attends the position hides it"
    assert bad.any() and not bad.all()
    assert_close(got[~bad], want[~bad], "the rows that do not")


def test_attention_of_as_many_requests_as_allowed(env):
    g, t = env
    for n_q, n_kv, d, B in ((8, 1, 512, 4096), (4, 2, 64, 4096), (2, 2, 128, 33)):
        page = 16
        r = np.random.RandomState(B)
        kv_len = r.randint(1, 20, B)
        fresh = np.ones(B, np.int64)
        fresh[r.rand(B) < 0.2] = 0
        pool = _random_pool(r, t, 64, page, n_kv, d)
        table = r.randint(0, 64, (B, 2)).astype(np.int32)      # requests may share pages
        cu = np.concatenate([[0], np.cumsum(fresh)]).astype(np.int32)
        q = (2 * r.randn(int(cu[-1]), n_q * d)).astype(np.float32)
        x = _unpack(pool, d)
        got = _attn_run(g, t, pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, d ** -0.5)
        for b in r.permutation(np.nonzero(fresh)[0])[:60]:
            j = np.arange(kv_len[b])
            slots = table[b, j // page] * page + j % page
            want = kv4.attention(q[cu[b]:cu[b + 1]].reshape(1, n_q, d), x[0, slots], x[1, slots], kv_len[b], 0, d ** -0.5)
            assert_close(got[cu[b]], want.reshape(-1), "request %d of %d" % (b, B))
    assert g.device_status(reset=True) == 0


def test_attention_reads_and_writes_columns_of_wider_rows(env):
    """q a column range of a QKV row, out a column range that is not 16-byte aligned; a stream of the
    caller's with no workspace given."""
    g, t = env
    kv_len, fresh, n_q, n_kv, d, page = [300, 35], [1, 3], 6, 2, 128, 32
    r = np.random.RandomState(50)
    pool, table, cu, q = _attn_case(r, t, kv_len, fresh, n_q, n_kv, d, page)
    want = _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, d ** -0.5)
    wide = t.full((len(q), 8 + n_q * d + 512), float("nan"), device="cuda")
    wide[:, 8:8 + n_q * d] = _cu(t, q)
    out = t.full((len(q), n_q * d + 7), 4.0, device="cuda")
    args = [_cu(t, cu), _cu(t, kv_len, np.int32), _cu(t, table), _cu(t, pool.bytes)]
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    g.kv4_attn(wide[:, 8:], n_q, n_kv, d, *args, page, 0, d ** -0.5, out[:, 3:], stream=s)
    s.synchronize()
    got = out.cpu().numpy()
    assert_close(got[:, 3:3 + n_q * d], want, "attention")
    assert np.all(got[:, :3] == 4.0) and np.all(got[:, 3 + n_q * d:] == 4.0)
    with pytest.raises(g.GemError) as e:
        g.kv4_attn(wide[:, 8:], n_q, n_kv, d, *args, page, 0, d ** -0.5, wide[:, 8:])
    assert e.value.status == 1


def test_two_captured_steps_share_a_workspace_in_turn(env):
    g, t = env
    n_q, n_kv, d, page = 8, 2, 128, 16
    ws = t.empty(g.kv4_attn_workspace(2, 2, n_q, n_kv, d), dtype=t.uint8, device="cuda")
    graphs = []
    for k in range(2):
        r = np.random.RandomState(60 + k)
        kv_len = [1500 - 1000 * k, 77]
        pool, table, cu, q = _attn_case(r, t, kv_len, [1, 1], n_q, n_kv, d, page)
        want = _attn_want(pool, table, cu, q, kv_len, n_q, n_kv, d, page, 0, d ** -0.5)
        x = [_cu(t, q), _cu(t, cu), _cu(t, kv_len, np.int32), _cu(t, table), _cu(t, pool.bytes)]
        out = t.zeros(2, n_q * d, device="cuda")
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            g.kv4_attn(x[0], n_q, n_kv, d, x[1], x[2], x[3], x[4], page, 0, d ** -0.5, out, workspace=ws)
        graphs.append((graph, out, want, x))
    for _ in range(10):
        for graph, _, _, _ in graphs:
            graph.replay()
    t.cuda.synchronize()
    for _, out, want, _ in graphs:
        assert_close(out.cpu().numpy(), want, "attention")


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing of the library has run in the process: every call's set-up happens under capture."""
    import subprocess
    import sys

    from conftest import ROOT
    code = """
import torch as t, q4_gemv_gqa_gb300 as g
i32 = dict(dtype=t.int32, device="cuda")
n_q, n_kv, d, page = 4, 2, 64, 16
pool = t.zeros((4, g.kv4_page_bytes(n_kv, d, page)), dtype=t.uint8, device="cuda")
qkv = t.randn(2, (n_q + 2 * n_kv) * d, device="cuda")
table, ring = t.full((1, 2), -1, **i32), t.arange(4, **i32)
rin, rout = t.tensor([0, 4], device="cuda"), t.zeros(2, dtype=t.int64, device="cuda")
cached, fresh, kv, cu = t.zeros(1, **i32), t.full((1,), 2, **i32), t.zeros(1, **i32), t.zeros(2, **i32)
slot, pos, seq = (t.zeros(2, **i32) for _ in range(3))
out = t.zeros(2, n_q * d, device="cuda")
kk, vv = t.zeros(2, n_kv * d, device="cuda"), t.zeros(2, n_kv * d, device="cuda")
ws = t.zeros(48 << 20, dtype=t.uint8, device="cuda")
t.cuda.synchronize()
graph = t.cuda.CUDAGraph()
with t.cuda.graph(graph):
    g.kv_block_tables(cached, fresh, page, table, ring, rin, rout, kv, cu, slot, pos, seq)
    g.qknorm_mrope(qkv, n_q, n_kv, d, None, None, 1e-6, pos[None], [32], 1e4, qkv)
    g.kv4_append(qkv[:, n_q * d:(n_q + n_kv) * d], qkv[:, (n_q + n_kv) * d:], n_kv, d, slot, pool, page)
    g.kv4_gather(pool, page, n_kv, d, slot, kk, vv)
    g.kv4_attn(qkv, n_q, n_kv, d, cu, kv, table, pool, page, 0, 0.125, out, workspace=ws)
graph.replay()
t.cuda.synchronize()
# the first row attends itself alone: its output is its own value
want = vv[0].view(n_kv, 1, d).expand(n_kv, n_q // n_kv, d).reshape(-1)
assert kv.item() == 2 and slot.tolist() == [0, 1], (kv, slot)
assert t.allclose(out[0], want, rtol=1e-5, atol=1e-6), (out[0] - want).abs().max()
assert g.device_status() == 0
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=280)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("case", [(8, 4, 256, 6000, 16), (32, 4, 256, 6000, 16), (4, 2, 512, 6000, 12), (16, 2, 512, 6000, 12)], ids=str)
def test_attention_whose_value_scales_grow_in_part_of_the_dims(env, case):
    """The warps that share a head rescale their own sums when V's scales grow, and parts of a sequence
    are joined under the maximum of one of them: it has to be the same for all.  The scales of the last
    dims double every 32 positions for 256 positions, over and over, those of the first dims do not; the
    batch is large enough for every warp to pass several of them (the requests share their pages)."""
    g, t = env
    n_q, n_kv, d, L, B = case
    page = 64
    r = np.random.RandomState(70 + d + n_q)
    pool, table, _, _ = _attn_case(r, t, [L], [1], n_q, n_kv, d, page)
    tiles = pool.bytes.reshape(len(pool.bytes), n_kv, page // 16, 18 * d)
    scales = tiles[..., 16 * d:].view(np.float16).reshape(len(pool.bytes), n_kv, page // 16, 2, d // 32, 16)
    for j in range(0, L // 16 * 16, 16):
        at = scales[table[0, j // page], :, j % page // 16, 1, d // 64:]
        at[:] = (at.astype(np.float64) * 2.0 ** (j % 256 // 32 - 4)).astype(np.float16)
    x = _unpack(pool, d)
    slots = table[0, np.arange(L) // page] * page + np.arange(L) % page
    K, V = x[0, slots], x[1, slots]
    q = (2 * r.randn(B, n_q * d)).astype(np.float32)
    got = _attn_run(g, t, pool, np.repeat(table, B, 0), np.arange(B + 1, dtype=np.int32), q, [L] * B, n_q, n_kv, d, page, 0,
                    d ** -0.5)
    want = np.stack([kv4.attention(q[b].reshape(1, n_q, d), K, V, L, 0, d ** -0.5)[0] for b in range(B)])
    got = got.reshape(want.shape)
    for half in (slice(0, d // 2), slice(d // 2, d)):
        assert_close(got[..., half], want[..., half], "dims %s" % half, max_abs=2e-4 * np.abs(want[..., half]).max(), rel_l2=1e-5)


def test_attention_sums_do_not_drift_along_a_long_sequence(env):
    """Every warp sums some 80 steps of 32 positions here.  Scores and probabilities carry some 2^-22 each and
    the sums are rounded to nearest, 2^-24 a step, so their errors add up as a random walk: the result is
    within 2e-6.  (Kept in the tensor cores, which cut off toward zero, they would drift by 2^-25 a
    product, 5e-6 after 320.)"""
    g, t = env
    n_q, n_kv, d, page, L, B, new = 16, 8, 128, 128, 12000, 8, 26
    r = np.random.RandomState(80)
    pool, table, _, _ = _attn_case(r, t, [L], [1], n_q, n_kv, d, page)
    cu = (np.arange(B + 1) * new).astype(np.int32)
    q = (2 * r.randn(B * new, n_q * d)).astype(np.float32)
    got = _attn_run(g, t, pool, np.repeat(table, B, 0), cu, q, [L] * B, n_q, n_kv, d, page, 0, d ** -0.5)
    x = _unpack(pool, d)
    slots = table[0, np.arange(L) // page] * page + np.arange(L) % page
    K, V = x[0, slots], x[1, slots]
    rows = r.permutation(B * new)[:24]
    want = np.stack([kv4.attention(q[i].reshape(1, n_q, d), K, V, L - new + 1 + i % new, 0, d ** -0.5)[0] for i in rows])
    assert_close(got[rows].reshape(want.shape), want, "attention", max_abs=1e-5 * np.abs(want).max(), rel_l2=2e-6)
