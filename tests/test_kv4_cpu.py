"""The paged 4-bit KV cache without a GPU: the oracle against known answers and invariants, and the
library's host-side refusals, which come before any CUDA call."""
import ctypes as C

import numpy as np
import pytest

from oracle import kv4

OK, INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 7
D = C.c_void_p(0x1000)      # a device pointer that no call reaches
ODD = C.c_void_p(0x1004)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._build_module().build()
    from q4_gemv_gqa_gb300 import _lib
    return _lib.load()


# ---- the oracle -------------------------------------------------------------------------------


def test_quantise_known_block():
    x = np.arange(-16, 16, dtype=np.float32) / 2      # -8 .. 7.5: the scale is exactly 1
    codes, scales = kv4.quantise(x)
    assert scales[0] == 1.0
    # halves go to the even code: -7.5 -> -8, -6.5 -> -6, 0.5 -> 0, 7.5 -> 8 which is held to 7
    want = np.clip(8 + np.rint(x), 0, 15)
    assert np.array_equal(codes[0], want) and codes[0][1] == 0 and codes[0][3] == 2 and codes[0][31] == 15


def test_quantise_takes_the_first_of_equal_magnitudes_and_keeps_its_sign():
    x = np.zeros(32, np.float32)
    x[5], x[9] = 4.0, -4.0
    codes, scales = kv4.quantise(x)
    assert scales[0] == -0.5 and codes[0][5] == 0 and codes[0][9] == 15
    x[5], x[9] = -4.0, 4.0
    assert kv4.quantise(x)[1][0] == 0.5


def test_quantise_zero_huge_and_not_finite():
    assert np.all(kv4.quantise(np.zeros(32))[0] == 8) and kv4.quantise(np.zeros(32))[1][0] == 0
    x = np.full(32, 1e30, np.float32)
    codes, scales = kv4.quantise(x)
    assert scales[0] == -65504 and np.all(codes == 0)
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones(32, np.float32)
        x[3] = bad
        assert np.isnan(kv4.quantise(x)[1][0])


def test_quantise_is_within_half_a_step():
    x = np.random.RandomState(1).randn(500, 32).astype(np.float32)
    codes, scales = kv4.quantise(x)
    back = kv4.values(codes, scales).reshape(500, 32)
    s = np.abs(scales.astype(np.float64))
    # half a step, and one step where the value opposite to the largest one has no code of its own;
    # the scale's own rounding moves the largest value by at most 2^-11 of itself, 8 steps
    assert np.all(np.abs(back - x) <= s * (1.0 + 8 * 2.0 ** -11) + 1e-12)
    inner = np.abs(x) <= 7.5 * s
    assert np.all((np.abs(back - x) <= 0.5 * s * (1 + 1e-6))[inner])


def test_pool_rows_round_trip_and_do_not_overlap():
    pool = kv4.Pool(3, 32, 2, 64)
    r = np.random.RandomState(2)
    k, v = r.randn(96, 128).astype(np.float32), r.randn(96, 128).astype(np.float32)
    pool.append(k, v, r.permutation(96))
    r = np.random.RandomState(2)
    r.randn(96, 128), r.randn(96, 128)
    slots = r.permutation(96)
    for which, x in enumerate((k, v)):
        codes, scales = kv4.quantise(x.reshape(96, 2, 64))
        assert np.array_equal(pool.rows(slots, which), kv4.values(codes, scales).reshape(96, 128))
    assert pool.bytes.nbytes == 96 * 2 * 2 * (32 + 4)


def test_tables_hand_worked():
    # pages of 16; request 0 grows into a second page, 1 ends, 2 is new with 33 tokens, 3 idles
    table = np.full((4, 4), -1)
    table[0, 0], table[1, :2], table[3, 0] = 7, (3, 4), 5
    ring = np.array([0, 1, 2, 6, 8, 9, -1, -1, -1, -1])
    got = kv4.block_tables([16, 20, 0, 1], [1, -1, 33, 0], 16, table, ring, [0, 6], 40)
    assert got["table"].tolist() == [[7, 0, -1, -1], [3, 4, -1, -1], [1, 2, 6, -1], [5, -1, -1, -1]]
    assert got["ring_out"].tolist() == [4, 8] and got["ring"][6:8].tolist() == [3, 4]
    assert got["kv_len"].tolist() == [17, 0, 33, 1] and got["cu"].tolist() == [0, 1, 1, 34, 34]
    assert got["slot"][:3].tolist() == [0, 16, 17] and got["slot"][33] == 6 * 16 and got["slot"][34] == -1
    assert got["seq"][33] == 2 and got["pos"][33] == 32 and not got["refused"]


def test_tables_refusals_keep_the_rest_going():
    table = np.full((5, 2), -1)
    table[1, 0] = 3
    # 2 free pages: request 0 wants 3 of them, 1 needs none, 2 wants one (the sum is past 2), 3 has a
    # bad length, 4 wants 3 more
    got = kv4.block_tables([0, 4, 0, -1, 0], [40, 1, 1, 1, 33], 16, np.hstack([table, table]), [1, 2, 0, 0], [0, 2], 64)
    assert got["refused"] == [0, 2, 3, 4] and got["kv_len"].tolist() == [0, 5, 0, -1, 0]
    got = kv4.block_tables([0, 4], [40, 1], 16, table[:2], [1, 2, 0, 0], [0, 2], 64)
    assert got["refused"] == [0] and got["kv_len"].tolist() == [0, 5] and got["slot"][0] == 3 * 16 + 4


def test_mrope_one_axis_keeps_norms_and_equal_axes_agree():
    r = np.random.RandomState(3)
    x = r.randn(5, 3 * 64)
    pos = np.arange(5)[None] + 100
    one = kv4.qknorm_mrope(x, 2, 1, 64, None, None, 0.0, pos, [32], 1e4)
    assert np.allclose(np.linalg.norm(one), np.linalg.norm(x), rtol=1e-13)
    for inter in (False, True):
        three = kv4.qknorm_mrope(x, 2, 1, 64, None, None, 0.0, np.repeat(pos, 3, 0), [12, 10, 10], 1e4, inter)
        assert np.array_equal(one, three)
    assert kv4.axis_of([4, 2, 2], True).tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    assert kv4.axis_of([4, 2, 2], False).tolist() == [0, 0, 0, 0, 1, 1, 2, 2]


def test_attention_of_one_position_is_its_value_and_window_one_is_the_last():
    r = np.random.RandomState(4)
    q, k, v = r.randn(1, 4, 64), r.randn(9, 2, 64), r.randn(9, 2, 64)
    assert np.allclose(kv4.attention(q, k[:1], v[:1], 1, 0, 1.0)[0], np.repeat(v[0], 2, 0))
    assert np.allclose(kv4.attention(q, k, v, 9, 1, 1.0)[0], np.repeat(v[8], 2, 0))


# ---- host-side refusals ------------------------------------------------------------------------


def test_page_bytes(lib):
    assert lib.gem_kv4_page_bytes(8, 128, 16) == kv4.page_bytes(8, 128, 16) == 16 * 8 * 144
    for n_kv, d, page in ((0, 128, 16), (-1, 128, 16), (8, 96, 16), (8, 128, 24), (8, 128, 512), (8, 128, 0), (8, 1024, 16)):
        assert lib.gem_kv4_page_bytes(n_kv, d, page) == 0


def _tables(lib, **kw):
    a = dict(cached=D, fresh=D, B=2, page=16, table=D, max_pages=4, ring=D, n_pages=8, ring_in=D,
             ring_out=C.c_void_p(0x2000), kv_len=C.c_void_p(0x3000), cu=D, slot=D, pos=D, seq=D, T_cap=8)
    a.update(kw)
    return lib.gem_kv_block_tables(*a.values(), None, None)


def test_tables_refusals(lib):
    for kw in (dict(B=-1), dict(max_pages=-1), dict(n_pages=-1), dict(T_cap=-1), dict(cached=None), dict(fresh=None),
               dict(table=None), dict(ring=None), dict(ring_in=None), dict(ring_out=None), dict(kv_len=None),
               dict(cu=None), dict(slot=None), dict(pos=None), dict(seq=None), dict(ring_out=D), dict(kv_len=D)):
        assert _tables(lib, **kw) == INVALID, kw
    for kw in (dict(B=4097), dict(page=8), dict(page=48), dict(page=512), dict(n_pages=1 << 27), dict(max_pages=1 << 27),
               dict(T_cap=1 << 31)):
        assert _tables(lib, **kw) == UNSUPPORTED, kw


def _mrope(lib, **kw):
    secs = (16, 8, 8)
    a = dict(qkv=D, ldqkv=512, T=3, n_q=4, n_kv=2, d=64, gq=None, gk=None, eps=1e-6, pos=D, ldpos=3,
             n_axes=3, sections=(C.c_int32 * 3)(*secs), inter=0, theta=1e4,
             out=C.c_void_p(0x9000), ldo=384)
    a.update(kw)
    return lib.gem_qknorm_mrope(*a.values(), None, None)


def test_mrope_refusals(lib):
    assert _mrope(lib, T=0) == OK and _mrope(lib, n_q=0, n_kv=0) == OK
    for kw in (dict(T=-1), dict(n_q=-1), dict(n_kv=-1), dict(d=0), dict(eps=-1.0), dict(eps=float("nan")), dict(inter=2),
               dict(theta=0.0), dict(theta=float("nan")), dict(theta=float("inf")), dict(qkv=None), dict(out=None),
               dict(pos=None), dict(ldqkv=383), dict(ldo=383), dict(ldpos=2), dict(out=D, ldo=511),
               dict(sections=None), dict(sections=(C.c_int32 * 3)(16, 16, 8)), dict(sections=(C.c_int32 * 3)(0, 0, 0)),
               dict(sections=(C.c_int32 * 3)(16, -1, 8)), dict(sections=(C.c_int32 * 3)(10, 12, 10), inter=1)):
        assert _mrope(lib, **kw) == INVALID, kw
    for kw in (dict(d=65), dict(d=514, ldqkv=4000, ldo=4000), dict(n_axes=0), dict(n_axes=5)):
        assert _mrope(lib, **kw) == UNSUPPORTED, kw


def _append(lib, **kw):
    a = dict(k=D, ldk=128, v=D, ldv=128, T=3, n_kv=2, d=64, slot=D, pool=D, n_pages=4, page=16)
    a.update(kw)
    return lib.gem_kv4_append(*a.values(), None, None)


def _gather(lib, **kw):
    a = dict(pool=D, n_pages=4, page=16, n_kv=2, d=64, slot=D, T=3, k=D, ldk=128, v=D, ldv=128)
    a.update(kw)
    return lib.gem_kv4_gather(*a.values(), None, None)


def test_append_and_gather_refusals(lib):
    for f in (_append, _gather):
        assert f(lib, T=0) == OK and f(lib, n_kv=0) == OK
        for kw in (dict(T=-1), dict(n_kv=-1), dict(d=0), dict(n_pages=-1), dict(slot=None), dict(pool=None),
                   dict(ldk=127), dict(ldv=127)):
            assert f(lib, **kw) == INVALID, (f, kw)
        for kw in (dict(d=32, ldk=999, ldv=999), dict(d=96, ldk=999, ldv=999), dict(page=24), dict(page=8),
                   dict(n_pages=1 << 27)):
            assert f(lib, **kw) == UNSUPPORTED, (f, kw)
        assert f(lib, pool=ODD) == MISALIGNED
    assert _append(lib, k=None) == INVALID and _append(lib, v=None) == INVALID
    assert _gather(lib, k=None, v=None) == OK


def _attn(lib, **kw):
    a = dict(q=D, ldq=256, T=3, cu=D, kv_len=D, B=2, n_q=4, n_kv=2, d=64, table=D, max_pages=4, pool=D, n_pages=4,
             page=16, window=0, scale=0.125, out=C.c_void_p(0x9000), ldo=256, ws=C.c_void_p(0x10000), ws_bytes=1 << 30)
    a.update(kw)
    return lib.gem_kv4_attn(*a.values(), None, None)


def test_attn_refusals(lib):
    assert _attn(lib, T=0) == OK and _attn(lib, B=0) == OK and _attn(lib, n_q=0) == OK
    for kw in (dict(T=-1), dict(B=-1), dict(n_q=-4), dict(n_kv=-2), dict(n_q=5), dict(n_kv=0), dict(window=-1),
               dict(max_pages=-1), dict(n_pages=-1), dict(q=None), dict(out=None), dict(cu=None), dict(kv_len=None),
               dict(table=None), dict(pool=None), dict(ldq=252), dict(ldo=255), dict(d=0), dict(out=D, q=D)):
        assert _attn(lib, **kw) == INVALID, kw
    for kw in (dict(n_q=18, ldq=9999 * 4, ldo=9999), dict(d=96, ldq=800, ldo=800), dict(page=24), dict(B=4097),
               dict(T=1 << 31), dict(T=1 << 30), dict(max_pages=1 << 27), dict(n_pages=1 << 27)):
        assert _attn(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(q=ODD), dict(ldq=257), dict(pool=ODD)):
        assert _attn(lib, **kw) == MISALIGNED, kw
