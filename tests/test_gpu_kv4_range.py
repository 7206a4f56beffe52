"""Paged 4-bit attention at the ends of its value range, row by row and block by block.

A result is a weighted mean of the cached values, so its error is measured against the same mean of
their magnitudes, W = sum_j softmax_j |V_j|, over a row's block of 32 dims (no cancellation, and no block
hides another).  From the arithmetic, relative to W:
  - a probability enters as hi + lo of 11 bits each, what is left is below 2^-22, and the tensor cores
    cut a sum of 16 products off at 2^-24 of its largest, four times a step: 2^-22 + 2^-22;
  - a score x = q.K scale log2(e) has q's split, 2^-22 of sum |q K|, and the rounding of some ten sums, 2^-24
    of |x| each; the inputs here keep sum |q K| scale log2(e) below 32 and |x| of what counts below 12, so p is
    off by ln 2 (32 * 2^-22 + 120 * 2^-24) = 1.0e-5 at worst if all of it adds up; the signs are random,
    so that a fifth of it, 2e-6, is left;
  - the exponential is within 2^-22, the sums and joins add some ten roundings of 2^-24.
Together below 4e-6 in the 2-norm of a block.
"""
import numpy as np
import pytest

from oracle import kv4
from test_gpu_kv4 import _attn_case, _attn_run, _unpack, env  # noqa: F401

pytestmark = pytest.mark.gpu

TOL = 4e-6


def _scales(pool, table, b, L, which):
    """A view of request b's scales of K (0) or V (1): [L] rows of views [n_kv, d / 32]."""
    d, page, n_kv = pool.d, pool.page, pool.n_kv
    tiles = pool.bytes.reshape(len(pool.bytes), n_kv, page // 16, 18 * d)
    s = tiles[..., 16 * d:].view(np.float16).reshape(len(pool.bytes), n_kv, page // 16, 2, d // 32, 16)
    return [s[table[b, j // page], :, j % page // 16, which, :, j % 16] for j in range(L)]


def _check(pool, table, cu, q, kv_len, heads, window, scale, got, tol=TOL):
    """Every (row, head, block of 32 dims) against the oracle, relative to the weighted magnitudes."""
    n_q, n_kv, d, page = heads
    x = _unpack(pool, d)
    worst = 0.0
    for b, L in enumerate(kv_len):
        n = cu[b + 1] - cu[b]
        slots = table[b, np.arange(L) // page] * page + np.arange(L) % page
        rows = q[cu[b]:cu[b + 1]].reshape(n, n_q, d)
        K, V = x[0, slots], x[1, slots]
        want = kv4.attention(rows, K, V, L, window, scale).reshape(n, n_q, -1, 32)
        size = kv4.attention(rows, K, np.abs(V), L, window, scale).reshape(n, n_q, -1, 32)
        have = got[cu[b]:cu[b + 1]].reshape(want.shape).astype(np.float64)
        assert np.all(np.isfinite(have)), "not finite"
        rel = np.linalg.norm(have - want, axis=-1) / np.linalg.norm(size, axis=-1)
        worst = max(worst, rel.max())
    assert worst <= tol, "worst block is %.2e off" % worst


# (kv lengths, new tokens, n_q, n_kv, d, page, window): one for each form of the kernel
SHAPES = [
    ([900], [1], 8, 2, 128, 32, 0), ([300, 77], [1, 1], 4, 2, 64, 16, 0), ([500], [1], 8, 1, 128, 64, 0),
    ([400], [5], 8, 2, 128, 32, 0), ([333], [1], 8, 1, 64, 16, 0), ([260], [6], 6, 2, 64, 32, 0),
    ([700], [1], 8, 4, 256, 32, 200), ([300], [1], 8, 1, 256, 16, 0), ([600], [1], 4, 2, 512, 64, 0),
    ([500], [1], 8, 1, 512, 32, 0),
]
IDS = lambda c: "kv%d_new%d_G%d_d%d_w%d" % (max(c[0]), max(c[1]), c[2] // c[3], c[4], c[6])  # noqa: E731


def _prepared(case, seed):
    kv_len, fresh, n_q, n_kv, d, page, window = case
    r = np.random.RandomState(seed + d + n_q)
    pool, table, cu, q = _attn_case(r, None, kv_len, fresh, n_q, n_kv, d, page)
    q *= np.float32(0.5)
    return r, pool, table, cu, q, (n_q, n_kv, d, page), window, d ** -0.5


def _go(env, case, pool, table, cu, q, scale):
    g, t = env
    kv_len, _, n_q, n_kv, d, page, window = case
    got = _attn_run(g, t, pool, table, cu, q, kv_len, n_q, n_kv, d, page, window, scale)
    _check(pool, table, cu, q, kv_len, (n_q, n_kv, d, page), window, scale, got)
    assert g.device_status(reset=True) == 0


@pytest.mark.parametrize("case", SHAPES, ids=IDS)
def test_blocks_whose_value_scales_differ_by_powers_of_two(env, case):
    """V's scales of each block of dims around a size of its own, 2^-12 to 2^12."""
    r, pool, table, cu, q, _, _, scale = _prepared(case, 1)
    size = 2.0 ** np.linspace(-12, 12, pool.nb)[r.permutation(pool.nb)]
    for b, L in enumerate(case[0]):
        for s in _scales(pool, table, b, L, 1):
            s[:] = (s.astype(np.float64) * size).astype(np.float16)
    _go(env, case, pool, table, cu, q, scale)


@pytest.mark.parametrize("near", [False, True], ids=["apart", "in_one_step"])
@pytest.mark.parametrize("case", SHAPES, ids=IDS)
def test_a_position_with_huge_value_scales_and_no_weight(env, case, near):
    """One position in eighty (or in twenty) has V scales of 30000, the others of some 0.02, and a score of -60
    or less in every row: what follows it, and what shares its step, keep their bits."""
    r, pool, table, cu, q, heads, _, scale = _prepared(case, 2)
    n_q, n_kv, d, _ = heads
    # the first dim of every row and of K says how much a position counts
    q.reshape(len(q), n_q, d)[..., 0] = 16.0
    for b, L in enumerate(case[0]):
        ks, vs = (_scales(pool, table, b, L, w) for w in (0, 1))
        for j in range(L):
            vs[j][:] = (vs[j].astype(np.float64) / 10).astype(np.float16)
            far = j % (20 if near else 80) == 3
            slot = table[b, j // pool.page] * pool.page + j % pool.page
            for h in range(n_kv):
                codes = r.randint(0, 16, (pool.nb, 32)).astype(np.uint8)
                scales = ks[j][h].copy()
                codes[0, 0] = 8
                if far:
                    codes[0], codes[0, 0] = 8, 0
                    scales[0] = np.float16(4.0 * np.sqrt(d / 64))       # a score of 16 * -8 * 4 / 8
                pool.write(slot, h, 0, codes, scales)
            if far:
                vs[j][:] = np.float16(30000.0)
    _go(env, case, pool, table, cu, q, scale)


@pytest.mark.parametrize("case", [c for c in SHAPES if c[2] > c[3]], ids=IDS)
def test_rows_of_a_group_that_look_at_positions_of_different_sizes(env, case):
    """V's scales of alternate positions 2^20 apart; the even query heads look at the small ones alone, the odd
    ones at the large (the first two dims of K take 40 off the other kind's scores)."""
    r, pool, table, cu, q, heads, _, scale = _prepared(case, 3)
    n_q, n_kv, d, _ = heads
    q3 = q.reshape(len(q), n_q, d)
    q3[:, 0::2, :2], q3[:, 1::2, :2] = (16.0, 0.0), (0.0, 16.0)
    for b, L in enumerate(case[0]):
        ks, vs = (_scales(pool, table, b, L, w) for w in (0, 1))
        for j in range(L):
            slot = table[b, j // pool.page] * pool.page + j % pool.page
            for h in range(n_kv):
                codes, scales = np.full((pool.nb, 32), 8, np.uint8), ks[j][h].copy()
                codes[1:] = r.randint(0, 16, (pool.nb - 1, 32))
                codes[0, 1 - j % 2] = 0
                scales[0] = np.float16(2.5 * np.sqrt(d / 64))
                pool.write(slot, h, 0, codes, scales)
            vs[j][:] = (vs[j].astype(np.float64) * (2.0 ** 11 if j % 2 else 2.0 ** -9)).astype(np.float16)
    _go(env, case, pool, table, cu, q, scale)


@pytest.mark.parametrize("case", SHAPES, ids=IDS)
def test_blocks_of_q_and_k_that_differ_by_powers_of_two(env, case):
    """q of each block of dims at a size of its own, 2^-12 to 2^12, K's scales at the inverse: every block has
    the same part in the scores.  (Dims of V are left alone.)"""
    r, pool, table, cu, q, heads, _, scale = _prepared(case, 4)
    size = 2.0 ** np.linspace(-12, 12, pool.nb)[r.permutation(pool.nb)]
    for b, L in enumerate(case[0]):
        for s in _scales(pool, table, b, L, 0):
            s[:] = (s.astype(np.float64) / size).astype(np.float16)
    q.reshape(len(q), heads[0], pool.nb, 32)[:] *= size[:, None].astype(np.float32)
    _go(env, case, pool, table, cu, q, scale)


@pytest.mark.parametrize("power", [-100, 112, 118])
@pytest.mark.parametrize("case", SHAPES, ids=IDS)
def test_q_of_any_size_with_a_scale_to_match(env, case, power):
    r, pool, table, cu, q, _, _, scale = _prepared(case, 5)
    q *= np.float32(2.0 ** power)
    _go(env, case, pool, table, cu, q, scale * 2.0 ** -power)


@pytest.mark.parametrize("bits", [0x7e00, 0x7c00, 0xfc00])
@pytest.mark.parametrize("case", SHAPES, ids=IDS)
def test_value_scales_that_are_not_finite_show_at_positions_of_no_weight(env, case, bits):
    """A scale of V that is not finite, at a position whose probability underflows to 0 in every row: the rows
    that attend it have NaN in its block of dims, in the steps with masked positions as in the others."""
    g, t = env
    kv_len, fresh, n_q, n_kv, d, page, window = case
    r, pool, table, cu, q, _, _, scale = _prepared(case, 6)
    q.reshape(len(q), n_q, d)[..., 0] = 16.0
    want = np.zeros((len(q), n_q, d), bool)
    for b, L in enumerate(kv_len):
        ks, vs = (_scales(pool, table, b, L, w) for w in (0, 1))
        last = L - fresh[b] - 1                       # every row attends it, and it shares a step with later ones
        first = max(0, L - window) if window else 0   # a step that may be whole
        for j, blk in ((last, 0), (first + 40, 1)):
            slot = table[b, j // page] * page + j % page
            codes, scales = r.randint(0, 16, (pool.nb, 32)).astype(np.uint8), ks[j][n_kv - 1].copy()
            codes[0], codes[0, 0] = 8, 0
            scales[0] = np.float16(100.0 * np.sqrt(d / 64))             # a score of 16 * -8 * 100 / 8
            pool.write(slot, n_kv - 1, 0, codes, scales)
            vs[j][n_kv - 1, blk] = np.array([bits], np.uint16).view(np.float16)[0]
            want[cu[b]:cu[b + 1], (n_kv - 1) * (n_q // n_kv):, blk * 32:blk * 32 + 32] = True
    got = _attn_run(g, t, pool, table, cu, q, kv_len, n_q, n_kv, d, page, window, scale)
    assert np.array_equal(np.isnan(got).reshape(want.shape), want)
