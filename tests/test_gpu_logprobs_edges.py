"""gem_logprobs at the edges of its call: infinite tokens, the least and largest scales, arguments it has no use for."""
import numpy as np
import pytest

from oracle import fp8
from test_gpu_logprobs import _check, _logits, _run, env  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_workspace_may_be_given(env):  # noqa: F811
    """Calls that pass one, as the other calls with scratch take it, give what calls without one give."""
    gem, t = env
    y = _logits(5, 9001, 1)
    scratch = t.empty(1 << 20, dtype=t.uint8, device="cuda")
    scratch.fill_(0xA5)
    a, b = _run(env, y, [0, 1, 2, 3, 9000], 7), _run(env, y, [0, 1, 2, 3, 9000], 7, workspace=scratch)
    assert all(np.array_equal(a[n], b[n]) for n in a)
    assert bool((scratch == 0xA5).all())
    for bad in (scratch.float(), scratch.cpu(), scratch[::2]):
        with pytest.raises(ValueError):
            _run(env, y, [0, 1, 2, 3, 4], 7, workspace=bad)


@pytest.mark.parametrize("T", [1, 3, 6, 400])
@pytest.mark.parametrize("N", [5000, 30000, 100001])
def test_rank_of_one_of_several_infinite_tokens(env, T, N):  # noqa: F811
    """Equal entries go by lowest index, +inf among them, wherever in the row they lie."""
    T = T if N < 100000 else min(T, 40)
    y = _logits(T, N, 11)
    at = [5, 17, N // 7, N // 2, N // 2 + 3, N - 2]
    y[:, at] = np.inf
    y[:, N // 3] = np.nan
    for q in range(0, 6, 1 if T < 10 else 3):
        tokens = [at[(q + t) % 6] for t in range(T)]
        got = _run(env, y, tokens, 8)
        assert got["rank"].tolist() == [1 + (q + t) % 6 for t in range(T)]
        assert (got["idx"][:, :6] == at).all()
        assert np.isnan(got["logp"]).all() and np.isnan(got["val"]).all() and np.isnan(got["entropy"]).all()
    y[:, N // 3], y[:, at[1:]] = 0, 0
    _check(_run(env, y, [N // 3] * T, 3), y, [N // 3] * T, 3)


@pytest.mark.parametrize("scale", [2.0 ** 100, 1e20, 0.25, 1e-25, 2.0 ** -100])
@pytest.mark.parametrize("T,N", [(3, 6001), (9, 30000)])
def test_scales_and_logits_over_their_whole_range(env, T, N, scale):  # noqa: F811
    """Differences of logits that pass the type's largest value before they are scaled, and scales at their limits."""
    y = _logits(T, N, 12)
    y[1:] = np.clip(y[1:].astype(np.float64) * 2e38, -3.4e38, 3.4e38).astype(np.float32)
    y[2, ::3] = -np.inf
    y[2, 4::3] = -3.4028235e38
    tokens = [4 + 3 * t for t in range(T)]
    got, want = _run(env, y, tokens, 12, scale), fp8.scores(y, tokens, 12, scale)
    assert np.array_equal(got["rank"], want["rank"]) and np.array_equal(got["idx"], want["idx"])
    # one entry has all the weight (a row of ordinary logits: all of them with the small scales, and as little with the large
    # ones), so that log s is off by 2^-24 (128 + 4 + 4 spread) and the values by two roundings more
    lse = 2.0 ** -24 * (128 + 4 + 4 * want["spread"])
    for name, n in (("logp", lse), ("val", lse[:, None])):
        with np.errstate(over="ignore"):
            w = want[name].astype(np.float32).astype(np.float64)  # past the largest number: infinite
        fine = np.isfinite(w)
        assert np.array_equal(got[name][~fine], w[~fine])
        assert np.all(np.abs(np.where(fine, got[name] - np.where(fine, w, 0), 0)) <= n + 2.0 ** -22 * np.abs(np.where(fine, w, 0)))
    assert np.all(np.abs(got["entropy"] - want["entropy"]) <= 2.0 ** -24 * (128 + 4) * (2 + 4 * want["spread"] + want["entropy"]))


def test_scales_out_of_range_are_refused(env):  # noqa: F811
    gem, t = env
    y, lp = t.zeros(2, 100, device="cuda"), t.zeros(2, device="cuda")
    tok = t.zeros(2, dtype=t.int32, device="cuda")
    for scale in (2.0 ** 101, 3e38, 2.0 ** -101, 1e-40):
        with pytest.raises(gem.GemError):
            gem.logprobs(y, tok, lp, scale=scale)


def test_one_entry_far_above_very_many(env):  # noqa: F811
    """Sums of 2^29 and more that a far larger entry takes the weight from."""
    gem, t = env
    N = 1 << 30
    y = t.zeros(1, N, device="cuda")
    y[0, N - 9] = 1e38
    for rows in (y, t.cat([y] * 5)):
        T = rows.shape[0]
        tokens = t.full((T,), N - 9, dtype=t.int32, device="cuda")
        logp, ent, rank = t.full((T,), -7.0, device="cuda"), t.full((T,), -7.0, device="cuda"), t.zeros(T, dtype=t.int32, device="cuda")
        gem.logprobs(rows, tokens, logp, ent, rank)
        assert not logp.any() and not ent.any() and bool((rank == 1).all())


@pytest.mark.parametrize("N,k", [(32000, 5), (151669, 20)])
def test_little_is_added_to_the_last_rounding(env, N, k):  # noqa: F811
    """In the mean square over many rows: one rounding of the result (a unit of its last place / sqrt 12), and 2^-23 for
    the sum, whose terms' errors of up to 2^-22 are averaged."""
    y = _logits(300, N, 13)
    tokens = np.random.RandomState(14).randint(0, N, 300)
    got, want = _run(env, y, tokens, k), fp8.scores(y, tokens, k)
    for name in ("logp", "val"):
        last = np.spacing(np.abs(want[name]).astype(np.float32)).astype(np.float64)
        assert np.mean((got[name] - want[name]) ** 2) <= np.mean(last ** 2) / 12 + 2.0 ** -46, name
