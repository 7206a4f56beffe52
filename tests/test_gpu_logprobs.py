"""gem_logprobs on the GPU against the 64-bit oracle."""
import numpy as np
import pytest

from oracle import fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import q4_gemv_gqa_gb300 as gem
    torch.cuda.set_device(0)
    return gem, torch


def _run(env, y, tokens, k, scale=1.0, **kw):
    gem, t = env
    T = y.shape[0]
    f = lambda *s: t.full(s, -7.0, device="cuda")  # noqa: E731
    i = lambda *s: t.full(s, -7, dtype=t.int32, device="cuda")  # noqa: E731
    d = dict(logp=f(T), entropy=f(T), rank=i(T), idx=i(T, k), val=f(T, k))
    yd = y if isinstance(y, t.Tensor) else t.from_numpy(y).cuda()
    gem.logprobs(yd, t.tensor(np.asarray(tokens), dtype=t.int32, device="cuda"), d["logp"], d["entropy"], d["rank"],
                 d["idx"] if k else None, d["val"] if k else None, scale=scale, **kw)
    return {n: v.cpu().numpy() for n, v in d.items()}


def _check(got, y, tokens, k, scale=1.0, dup=None):
    """Indices and ranks equal.  Values: e^d is off by 2^-22 and by d's own two roundings times |d|, a thread adds
    at most 128 numbers one after the other; log p adds its own roundings."""
    want = fp8.scores(y, tokens, k, scale)
    assert np.array_equal(got["rank"], want["rank"]), (got["rank"], want["rank"])
    assert np.array_equal(got["idx"], want["idx"])
    lse = 2.0 ** -24 * (128 + 4 + 4 * want["spread"])
    for name, w, n in (("logp", want["logp"], lse), ("val", want["val"], lse[:, None]),
                       ("entropy", want["entropy"], 2.0 ** -24 * (128 + 4) * (2 + 4 * want["spread"] + want["entropy"]))):
        v = got[name].astype(np.float64)
        assert np.array_equal(np.isfinite(v), np.isfinite(w)) and np.array_equal(np.isnan(v), np.isnan(w)), name
        fine = np.isfinite(w)
        tol = np.broadcast_to(n, w.shape) + 2.0 ** -22 * np.abs(np.where(fine, w, 0))
        assert np.all((np.abs(np.where(fine, v - np.where(fine, w, 0), 0)) <= np.where(fine, tol, 1))), (name, np.max(np.abs(v - w)[fine]))


def _logits(T, N, seed, coarse=False, masked=0.0):
    r = np.random.RandomState(seed)
    y = (r.randn(T, N) * r.uniform(0.2, 5, (T, 1))).astype(np.float32)
    if coarse:
        y = (np.round(y * 4) / 4).astype(np.float32)     # many equal values
    if masked:
        y[r.rand(T, N) < masked] = -np.inf
        y[:, N // 2] = np.where(np.isfinite(y[:, N // 2]), y[:, N // 2], 0)
    return y


@pytest.mark.parametrize("N", [1, 2, 31, 33, 257, 1000, 2047, 2049, 4096, 8191, 32003, 65536, 151669, 262144, 262145])
@pytest.mark.parametrize("T,k", [(1, 0), (1, 64), (3, 5), (2, 1), (160, 20)])
def test_scores(env, N, T, k):
    if T == 160 and N > 40000:
        T = 5
    k = min(k, N)
    y = _logits(T, N, N + T, coarse=T == 3)
    tokens = np.random.RandomState(T).randint(0, N, T)
    tokens[0] = N - 1
    if T > 1:
        tokens[1] = int(fp8.order(y[1])[0])
    _check(_run(env, y, tokens, k), y, tokens, k)


@pytest.mark.parametrize("N", [40, 5000, 100000])
def test_masked_rows_and_ties(env, N):
    y = _logits(6, N, 1, coarse=True, masked=0.7)
    y[1] = 2.5                                          # all equal: the list is 0, 1, 2, ..
    y[2] = -3.4028235e38                                # masked by the type's lowest value, one left
    y[2, N - 1] = 1.0
    y[3] = -np.inf                                      # fewer left than the list is long
    y[3, [0, N // 3, N - 2]] = [1.0, 2.0, 2.0]
    y[4] = -3.4028235e38
    y[5] = np.where(np.arange(N) % 2, np.float32(0.0), np.float32(-0.0))
    tokens = [N // 2, N - 1, 3, N // 3, N - 1, 7]
    _check(_run(env, y, tokens, 33), y, tokens, 33)


@pytest.mark.parametrize("left", [1, 3, 19, 20, 21, 200])
@pytest.mark.parametrize("N", [300, 4099, 151669])
def test_few_entries_that_are_not_banned(env, left, N):
    """Grammars leave a handful of tokens: the list goes on with banned ones, by index."""
    r = np.random.RandomState(left)
    y = np.full((70, N), -np.inf, np.float32)
    tokens = np.zeros(70, np.int64)
    for t in range(70):
        at = r.choice(N, min(left, N), replace=False) if t % 3 else np.arange(N - min(left, N), N)
        y[t, at] = r.randn(at.size).round(1)
        tokens[t] = at[0] if t % 2 else r.randint(N)
    y[5, ::2] = np.nan                                   # and NaN behind them
    y[6, 1:70] = np.nan
    for k in (1, 20, 64):
        _check(_run(env, y, tokens, k), y, tokens, k)


def test_sorted_rows(env):
    """The list's order in the row: the largest first, last, or in the threads' own strides."""
    N = 70000
    up = np.arange(N, dtype=np.float32) / 7000
    rows = [up, up[::-1], np.roll(up, N // 2), up.reshape(-1, 7).T.reshape(-1), np.resize(up[::1000], N)]
    for stride in (32, 128, 256, 512, 1024, 2048):
        z = np.zeros(N, np.float32)
        z[5::stride] = 3 + np.arange(z[5::stride].size, dtype=np.float32) / 100
        rows.append(z)
    y = np.ascontiguousarray(np.stack(rows))
    tokens = np.arange(len(rows)) * 6000 + 5
    for k in (1, 20, 64):
        _check(_run(env, y, tokens, k), y, tokens, k)


def test_not_finite_rows_keep_to_themselves(env):
    for N in (100, 30000):
        y = _logits(7, N, 2)
        y[1, 60], y[2, 99], y[3], y[5, 3] = np.nan, np.inf, -np.inf, np.nan
        y[5, 50:90] = -np.nan
        tokens = [0, 1, 2, 3, 4, 60, 6]
        got = _run(env, y, tokens, 9)
        for n in ("logp", "entropy", "val"):
            assert np.isnan(got[n][[1, 2, 3, 5]]).all() and np.isfinite(got[n][[0, 4, 6]]).all()
        _check(got, y, tokens, 9)


def test_rows_of_nan(env):
    y = np.full((2, 3000), np.nan, np.float32)
    y[1, 2500:2503] = [1, -np.inf, 2]
    got = _run(env, y, [5, 2501], 6)
    assert got["idx"].tolist() == [[0, 1, 2, 3, 4, 5], [2502, 2500, 2501, 0, 1, 2]] and got["rank"].tolist() == [6, 3]


def test_tokens_that_are_not_there(env):
    gem, t = env
    y = _logits(5, 777, 3)
    gem.device_status(reset=True)
    got = _run(env, y, [-1, 3, 777, -2, 2 ** 31 - 1], 2)
    assert gem.device_status(reset=True) == gem.DEVFLAG_POS_RANGE
    assert got["logp"][0] == 0 and got["rank"][0] == 0 and np.isnan(got["logp"][[2, 3, 4]]).all() and not got["rank"][[2, 3, 4]].any()
    want = fp8.scores(y, [-1, 3, 777, -2, 5000], 2)
    assert np.array_equal(got["idx"], want["idx"]) and np.allclose(got["entropy"], want["entropy"], atol=1e-5)
    assert got["rank"][1] == want["rank"][1]
    status = t.zeros(1, dtype=t.int32, device="cuda")
    _run(env, y, [0, 1, 2, 3, -9], 0, status=status)
    assert int(status) == gem.DEVFLAG_POS_RANGE and gem.device_status() == 0


def test_scale_and_large_logits(env):
    y = _logits(4, 5000, 4)
    tokens = [1, 2, 3, 4]
    for scale in (0.25, 1.7, 1e-3, 40.0):
        _check(_run(env, y, tokens, 8, scale), y, tokens, 8, scale)
    big = (y * 1e30).astype(np.float32)                 # one entry has all the weight
    got = _run(env, big, tokens, 2)
    want = fp8.scores(big, tokens, 2)
    assert np.array_equal(got["idx"], want["idx"]) and np.array_equal(got["rank"], want["rank"])
    assert np.all(got["entropy"] == 0) and np.all(got["val"][:, 0] == 0)
    assert np.allclose(got["logp"], want["logp"], rtol=1e-6)


def test_outputs_that_are_left_out(env):
    gem, t = env
    y = _logits(3, 9000, 5)
    yd = t.from_numpy(y).cuda()
    tok = t.tensor([1, 2, 3], dtype=t.int32, device="cuda")
    want = fp8.scores(y, [1, 2, 3], 4)
    ent, rank = t.zeros(3, device="cuda"), t.zeros(3, dtype=t.int32, device="cuda")
    gem.logprobs(yd, None, None, entropy=ent)
    assert np.allclose(ent.cpu().numpy(), want["entropy"], atol=1e-5)
    gem.logprobs(yd, tok, None, rank=rank)
    assert np.array_equal(rank.cpu().numpy(), want["rank"])
    idx, val = t.zeros(3, 4, dtype=t.int32, device="cuda"), t.zeros(3, 4, device="cuda")
    gem.logprobs(yd, None, None, idx=idx, val=val)
    assert np.array_equal(idx.cpu().numpy(), want["idx"]) and np.allclose(val.cpu().numpy(), want["val"], atol=1e-5)
    logp = t.zeros(3, device="cuda")
    gem.logprobs(yd, tok, logp)
    assert np.allclose(logp.cpu().numpy(), want["logp"], atol=1e-5)
    with pytest.raises(gem.GemError):
        gem.logprobs(yd, None, logp)
    with pytest.raises(ValueError):
        gem.logprobs(yd, tok, logp, idx=idx)
    with pytest.raises(ValueError):
        gem.logprobs(yd, tok.long(), logp)


@pytest.mark.parametrize("off,pad", [(0, 8), (1, 6), (2, 0), (3, 1)])
def test_strides_and_alignment(env, off, pad):
    """Columns of a padded vocabulary: what lies behind a row's entries is not read as one."""
    gem, t = env
    y = _logits(4, 6001, 6)
    wide = t.full((4, off + 6001 + pad), 1e30, device="cuda")
    wide[:, off:off + 6001] = t.from_numpy(y).cuda()
    _check(_run(env, wide[:, off:off + 6001], [0, 6000, 5, 6], 12), y, [0, 6000, 5, 6], 12)


def test_row_offsets_past_32_bits(env):
    gem, t = env
    ld = 1 << 30
    y = _logits(4, 3001, 7)
    far = t.empty(3 * ld + 3001, device="cuda").as_strided((4, 3001), (ld, 1))
    far.copy_(t.from_numpy(y).cuda())
    _check(_run(env, far, [0, 1, 2, 3], 7), y, [0, 1, 2, 3], 7)


def test_many_rows(env):
    """More rows than a grid holds at once."""
    y = _logits(5000, 700, 8)
    tokens = np.random.RandomState(1).randint(0, 700, 5000)
    _check(_run(env, y, tokens, 3), y, tokens, 3)


def test_no_rows(env):
    gem, t = env
    _run(env, np.zeros((0, 10), np.float32), np.zeros(0, np.int32), 2)
    y = _logits(3, 50, 1)
    got = _run(env, y, [1, 2, 3], 50)                    # the list is the whole row
    _check(got, y, [1, 2, 3], 50)


def test_agrees_with_top_k_and_argmax(env):
    gem, t = env
    y = t.from_numpy(_logits(4, 50000, 10, coarse=True)).cuda()
    got = _run(env, y, [0, 0, 0, 0], 30)
    idx, val = t.zeros(4, 30, dtype=t.int32, device="cuda"), t.zeros(4, 30, device="cuda")
    gem.topk(y, 30, idx, val)
    am = t.zeros(4, dtype=t.int32, device="cuda")
    gem.argmax(y, am)
    assert np.array_equal(got["idx"], idx.cpu().numpy()) and np.array_equal(got["idx"][:, 0], am.cpu().numpy())
