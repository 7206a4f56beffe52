"""The 8-bit floating-point path on the GPU against the 64-bit oracle: gem_rmsnorm_fp8, gem_quant_fp8 and
gem_fp8_gemm, alone, chained as in a layer, and at their calls' edges."""
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


def _dev(t, a):
    return t.from_numpy(np.ascontiguousarray(a)).cuda()


def _u8(t):
    return t.view(__import__("torch").uint8).cpu().numpy()


def _check_rows(codes, scales, y, what=""):
    """Codes and scales are whole answers: equal to the oracle's."""
    c, s = fp8.quantise(y)
    got_c, got_s = _u8(codes), scales.cpu().numpy()
    assert np.array_equal(got_s, s, equal_nan=True), (what, np.argwhere(got_s != s)[:5])
    # zeros of either sign stand for the same value
    same = (got_c == c) | ((got_c & 127 == 0) & (c & 127 == 0))
    assert same.all(), (what, np.argwhere(~same)[:5], got_c[~same][:5], c[~same][:5])


def _rows(t, T, H):
    return t.full((T, H), 0xA5, dtype=t.uint8, device="cuda"), t.full((T, -(-H // 128)), -7.0, device="cuda")


# ---- rows in 8 bits ------------------------------------------------------------------------------


@pytest.mark.parametrize("T,H", [(1, 16), (1, 128), (3, 144), (2, 1008), (1, 2048), (8, 2560), (5, 4096), (700, 2560), (310, 5376),
                                 (2, 8192), (3, 8208), (2, 16384), (2, 32768), (1200, 256)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(env, T, H, residual):
    gem, t = env
    r = np.random.RandomState(T * 7 + H)
    x = (r.randn(T, H) * np.exp(r.randn(H))).astype(np.float32)
    res = (3 * r.randn(T, H)).astype(np.float32) if residual else None
    gamma = None if T == 5 else (1 + 0.1 * r.randn(H)).astype(np.float32)
    codes, scales = _rows(t, T, H)
    out = t.zeros(T, H, device="cuda")
    gem.rmsnorm_fp8(_dev(t, x), None if gamma is None else _dev(t, gamma), 1e-6, codes, scales,
                    residual=None if res is None else _dev(t, res), out=out)
    h, y = fp8.rmsnorm(x, res, gamma, 1e-6)
    assert np.array_equal(out.cpu().numpy(), h)
    _check_rows(codes, scales, y)


def test_norm_rows_of_every_size_at_once_and_in_place(env):
    gem, t = env
    r = np.random.RandomState(0)
    x = (r.randn(64, 640) * np.exp2(r.randint(-40, 40, (64, 1)))).astype(np.float32)
    x[5] = 0
    res = r.randn(64, 640).astype(np.float32)
    gamma = (1 + 0.1 * r.randn(640)).astype(np.float32)
    gamma[128:256] = 0                                 # a block of zeros
    gamma[256:384] *= np.float32(2.0 ** -103)          # blocks on either side of the least scale
    h, y = fp8.rmsnorm(x, res, gamma, 1e-6)
    for alias in ("x", "residual"):
        a, b = _dev(t, x), _dev(t, res)
        codes, scales = _rows(t, 64, 640)
        gem.rmsnorm_fp8(a, _dev(t, gamma), 1e-6, codes, scales, residual=b, out=a if alias == "x" else b)
        assert np.array_equal((a if alias == "x" else b).cpu().numpy(), h)
        _check_rows(codes, scales, y, alias)


def test_norm_not_finite_rows_keep_to_themselves(env):
    gem, t = env
    x = np.random.RandomState(1).randn(6, 512).astype(np.float32)
    x[1, 300], x[2, 5], x[4, 511] = np.nan, np.inf, 3e38
    codes, scales = _rows(t, 6, 512)
    gem.rmsnorm_fp8(_dev(t, x), None, 1e-6, codes, scales)
    s = scales.cpu().numpy()
    for bad in (1, 2, 4):
        assert np.isnan(s[bad]).all() and not _u8(codes)[bad].any()
    _check_rows(codes[[0, 3, 5]], scales[[0, 3, 5]], fp8.rmsnorm(x[[0, 3, 5]], None, None, 1e-6)[1])


@pytest.mark.parametrize("H", [256, 640])
def test_norm_strides(env, H):
    """Columns of wider tensors; what lies beside them is left alone."""
    gem, t = env
    r = np.random.RandomState(2)
    wide = r.randn(9, H + 64).astype(np.float32)
    x = _dev(t, wide)[:, 32:32 + H]
    cw = t.full((9, H + 48), 0x5A, dtype=t.uint8, device="cuda")
    sw = t.full((9, H // 128 + 3), -7.0, device="cuda")
    ow = t.full((9, H + 8), -7.0, device="cuda")
    gem.rmsnorm_fp8(x, None, 1e-6, cw[:, 16:16 + H], sw[:, 1:1 + H // 128], out=ow[:, 4:4 + H])
    h, y = fp8.rmsnorm(wide[:, 32:32 + H], None, None, 1e-6)
    _check_rows(cw[:, 16:16 + H].contiguous(), sw[:, 1:1 + H // 128], y)
    assert np.array_equal(ow[:, 4:4 + H].cpu().numpy(), h)
    assert (cw[:, :16] == 0x5A).all() and (cw[:, 16 + H:] == 0x5A).all()
    assert (sw[:, 0] == -7).all() and (sw[:, 1 + H // 128:] == -7).all() and (ow[:, :4] == -7).all() and (ow[:, 4 + H:] == -7).all()


@pytest.mark.parametrize("T,H", [(1, 16), (1, 6144), (3, 1200), (61, 9728), (2, 21504), (130, 2064)])
@pytest.mark.parametrize("gate", ["none", "silu", "gelu"])
def test_quant(env, T, H, gate):
    gem, t = env
    r = np.random.RandomState(T + H)
    both = (r.randn(T, 2 * H) * np.repeat([2.0, 1.0], H) * np.exp(0.7 * r.randn(2 * H))).astype(np.float32)
    d = _dev(t, both)
    codes, scales = _rows(t, T, H)
    if gate == "none":
        gem.quant_fp8(d[:, H:], codes, scales)
        y = both[:, H:].astype(np.float64)
    else:
        act = 0 if gate == "silu" else 1
        gem.quant_fp8(d[:, :H], codes, scales, up=d[:, H:], act=act)
        y = fp8.gated(both[:, :H], both[:, H:], act)
    _check_rows(codes, scales, y, gate)


def test_quant_every_border(env):
    """Values on the borders of codes and scales, and next to them, at many scales."""
    gem, t = env
    mids = np.concatenate([fp8._MID, fp8._GRID[1:], [448.0]]).astype(np.float32)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(1e9))])
    near = near[near <= 448]
    rows = np.zeros((60, 1024), np.float32)
    rows[:, :near.size] = near
    rows[:, 127::128] = 448                            # every block at the same scale
    rows *= np.where(np.arange(1024) % 2, -1, 1)
    rows *= np.exp2(np.arange(-90, 90, 3, dtype=np.float64)).astype(np.float32)[:, None]
    codes, scales = _rows(t, 60, 1024)
    gem.quant_fp8(_dev(t, rows), codes, scales)
    _check_rows(codes, scales, rows.astype(np.float64))
    tops = np.float32([448, np.nextafter(np.float32(448), np.float32(449)), 224, np.nextafter(np.float32(224), np.float32(225)), 2.0 ** -100,
                       np.nextafter(np.float32(2.0 ** -100), np.float32(0)), 1e-40, 0, 3.4e38, 1])
    rows = np.zeros((tops.size, 128), np.float32)
    rows[:, 3], rows[:, 70] = tops, -tops / 3
    codes, scales = _rows(t, tops.size, 128)
    gem.quant_fp8(_dev(t, rows), codes, scales)
    _check_rows(codes, scales, rows.astype(np.float64))


@pytest.mark.parametrize("act", [0, 1])
def test_quant_gate_over_its_whole_range(env, act):
    gem, t = env
    x = np.linspace(-120, 120, 128 * 512).astype(np.float32).reshape(512, 128)
    x[0, :8] = [0.0, -0.0, 1e-30, -1e-30, 1e-40, 1e15, -1e15, 3e38]
    up = np.random.RandomState(5).randn(512, 128).astype(np.float32)
    up[0, :8] = 1
    x[1], up[1] = -80.0, 2.0 ** 90                    # a tiny gate times large values
    codes, scales = _rows(t, 512, 128)
    gem.quant_fp8(_dev(t, x), codes, scales, up=_dev(t, up), act=act)
    _check_rows(codes, scales, fp8.gated(x, up, act))


def test_quant_borders_of_the_gated_value_are_decided_exactly(env):
    """Values of up chosen so that the product falls within a few units of fp32's last place of a border: the
    decision has to be the 64-bit one."""
    gem, t = env
    r = np.random.RandomState(6)
    x = r.uniform(0.5, 4, (400, 256)).astype(np.float32)
    gate = fp8.gated(x, np.ones_like(x), 0)
    want = r.choice(fp8._MID[60:], (400, 256))         # borders, at scale 1
    up = (want / gate).astype(np.float32)
    up = (up.view(np.int32) + r.randint(-1, 2, up.shape)).astype(np.int32).view(np.float32)
    x[:, ::128], up[:, ::128] = 30.0, np.float32(440 / 30)   # the block's largest: scale 1
    y = fp8.gated(x, up, 0)
    codes, scales = _rows(t, 400, 256)
    gem.quant_fp8(_dev(t, x), codes, scales, up=_dev(t, up))
    _check_rows(codes, scales, y)


def test_quant_not_finite_blocks(env):
    gem, t = env
    x = np.random.RandomState(7).randn(4, 384).astype(np.float32)
    x[0, 130], x[1, 0], x[2, 383] = np.nan, np.inf, -np.inf
    codes, scales = _rows(t, 4, 384)
    gem.quant_fp8(_dev(t, x), codes, scales)
    _check_rows(codes, scales, x.astype(np.float64))
    up = np.ones_like(x)
    up[3, 200] = np.nan
    x[2, 383] = -200.0
    codes, scales = _rows(t, 4, 384)
    gem.quant_fp8(_dev(t, x), codes, scales, up=_dev(t, up))
    bad = np.isnan(scales.cpu().numpy())
    assert bad.tolist() == [[False, True, False], [True, False, False], [False] * 3, [False, True, False]]


def test_row_offsets_past_32_bits(env):
    gem, t = env
    H, T = 128, 5
    ld = 1 << 30
    x = t.zeros((T - 1) * ld + H, device="cuda").as_strided((T, H), (ld, 1))
    rows = np.random.RandomState(8).randn(T, H).astype(np.float32)
    x.copy_(_dev(t, rows))
    codes = t.zeros((T - 1) * ld + H, dtype=t.uint8, device="cuda").as_strided((T, H), (ld, 1))
    scales = t.zeros(T, 1, device="cuda")
    gem.rmsnorm_fp8(x, None, 1e-6, codes, scales)
    _check_rows(codes.contiguous(), scales, fp8.rmsnorm(rows, None, None, 1e-6)[1])
    gem.quant_fp8(x, codes, scales, up=x)
    _check_rows(codes.contiguous(), scales, fp8.gated(rows, rows, 0))


# ---- the product -----------------------------------------------------------------------------------


def _operands(M, K, N, seed=0):
    r = np.random.RandomState(seed + M + 3 * K + 7 * N)
    W = fp8.encode(np.clip(r.randn(N, K) * 60, -448, 448))
    ws = np.exp(r.randn(-(-N // 128), -(-K // 128)) - 4).astype(np.float32)
    x, xs = fp8.quantise(r.randn(M, K) * np.exp(r.randn(K)))
    return W, ws, x, xs


# A block's 128 products are exact in fp32 and summed in four tensor instructions of 32, each of whose terms may
# be cut at 2^-24 of the largest: 4 * 33 cuts.  The blocks' sums are scaled (two roundings) and added in fp32.
def _tol(K, most):
    return (132 + -(-K // 128) + 3) * 2.0 ** -24 * most


def _product(env, W, ws, x, xs, res=None, **kw):
    gem, t = env
    M, N = x.shape[0], W.shape[0]
    y = t.full((M, N), -7.0, device="cuda")
    gem.fp8_gemm(_dev(t, W), _dev(t, ws), _dev(t, x), _dev(t, xs), y, residual=None if res is None else _dev(t, res), **kw)
    return y


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 61, 64, 65, 96, 127, 128, 129, 200, 255, 256, 257, 300, 513])
@pytest.mark.parametrize("K,N", [(256, 512), (1008, 1201), (2048, 384)])
def test_gemm(env, M, K, N):
    W, ws, x, xs = _operands(M, K, N)
    y = _product(env, W, ws, x, xs)
    want, most = fp8.gemm(W, ws, x, xs)
    assert np.all(np.abs(y.cpu().numpy() - want) <= _tol(K, most))
    assert env[0].device_status() == 0


@pytest.mark.parametrize("M,K,N", [(1, 16, 1), (1, 16, 8), (3, 32, 5), (5, 144, 130), (64, 128, 127), (130, 112, 129), (1, 128, 4099), (1, 5376, 1000),
                                   (70, 640, 2), (258, 16, 300), (1, 21504, 136), (40, 9728, 200), (140, 6144, 96)])
@pytest.mark.parametrize("residual", [False, True])
def test_gemm_odd_sizes(env, M, K, N, residual):
    W, ws, x, xs = _operands(M, K, N, 1)
    res = np.random.RandomState(4).randn(M, N).astype(np.float32) if residual else None
    y = _product(env, W, ws, x, xs, res)
    want, most = fp8.gemm(W, ws, x, xs, res)
    assert np.all(np.abs(y.cpu().numpy() - want) <= _tol(K, most))


@pytest.mark.parametrize("M,K,N", [(8, 5376, 21504), (61, 21504, 5376), (300, 2560, 19456), (2000, 2048, 4096), (1, 2048, 4096), (1000, 1008, 1201),
                                   (4000, 256, 8192), (8192, 512, 512), (97, 9728, 2560)])
def test_gemm_large(env, M, K, N):
    """Against a 64-bit product on the GPU; the error of the whole result stays near fp32's rounding."""
    gem, t = env
    g = t.Generator(device="cuda").manual_seed(M)
    f8 = t.float8_e4m3fn
    w = (t.randn(N, K, generator=g, device="cuda") * 60).clamp_(-448, 448).to(f8)
    x = (t.randn(M, K, generator=g, device="cuda") * 100).clamp_(-448, 448).to(f8)
    ws = t.exp(t.randn(-(-N // 128), -(-K // 128), generator=g, device="cuda") - 4)
    xs = t.exp(t.randn(M, -(-K // 128), generator=g, device="cuda") - 4)
    y = t.full((M, N), -7.0, device="cuda")
    gem.fp8_gemm(w, ws, x, xs, y)
    X = x.double() * xs.double().repeat_interleave(128, 1)[:, :K]
    V = w.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    want = X @ V.T
    most = X.abs_() @ V.abs_().T
    off = (y.double() - want).abs_()
    assert bool((off <= _tol(K, most)).all())
    # the bound above for every result, and for all of them together a tenth of it: roundings do not all add up
    assert float(off.norm() / most.norm()) <= _tol(K, 1.0) / 10


def test_gemm_shows_every_product(env):
    """One code set per row and column: a result is one product, exactly, so that a wrong index shows."""
    M, K, N = 70, 272, 300
    r = np.random.RandomState(9)
    x, W = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
    k = r.permutation(np.resize(np.arange(K), max(M, N)))
    x[np.arange(M), k[:M]] = r.choice(126, M) + 1
    W[:] = r.choice(126, (N, K)) + 1
    ws, xs = np.exp2(r.randint(-9, 9, (3, 3))).astype(np.float32), np.exp2(r.randint(-9, 9, (M, 3))).astype(np.float32)
    y = _product(env, W, ws, x, xs)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), fp8.gemm(W, ws, x, xs)[0])


@pytest.mark.parametrize("K", [640, 1024, 1536, 2560, 3200, 5376, 9728])
@pytest.mark.parametrize("M", [1, 16, 31, 64, 127, 130, 300, 513])
def test_gemm_clusters_of_every_size(env, M, K):
    """Few rows of W and long ones: clusters of one to eight CTAs, whose parts lie where their operands were."""
    for N in (40, 200, 2560):
        W, ws, x, xs = _operands(M, K, N, M + K)
        want, most = fp8.gemm(W, ws, x, xs)
        got = [_product(env, W, ws, x, xs).cpu().numpy() for _ in range(3)]
        assert np.all(np.abs(got[0] - want) <= _tol(K, most))
        assert all(np.array_equal(g, got[0]) for g in got)


@pytest.mark.parametrize("M", [3, 50, 100, 260])
def test_gemm_strides_and_residual_in_place(env, M):
    gem, t = env
    K, N = 400, 260
    W, ws, x, xs = _operands(M, K, N, 2)
    xw = t.full((M, K + 48), 0x7F, dtype=t.uint8, device="cuda")      # NaN beside the row
    xw[:, 16:16 + K] = _dev(t, x)
    sw = t.full((M, 9), float("nan"), device="cuda")
    sw[:, 2:6] = _dev(t, xs)
    for off, pad in ((0, 4), (1, 3), (4, 8)):                        # aligned and unaligned rows of y
        res = np.random.RandomState(M).randn(M, N).astype(np.float32)
        yw = t.full((M, off + N + pad), -7.0, device="cuda")
        y = yw[:, off:off + N]
        y.copy_(_dev(t, res))
        gem.fp8_gemm(_dev(t, W), _dev(t, ws), xw[:, 16:16 + K], sw[:, 2:6], y, residual=y)
        want, most = fp8.gemm(W, ws, x, xs, res)
        assert np.all(np.abs(y.cpu().numpy() - want) <= _tol(K, most))
        assert (yw[:, :off] == -7).all() and (yw[:, off + N:] == -7).all()


@pytest.mark.parametrize("M", [4, 40, 100, 300])
def test_gemm_not_finite_stays_where_it_belongs(env, M):
    K, N = 384, 300
    W, ws, x, xs = _operands(M, K, N, 3)
    x[1, 200], xs[2, 1], W[5, 300], ws[2, 0] = 0x7F, np.nan, 0xFF, np.inf
    y = _product(env, W, ws, x, xs).cpu().numpy()
    bad = np.zeros((M, N), bool)
    bad[1] = bad[2] = True
    bad[:, 5] = bad[:, 256:] = True
    assert not np.isfinite(y[bad]).any() and np.isfinite(y[~bad]).all()
    W, ws, x, xs = _operands(M, K, N, 3)
    want, most = fp8.gemm(W, ws, x, xs)
    keep = np.ix_([0] + list(range(3, M)), [n for n in range(256) if n != 5])
    assert np.all((np.abs(y - want) <= _tol(K, most))[keep])


def test_gemm_same_inputs_same_bits(env):
    for M in (8, 100, 300):
        W, ws, x, xs = _operands(M, 1024, 700, 5)
        a, b = _product(env, W, ws, x, xs), _product(env, W, ws, x, xs)
        assert env[1].equal(a, b)


def test_gemm_offsets_past_32_bits(env):
    gem, t = env
    M, K, N = 70000, 16, 32768                          # 2.3e9 results
    g = t.Generator(device="cuda").manual_seed(0)
    w = t.randn(N, K, generator=g, device="cuda").to(t.float8_e4m3fn)
    x = t.randn(M, K, generator=g, device="cuda").to(t.float8_e4m3fn)
    ws, xs = t.rand(N // 128, 1, generator=g, device="cuda"), t.rand(M, 1, generator=g, device="cuda")
    y = t.empty(M, N, device="cuda")
    gem.fp8_gemm(w, ws, x, xs, y)
    for lo in (0, 65530, M - 64):
        X, V = x[lo:lo + 64].double() * xs[lo:lo + 64].double(), w.double() * ws.double().repeat_interleave(128, 0)
        assert bool(((y[lo:lo + 64].double() - X @ V.T).abs() <= _tol(K, X.abs() @ V.abs().T)).all())
    del y
    ld = 1 << 30                                        # a few rows, far apart
    y = t.empty(3 * ld + 64, device="cuda").as_strided((4, 64), (ld, 1))
    xx = t.empty(3 * ld + 16, dtype=t.uint8, device="cuda").as_strided((4, 16), (ld, 1))
    xx.copy_(x[:4].view(t.uint8))
    gem.fp8_gemm(w[:64], ws[:1], xx, xs[:4], y)
    X, V = x[:4].double() * xs[:4].double(), w[:64].double() * ws[0].double()
    assert bool(((y.double() - X @ V.T).abs() <= _tol(K, X.abs() @ V.abs().T)).all())


def test_binding_refusals(env):
    gem, t = env
    x, c, s = t.zeros(4, 256, device="cuda"), t.zeros(4, 256, dtype=t.uint8, device="cuda"), t.zeros(4, 2, device="cuda")
    for bad in (lambda: gem.quant_fp8(x.double(), c, s), lambda: gem.quant_fp8(x, c.int(), s), lambda: gem.quant_fp8(x, c[:3], s),
                lambda: gem.quant_fp8(x, c, s[:, :1]), lambda: gem.quant_fp8(x.T, c, s), lambda: gem.quant_fp8(x.cpu(), c, s),
                lambda: gem.quant_fp8(x, c, s, up=x[:2]), lambda: gem.rmsnorm_fp8(x, t.zeros(255, device="cuda"), 1e-6, c, s),
                lambda: gem.rmsnorm_fp8(x, None, 1e-6, c, s, residual=x[:1]), lambda: gem.rmsnorm_fp8(x, None, 1e-6, c, s, out=x[:, :128]),
                lambda: gem.fp8_gemm(c, s, c, s, x), lambda: gem.fp8_gemm(c[:, ::2], s, c, s, x), lambda: gem.fp8_gemm(c, s[:1], c, s[:1], x),
                lambda: gem.fp8_gemm(c, s[:1], c, s, x[:, :3]), lambda: gem.fp8_gemm(c, s[:1], c, s, x, residual=t.zeros(4, 300, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gem.GemError):
        gem.quant_fp8(x[:, :250], c, s)


# ---- together ----------------------------------------------------------------------------------------


def _mlp(gem, t, T, H, F, V, seed=0):
    """Weights, buffers and one pass of what follows a layer's attention, up to the scores."""
    g = t.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: t.randn(*s, generator=g, device="cuda")  # noqa: E731
    f8 = t.float8_e4m3fn
    d = {}
    for name, n, k in (("gate_up", 2 * F, H), ("down", H, F), ("logits", V, H)):
        d[name] = (rnd(n, k) * 60).clamp_(-448, 448).to(f8)
        d[name + "_s"] = t.exp(0.3 * rnd(-(-n // 128), -(-k // 128))) / (60 * k ** 0.5)
    d.update(x=rnd(T, H), res=rnd(T, H), g1=1 + 0.1 * rnd(H), g2=1 + 0.1 * rnd(H), tokens=t.randint(0, V, (T,), generator=g, device="cuda").int(),
             h=t.empty(T, H, device="cuda"), c1=t.empty(T, H, dtype=f8, device="cuda"), s1=t.empty(T, -(-H // 128), device="cuda"),
             gu=t.empty(T, 2 * F, device="cuda"), c2=t.empty(T, F, dtype=f8, device="cuda"), s2=t.empty(T, -(-F // 128), device="cuda"),
             h2=t.empty(T, H, device="cuda"), c3=t.empty(T, H, dtype=f8, device="cuda"), s3=t.empty(T, -(-H // 128), device="cuda"),
             lg=t.empty(T, V, device="cuda"), logp=t.empty(T, device="cuda"), ent=t.empty(T, device="cuda"), rank=t.empty(T, dtype=t.int32, device="cuda"),
             idx=t.empty(T, 5, dtype=t.int32, device="cuda"), val=t.empty(T, 5, device="cuda"))

    def step(stream=None):
        F_ = d["gu"].shape[1] // 2
        gem.rmsnorm_fp8(d["x"], d["g1"], 1e-6, d["c1"], d["s1"], residual=d["res"], out=d["h"], stream=stream)
        gem.fp8_gemm(d["gate_up"], d["gate_up_s"], d["c1"], d["s1"], d["gu"], stream=stream)
        gem.quant_fp8(d["gu"][:, :F_], d["c2"], d["s2"], up=d["gu"][:, F_:], stream=stream)
        gem.fp8_gemm(d["down"], d["down_s"], d["c2"], d["s2"], d["h2"], residual=d["h"], stream=stream)
        gem.rmsnorm_fp8(d["h2"], d["g2"], 1e-6, d["c3"], d["s3"], stream=stream)
        gem.fp8_gemm(d["logits"], d["logits_s"], d["c3"], d["s3"], d["lg"], stream=stream)
        gem.logprobs(d["lg"], d["tokens"], d["logp"], d["ent"], d["rank"], d["idx"], d["val"], stream=stream)

    return d, step


_OUT = ("h", "gu", "h2", "lg", "logp", "ent", "rank", "idx", "val", "s1", "s2", "s3")


@pytest.mark.parametrize("T", [1, 9, 70, 300])
def test_layer_and_scores(env, T):
    """Each step against the oracle on what the step before it gave."""
    gem, t = env
    H, F, V = 512, 1040, 1000
    d, step = _mlp(gem, t, T, H, F, V, T)
    step()
    a = {k: v.cpu().numpy() if v.dtype != t.float8_e4m3fn else _u8(v) for k, v in d.items()}
    h, y = fp8.rmsnorm(a["x"], a["res"], a["g1"], 1e-6)
    assert np.array_equal(a["h"], h)
    _check_rows(d["c1"], d["s1"], y)
    want, most = fp8.gemm(a["gate_up"], a["gate_up_s"], a["c1"], a["s1"])
    assert np.all(np.abs(a["gu"] - want) <= _tol(H, most))
    _check_rows(d["c2"], d["s2"], fp8.gated(a["gu"][:, :F], a["gu"][:, F:], 0))
    want, most = fp8.gemm(a["down"], a["down_s"], a["c2"], a["s2"], a["h"])
    assert np.all(np.abs(a["h2"] - want) <= _tol(F, most))
    _check_rows(d["c3"], d["s3"], fp8.rmsnorm(a["h2"], None, a["g2"], 1e-6)[1])
    want, most = fp8.gemm(a["logits"], a["logits_s"], a["c3"], a["s3"])
    assert np.all(np.abs(a["lg"] - want) <= _tol(H, most))
    s = fp8.scores(a["lg"], a["tokens"], 5)
    assert np.array_equal(a["rank"], s["rank"]) and np.array_equal(a["idx"], s["idx"])
    assert np.allclose(a["logp"], s["logp"], rtol=0, atol=2e-5) and np.allclose(a["ent"], s["entropy"], rtol=0, atol=2e-5)


def test_layer_in_graphs_and_on_two_streams(env):
    """Two captured layers, each with buffers of its own, replayed at once on two streams and back to back, give
    what the eager calls give."""
    gem, t = env
    sets = [_mlp(gem, t, T, 512, 1040, 1000, T) for T in (9, 200)]
    want = []
    for d, step in sets:
        step()
        t.cuda.synchronize()
        want.append({k: d[k].clone() for k in _OUT})
    graphs, streams = [], [t.cuda.Stream() for _ in sets]
    for (d, step), s in zip(sets, streams):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=s):
            step()
        graphs.append(g)
    for _ in range(3):
        for d, _step in sets:
            for k in _OUT:
                d[k].zero_()
        t.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with t.cuda.stream(s):
                g.replay()
                g.replay()
        t.cuda.synchronize()
        for (d, _step), w in zip(sets, want):
            assert all(t.equal(d[k], w[k]) for k in _OUT)
    # eager calls on streams of their own, at once
    for (d, step), s in zip(sets, streams):
        for k in _OUT:
            d[k].zero_()
    t.cuda.synchronize()
    for (d, step), s in zip(sets, streams):
        step(stream=s)
    t.cuda.synchronize()
    for (d, _step), w in zip(sets, want):
        assert all(t.equal(d[k], w[k]) for k in _OUT)


# ---- waits that run out ---------------------------------------------------------------------------------


@pytest.mark.parametrize("M,K,N", [(4, 256, 64), (8, 2048, 384), (40, 1024, 700), (3, 4096, 640), (100, 2560, 19456), (300, 512, 512), (600, 1008, 1201), (300, 4096, 512)])
def test_gemm_wait_that_runs_out_is_reported(env, M, K, N):
    """The first stage of CTA 0 expects 16 bytes more than it gets: every wait behind it gives up after the limit, the
    call ends and says so, and the next one is right."""
    gem, t = env
    W, ws, x, xs = _operands(M, K, N, 6)
    d = [_dev(t, a) for a in (W, ws, x, xs)]
    y, status = t.full((M, N), -7.0, device="cuda"), t.zeros(1, dtype=t.int32, device="cuda")
    t.cuda.synchronize()
    gem.set_wait_limit(1_000_000)
    gem.set_test_injection(gem.INJECT_RING_SHORTFALL)
    try:
        gem.fp8_gemm(*d, y, status=status)
        t.cuda.synchronize()
    finally:
        gem.set_test_injection(0)
        gem.set_wait_limit(0)
    assert gem.status_from_flags(int(status)) == 6 and gem.device_status() == 0
    status.zero_()
    gem.fp8_gemm(*d, y, status=status)
    want, most = fp8.gemm(W, ws, x, xs)
    assert np.all(np.abs(y.cpu().numpy() - want) <= _tol(K, most)) and int(status) == 0


def test_gemm_clusters_on_several_streams(env):
    """Calls whose clusters share out K, of different widths, at once: none keeps another's tensor memory from it."""
    gem, t = env
    calls = []
    for i, (M, K, N) in enumerate([(8, 4096, 640), (24, 4096, 1100), (50, 2048, 384), (16, 1024, 2048), (100, 8192, 256)]):
        W, ws, x, xs = _operands(M, K, N, i)
        want, most = fp8.gemm(W, ws, x, xs)
        calls.append((want, _tol(K, most), [_dev(t, a) for a in (W, ws, x, xs)], t.zeros(40, M, N, device="cuda"), t.cuda.Stream()))
    t.cuda.synchronize()
    for r in range(40):
        for _, _, (W, ws, x, xs), y, s in calls:
            gem.fp8_gemm(W, ws, x, xs, y[r], stream=s)
    t.cuda.synchronize()
    for want, tol, _, y, _ in calls:
        got = y.cpu().numpy()
        assert (got == got[:1]).all()
        assert (np.abs(got[0] - want) <= tol).all()
    assert gem.device_status() == 0


@pytest.mark.parametrize("call", ["gem.rmsnorm_fp8(x, None, 1e-6, c, s)", "gem.quant_fp8(x, c, s)", "gem.fp8_gemm(c, s[:1], c, s, y)",
                                  "gem.fp8_gemm(c, s[:1], c.repeat(3, 1), s.repeat(3, 1), y.repeat(3, 1))", "gem.logprobs(x, None, None, x.new_empty(100))",
                                  "gem.fp8_gemm(c.new_zeros(64, 2048), x.new_ones(1, 16), c.new_zeros(8, 2048), x.new_ones(8, 16), x.new_zeros(8, 64))"])
def test_first_call_of_a_process_may_be_captured(call):
    """Whatever a call sets up in its process, it sets up without the stream."""
    import os
    import subprocess
    import sys
    code = """
import torch, q4_gemv_gqa_gb300 as gem
x = torch.ones(100, 128, device="cuda"); c = torch.zeros(100, 128, device="cuda", dtype=torch.uint8)
s = torch.ones(100, 1, device="cuda"); y = torch.ones(100, 100, device="cuda")
def run(): %s
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay(); torch.cuda.synchronize()
assert gem.device_status() == 0
""" % call
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240,
                          cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert done.returncode == 0, done.stderr[-2000:]
