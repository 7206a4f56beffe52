"""The 8-bit floating-point path at the edges of its calls: values, scales and strides at the ends of their ranges."""
import numpy as np
import pytest

from oracle import fp8
from test_gpu_fp8 import _check_rows, _dev, _operands, _product, _rows, _tol, _u8, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _gated(env, x, up, act):  # noqa: F811
    gem, t = env
    codes, scales = _rows(t, *x.shape)
    gem.quant_fp8(_dev(t, x), codes, scales, up=_dev(t, up), act=act)
    return codes, scales


@pytest.mark.parametrize("act", [0, 1])
def test_gate_of_values_whose_product_with_it_is_below_the_least_normal_one(env, act):  # noqa: F811
    """Blocks of tiny x (or of a tiny gate, or of tiny up) with factors that bring them back."""
    r = np.random.RandomState(act)
    T, H = 240, 256
    x, up = np.zeros((2, T, H), np.float32)
    x[:80] = (r.randint(1, 1 << r.randint(1, 23), (80, H)) * 2.0 ** -149).astype(np.float32)
    up[:80] = (r.randn(80, H) * np.exp2(r.uniform(60, 120, (80, 1)))).astype(np.float32)
    x[80:160] = r.uniform(*((-82.9, -75) if act == 0 else (-9.8, -9.4)), (80, H))
    up[80:160] = (r.randn(80, H) * np.exp2(r.uniform(30, 120, (80, 1)))).astype(np.float32)
    x[160:] = np.abs(r.randn(80, H) * np.exp2(r.uniform(50, 120, (80, 1)))).astype(np.float32)
    up[160:] = (r.randint(1, 1 << 20, (80, H)) * 2.0 ** -149).astype(np.float32)
    x[0], up[0] = 3 * 2.0 ** -149, 1e30
    codes, scales = _gated(env, x, up, act)
    y = fp8.gated(x, up, act)
    assert (np.abs(y).max(1) >= 2.0 ** -100).sum() > 200
    _check_rows(codes, scales, y)


@pytest.mark.parametrize("act", [0, 1])
def test_gate_at_its_lower_end(env, act):  # noqa: F811
    """The values on either side of z = -83, a block of each: zeros below it, e^-83 of x at it."""
    end = np.float32(-83) if act == 0 else np.float32(-9.809149)
    x = (np.full(64, end).view(np.int32) + np.arange(-32, 32)).astype(np.int32).view(np.float32)
    x = np.repeat(x[:, None], 128, 1)
    up = np.exp2(np.resize(np.arange(40, 120, dtype=np.float32), x.shape))
    y = fp8.gated(x, up, act)
    assert 20 < (y != 0).any(1).sum() < 44
    _check_rows(*_gated(env, x, up, act), y)


@pytest.mark.parametrize("act", [0, 1])
def test_infinite_gate_and_up(env, act):  # noqa: F811
    """A block with an infinity or a NaN on either side has no scale, whatever it meets; the others keep theirs."""
    r = np.random.RandomState(9)
    x, up = r.randn(12, 384).astype(np.float32), r.randn(12, 384).astype(np.float32)
    bad = np.zeros((12, 3), bool)
    for t, (a, b) in enumerate([(np.inf, 1), (-np.inf, 1), (np.nan, 1), (1, np.inf), (1, -np.inf), (1, np.nan), (-np.inf, 0), (np.inf, 0),
                                (-200, np.inf), (0, np.inf), (-np.inf, np.inf)]):
        x[t, 128 * (t % 3) + 7 * t], up[t, 128 * (t % 3) + 7 * t] = a, b
        bad[t, t % 3] = True
    codes, scales = _gated(env, x, up, act)
    assert np.array_equal(np.isnan(scales.cpu().numpy()), bad)
    with np.errstate(invalid="ignore"):
        _check_rows(codes, scales, fp8.gated(x, up, act))


@pytest.mark.parametrize("act", [0, 1])
def test_gated_values_past_the_largest_number(env, act):  # noqa: F811
    """Finite x and up whose product fp32 does not hold: the block has no scale.  Up to there it has."""
    x, up = np.full((40, 256), 3.0, np.float32), np.ones((40, 256), np.float32)
    x[:, 5] = np.exp2(np.arange(100, 120, 0.5)).astype(np.float32)
    up[:, 5] = -1.5 * 2.0 ** 17
    codes, scales = _gated(env, x, up, act)
    assert 10 < np.isnan(scales.cpu().numpy()[:, 0]).sum() < 30 and np.isfinite(scales.cpu().numpy()[:, 1]).all()
    _check_rows(codes, scales, fp8.gated(x, up, act))


@pytest.mark.parametrize("H", [128, 1280, 5376])
def test_norm_of_rows_over_the_whole_range(env, H):  # noqa: F811
    """gamma chosen so that every y is within fp32's last place of a border; rows are one row times powers of two, from squares
    of 2^-100 to sums of squares next to the largest number."""
    gem, t = env
    r = np.random.RandomState(H)
    base = r.uniform(1, 2, H).astype(np.float32) * r.choice([-1, 1], H)
    _, y = fp8.rmsnorm(base[None].astype(np.float32), None, None, 0.0)
    gamma = (r.choice(fp8._MID[70:126], H) / np.abs(y[0])).astype(np.float32)
    gamma[::128] = (440 / np.abs(y[0, ::128])).astype(np.float32)
    top = (127 - int(np.ceil(np.log2(4 * H)))) // 2
    k = np.arange(-48, top + 1)
    x = (base[None].astype(np.float64) * np.exp2(k.astype(np.float64))[:, None]).astype(np.float32)
    codes, scales = _rows(t, k.size, H)
    gem.rmsnorm_fp8(_dev(t, x), _dev(t, gamma), 0.0, codes, scales)
    _check_rows(codes, scales, fp8.rmsnorm(x, None, gamma, 0.0)[1])


def test_norm_of_zeros_with_the_least_eps(env):  # noqa: F811
    gem, t = env
    for eps in (1e-6, 1e-30, 1.2e-38, 1e-38, 1e-40, 1e-45):
        codes, scales = _rows(t, 3, 256)
        gem.rmsnorm_fp8(t.zeros(3, 256, device="cuda"), None, eps, codes, scales)
        assert not _u8(codes).any() and not scales.cpu().numpy().any()


def test_norm_product_with_gamma_past_the_largest_number(env):  # noqa: F811
    """h * gamma is formed in fp32: a block where it is not finite has no scale, up to there the codes are the exact ones."""
    gem, t = env
    r = np.random.RandomState(3)
    x = (r.uniform(1, 1.9, (4, 512)) * 2.0 ** 50).astype(np.float32)
    gamma = r.uniform(0.5, 1, 512).astype(np.float32)
    gamma[128:256] *= np.float32(2.0 ** 77)                 # products up to 1.9 * 2^127
    gamma[300] = 2.0 ** 78                                  # at least 2^128
    codes, scales = _rows(t, 4, 512)
    gem.rmsnorm_fp8(_dev(t, x), _dev(t, gamma), 1e-6, codes, scales)
    y = fp8.rmsnorm(x, None, gamma, 1e-6)[1]
    y[:, 300] = np.inf
    _check_rows(codes, scales, y)


@pytest.mark.parametrize("M", [3, 40, 100, 300])
def test_product_of_the_scales_at_its_ends(env, M):  # noqa: F811
    """xs * ws is formed in fp32: up to its largest number the results are right, past it they are not finite."""
    K, N = 384, 300
    W, ws, x, xs = _operands(M, K, N, 5)
    xs[1], ws[:] = xs[1] / xs[1].max() * 2.0 ** 100, ws / ws.max()
    ws[1] *= np.float32(2.0 ** 27.9)                        # rows 128 .. 255 of W
    x[1], W[128:256] = np.where(x[1] % 128 > 32, 8, x[1]), 1    # products of a few 2^-15
    xs[0], ws[2, 1] = 1.0, 2.0 ** 30
    xs[2], x[2, 128:256] = 2.0 ** 100, 0                    # nothing of row 2 in block 1
    y = _product(env, W, ws, x, xs).cpu().numpy()
    want, most = fp8.gemm(W, ws, x, xs)
    fine = np.ones((M, N), bool)
    fine[1, 256:] = fine[2, 256:] = False                   # 2^130
    assert np.all((np.abs(y - want) <= _tol(K, most))[fine & (most < 3e38)])
    assert not np.isfinite(y[2, 256:]).any()


@pytest.mark.parametrize("K", [256, 400])
def test_one_row_with_any_stride(env, K):  # noqa: F811
    """The stride of a single row leads nowhere, whatever it is."""
    gem, t = env
    W, ws, x, xs = _operands(1, K, 70, 1)
    d = [_dev(t, a) for a in (W, ws, x, xs)]
    y = t.zeros(1, 70, device="cuda")
    far = 1 << 45
    st = gem.lib.gem_fp8_gemm(d[0].data_ptr(), d[1].data_ptr(), 70, K, d[2].data_ptr(), far, d[3].data_ptr(), far, 1, y.data_ptr(), far,
                              None, None, t.cuda.current_stream().cuda_stream)
    assert st == 0
    want, most = fp8.gemm(W, ws, x, xs)
    assert np.all(np.abs(y.cpu().numpy() - want) <= _tol(K, most))
    codes, scales = _rows(t, 1, 256)
    row = np.random.RandomState(2).randn(1, 256).astype(np.float32)
    xd = _dev(t, row)
    assert gem.lib.gem_quant_fp8(xd.data_ptr(), far, xd.data_ptr(), far, 1, 256, 0, codes.data_ptr(), far, scales.data_ptr(), far,
                                 t.cuda.current_stream().cuda_stream) == 0
    _check_rows(codes, scales, fp8.gated(row, row, 0))


def test_norm_with_the_largest_eps(env):  # noqa: F811
    """Beside it a row whose squares' sum is next to the largest number."""
    gem, t = env
    r = np.random.RandomState(8)
    x = (r.randn(3, 256) * np.exp2([[3.0], [40.0], [58.0]])).astype(np.float32)
    x[2] = np.clip(x[2], -2.0 ** 59.4, 2.0 ** 59.4)
    codes, scales = _rows(t, 3, 256)
    gem.rmsnorm_fp8(_dev(t, x), None, 2.0 ** 127, codes, scales)
    _check_rows(codes, scales, fp8.rmsnorm(x, None, None, 2.0 ** 127)[1])
