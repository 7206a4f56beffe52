"""The 8-bit floating-point path and the scores without a GPU: the oracle against known answers and invariants,
and the library's host-side refusals, which come before any CUDA call."""
import ctypes as C
import math

import numpy as np
import pytest

from oracle import fp8

OK, INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 7
D = C.c_void_p(0x1000)      # a device pointer that no call reaches
ODD = C.c_void_p(0x1004)
BAD = C.c_void_p(0x1002)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__._build_module().build()
    from q4_gemv_gqa_gb300 import _lib
    return _lib.load()


# ---- the oracle -------------------------------------------------------------------------------


def test_codes_known_values():
    for code, want in ((0x00, 0.0), (0x01, 2.0 ** -9), (0x07, 7 * 2.0 ** -9), (0x08, 2.0 ** -6), (0x38, 1.0), (0x39, 1.125),
                       (0x7e, 448.0), (0xb8, -1.0), (0xfe, -448.0)):
        assert fp8.VALUES[code] == want
    assert np.isnan(fp8.VALUES[0x7f]) and np.isnan(fp8.VALUES[0xff])


def test_codes_agree_with_torch():
    import torch
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(every, nan=999.0), np.nan_to_num(fp8.VALUES, nan=999.0))
    x = np.random.RandomState(0).randn(5000).astype(np.float32) * np.exp2(np.random.RandomState(1).uniform(-12, 6, 5000)).astype(np.float32)
    x = np.clip(x, -448, 448)
    assert np.array_equal(torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), fp8.encode(x.astype(np.float64)))


def test_encode_every_code_and_every_border():
    finite = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    assert np.array_equal(fp8.encode(fp8.VALUES[finite]), finite)
    for c in range(126):
        mid = (fp8.VALUES[c] + fp8.VALUES[c + 1]) / 2
        even = c if c % 2 == 0 else c + 1
        got = fp8.encode(np.array([mid, np.nextafter(mid, 0), np.nextafter(mid, 999), -mid]))
        assert got.tolist() == [even, c, c + 1, even | 128]


def test_scale_is_the_smallest_power_of_two():
    for m, want in ((448.0, 1.0), (np.nextafter(448.0, 999), 2.0), (224.0, 0.5), (np.nextafter(224.0, 999), 1.0), (1.0, 2.0 ** -8),
                    (2.0 ** -100, 2.0 ** -108), (np.nextafter(2.0 ** -100, 0), 0.0), (0.0, 0.0), (3e38, 2.0 ** 120)):
        y = np.zeros((1, 128))
        y[0, 77] = -m
        codes, scales = fp8.quantise(y)
        assert scales[0, 0] == want
        assert want == 0 or 224 <= -fp8.VALUES[codes[0, 77]] <= 448
    for bad in (np.nan, np.inf, -np.inf):
        y = np.ones((1, 200))
        y[0, 130] = bad
        codes, scales = fp8.quantise(y)
        assert scales[0, 0] == 2.0 ** -8 and np.isnan(scales[0, 1]) and np.all(codes[0, 128:] == 0)


def test_rows_come_back_within_half_a_step():
    y = np.random.RandomState(2).randn(20, 300)
    codes, scales = fp8.quantise(y)
    back = fp8.values(codes, scales)
    s = np.repeat(scales, 128, 1)[:, :300]
    assert np.all(np.abs(back - y) <= np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10))


def test_norm_and_gate_known_answers():
    x = np.full((1, 16), 3.0, np.float32)
    h, y = fp8.rmsnorm(x, -x + 1, None, 0.0)
    assert np.all(h == 1) and np.all(y == 1)
    one = np.ones((1, 1), np.float32)
    assert math.isclose(fp8.gated(one, one, 0)[0, 0], math.e / (1 + math.e), rel_tol=1e-15)
    want = 0.5 * (1 + math.tanh(math.sqrt(2 / math.pi) * 1.044715))
    assert math.isclose(fp8.gated(one, one, 1)[0, 0], want, rel_tol=1e-14)


def test_gemm_is_the_dense_product_of_the_values():
    r = np.random.RandomState(3)
    W, ws = fp8.encode(r.randn(150, 272)), r.rand(2, 3).astype(np.float32)
    x, xs = fp8.quantise(r.randn(4, 272))
    y, most = fp8.gemm(W, ws, x, xs)
    for m, n in ((0, 0), (3, 127), (2, 128), (1, 149)):
        want = sum(fp8.VALUES[x[m, k]] * float(xs[m, k // 128]) * fp8.VALUES[W[n, k]] * float(ws[n // 128, k // 128]) for k in range(272))
        assert abs(y[m, n] - want) <= 1e-13 * most[m, n]


def test_scores_known_answers():
    y = np.array([[0.0, math.log(2), math.log(2), -np.inf, math.log(5)]], np.float32)
    got = fp8.scores(y, [2], 4)
    assert np.allclose(got["logp"], math.log(0.2), atol=1e-7) and got["rank"][0] == 3
    assert got["idx"][0].tolist() == [4, 1, 2, 0]
    p = np.array([0.1, 0.2, 0.2, 0.5])
    assert np.allclose(got["entropy"], -(p * np.log(p)).sum(), atol=1e-7)
    assert np.allclose(fp8.scores(np.zeros((1, 1000), np.float32), [999], 1)["entropy"], math.log(1000))
    nan = fp8.scores(np.array([[1, np.nan, 2]], np.float32), [1], 3)
    assert np.isnan(nan["logp"][0]) and nan["idx"][0].tolist() == [2, 0, 1] and nan["rank"][0] == 3
    none = fp8.scores(np.full((1, 3), -np.inf, np.float32), [-1], 1)
    assert none["logp"][0] == 0 and none["rank"][0] == 0 and np.isnan(none["entropy"][0])


# ---- refusals ---------------------------------------------------------------------------------


def test_norm_refusals(lib):
    def f(x=D, ldx=256, res=None, ldr=0, out=None, ldo=0, T=2, H=256, gamma=None, eps=1e-6, codes=D, ldc=256, scales=D, lds=2):
        return lib.gem_rmsnorm_fp8(x, ldx, res, ldr, out, ldo, T, H, gamma, eps, codes, ldc, scales, lds, None)

    assert f(T=0) == OK and f(H=0, ldx=0) == OK
    assert f(T=-1) == INVALID and f(H=-16) == INVALID and f(eps=-1.0) == INVALID and f(eps=math.nan) == INVALID and f(eps=math.inf) == INVALID
    assert f(x=None) == INVALID and f(codes=None) == INVALID and f(scales=None) == INVALID
    assert f(ldx=252) == INVALID and f(res=D, ldr=252) == INVALID and f(out=D, ldo=252) == INVALID and f(ldc=240) == INVALID and f(lds=1) == INVALID
    assert f(out=D, ldo=512) == INVALID                       # out is x, with another stride
    assert f(res=C.c_void_p(0x2000), ldr=256, out=C.c_void_p(0x2000), ldo=512) == INVALID
    assert f(H=250) == UNSUPPORTED and f(H=32784, ldx=40000) == UNSUPPORTED and f(T=1 << 31) == UNSUPPORTED
    assert f(x=ODD) == MISALIGNED and f(ldx=258) == MISALIGNED and f(res=ODD, ldr=256) == MISALIGNED and f(out=ODD, ldo=256) == MISALIGNED
    assert f(gamma=ODD) == MISALIGNED and f(codes=ODD) == MISALIGNED and f(ldc=264) == MISALIGNED and f(scales=BAD) == MISALIGNED


def test_quant_refusals(lib):
    def f(x=D, ldx=256, up=None, ldu=0, T=2, H=256, act=0, codes=D, ldc=256, scales=D, lds=2):
        return lib.gem_quant_fp8(x, ldx, up, ldu, T, H, act, codes, ldc, scales, lds, None)

    assert f(T=0) == OK and f(H=0, ldx=0) == OK
    assert f(T=-1) == INVALID and f(act=2) == INVALID and f(act=-1) == INVALID and f(x=None) == INVALID
    assert f(ldx=252) == INVALID and f(up=D, ldu=252) == INVALID and f(ldc=240) == INVALID and f(lds=1) == INVALID
    assert f(H=24, ldx=256) == UNSUPPORTED and f(T=1 << 31) == UNSUPPORTED
    assert f(x=ODD) == MISALIGNED and f(up=ODD, ldu=256) == MISALIGNED and f(up=D, ldu=257) == MISALIGNED and f(codes=ODD) == MISALIGNED


def test_gemm_refusals(lib):
    def f(W=D, ws=D, N=256, K=256, x=D, ldx=256, xs=D, ldxs=2, M=2, y=D, ldy=256, res=None, status=None):
        return lib.gem_fp8_gemm(W, ws, N, K, x, ldx, xs, ldxs, M, y, ldy, res, status, None)

    assert f(M=0) == OK and f(N=0) == OK
    assert f(M=-1) == INVALID and f(N=-1) == INVALID and f(K=-16) == INVALID and f(K=0) == INVALID
    assert f(W=None) == INVALID and f(ws=None) == INVALID and f(x=None) == INVALID and f(xs=None) == INVALID and f(y=None) == INVALID
    assert f(ldx=240) == INVALID and f(ldxs=1) == INVALID and f(ldy=255) == INVALID
    assert f(K=250) == UNSUPPORTED and f(M=1 << 31) == UNSUPPORTED and f(N=1 << 31) == UNSUPPORTED
    assert f(W=ODD) == MISALIGNED and f(x=ODD) == MISALIGNED and f(ldx=264) == MISALIGNED
    assert f(ws=BAD) == MISALIGNED and f(y=BAD) == MISALIGNED and f(res=BAD) == MISALIGNED and f(status=BAD) == MISALIGNED


def test_logprobs_refusals(lib):
    def f(y=D, ldy=1000, T=4, N=1000, scale=1.0, tok=D, logp=D, rank=D, ent=D, k=5, idx=D, val=D, status=None):
        return lib.gem_logprobs(y, ldy, T, N, scale, tok, logp, rank, ent, k, idx, val, status, None)

    assert f(T=0) == OK
    assert f(T=-1) == INVALID and f(N=0) == INVALID and f(k=-1) == INVALID and f(N=4, k=5) == INVALID
    assert f(scale=0.0) == INVALID and f(scale=-1.0) == INVALID and f(scale=math.nan) == INVALID and f(scale=math.inf) == INVALID
    assert f(y=None) == INVALID and f(ldy=999) == INVALID and f(idx=None) == INVALID and f(val=None) == INVALID and f(tok=None) == INVALID
    assert f(k=65) == UNSUPPORTED and f(N=1 << 31, ldy=1 << 31) == UNSUPPORTED and f(T=1 << 28) == UNSUPPORTED
    assert f(y=BAD) == MISALIGNED and f(tok=BAD) == MISALIGNED and f(logp=BAD) == MISALIGNED and f(val=BAD) == MISALIGNED
    assert f(rank=BAD) == MISALIGNED and f(ent=BAD) == MISALIGNED and f(idx=BAD) == MISALIGNED and f(status=BAD) == MISALIGNED


def test_binding_refuses_other_devices_and_shapes(lib):
    import q4_gemv_gqa_gb300 as gem
    import torch
    if torch.cuda.is_available():
        pytest.skip("the CPU's own refusals")
    t = torch.zeros(2, 256)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        gem.quant_fp8(t, torch.zeros(2, 256, dtype=torch.uint8), torch.zeros(2, 2))
