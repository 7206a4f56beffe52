"""Bounded waits behind a long kernel.  A call may begin while the kernel before it on the stream still runs; that
kernel's time is not part of its waits, however low their limit is."""
import numpy as np
import pytest

from oracle import fp8
from test_gpu_fp8 import _dev, _operands, _tol, env  # noqa: F401

pytestmark = pytest.mark.gpu

LIMIT_NS = 1_000_000


@pytest.fixture(scope="module")
def long_kernel(env):  # noqa: F811
    """A kernel of the library that takes several times the limit on 16 SMs, and leaves the others to the next."""
    gem, t = env
    y, out = t.zeros(1, 1 << 30, device="cuda"), t.zeros(1, device="cuda")
    run = lambda: gem.logprobs(y, None, None, out)  # noqa: E731
    run()
    a, b = t.cuda.Event(enable_timing=True), t.cuda.Event(enable_timing=True)
    a.record()
    run()
    b.record()
    t.cuda.synchronize()
    assert a.elapsed_time(b) > 2e-6 * LIMIT_NS
    return run


def _behind(env, long_kernel, call):  # noqa: F811
    """`call` behind the long kernel under the low limit, three times; device flags set by then."""
    gem, t = env
    call()
    t.cuda.synchronize()
    gem.device_status(reset=True)
    gem.set_wait_limit(LIMIT_NS)
    try:
        for _ in range(3):
            long_kernel()
            call()
            t.cuda.synchronize()
    finally:
        gem.set_wait_limit(0)
    return gem.device_status(reset=True)


@pytest.mark.parametrize("M,K,N", [(4, 256, 64), (8, 5376, 21504), (40, 1024, 700), (3, 4096, 640), (61, 21504, 384), (100, 2560, 9728), (300, 512, 512),
                                   (600, 1008, 1201), (300, 4096, 512)])
def test_block_scaled_product(env, long_kernel, M, K, N):  # noqa: F811
    gem, t = env
    W, ws, x, xs = _operands(M, K, N, 6)
    d, y = [_dev(t, a) for a in (W, ws, x, xs)], t.full((M, N), -7.0, device="cuda")
    assert _behind(env, long_kernel, lambda: gem.fp8_gemm(*d, y)) == 0
    want, most = fp8.gemm(W, ws, x, xs)
    assert np.all(np.abs(y.cpu().numpy() - want) <= _tol(K, most))


def _blocks(t, N, K, size):
    """Weights of N rows in blocks of 32 values and `size` bytes, each with a scale of 2^-7."""
    W = t.randint(0, 256, (N, K // 32, size), generator=t.Generator(device="cuda").manual_seed(0), device="cuda", dtype=t.uint8)
    W[:, :, 0], W[:, :, 1] = 0, 0x20
    return W.view(-1)


@pytest.mark.parametrize("B", [1, 2, 4, 8, 16, 32])
@pytest.mark.parametrize("K,N", [(5376, 21504), (21504, 5376)])
def test_q4_0_products(env, long_kernel, B, K, N):  # noqa: F811
    gem, t = env
    W, x, y = _blocks(t, N, K, 18), t.randn(B, K, device="cuda"), t.zeros(B, N, device="cuda")
    calls = [lambda: gem.q4_0_gemm(W, None, N, K, x, y), lambda: gem.q4_0_gemm(W, W, N, K, x, y)]
    if B <= 8:
        calls += [lambda: gem.q4_0_gemv(W, N, K, x, y), lambda: gem.q4_0_gemv(W, N, K, x, y, shared_records=True)]
    for call in calls:
        call()
        want = y.clone()
        assert _behind(env, long_kernel, call) == 0
        assert t.equal(y, want)


@pytest.mark.parametrize("B", [1, 2, 4, 8])
def test_q8_0_products(env, long_kernel, B):  # noqa: F811
    gem, t = env
    N, K = 65536, 5376
    W, x, y = _blocks(t, N, K, 34), t.randn(B, K, device="cuda"), t.zeros(B, N, device="cuda")
    call = lambda: gem.q8_0_gemv(W, N, K, x, y)  # noqa: E731
    call()
    want = y.clone()
    assert _behind(env, long_kernel, call) == 0
    assert t.equal(y, want)
