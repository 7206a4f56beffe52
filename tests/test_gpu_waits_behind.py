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
