"""Scratch that a binding allocates itself belongs to the stream of the call.  The library's entry points are
replaced, so that nothing is launched: the test looks at the memory that they would have been given."""
import pytest

from test_gpu_kv4 import env  # noqa: F401

pytestmark = pytest.mark.gpu


def _calls(g, t):
    f = lambda *shape: t.zeros(shape, device="cuda")  # noqa: E731
    i = lambda *shape: t.zeros(shape, dtype=t.int32, device="cuda")  # noqa: E731
    W = t.zeros(512 * 256 // 32 * 18, dtype=t.uint8, device="cuda")
    pool = t.zeros((4, g.kv4_page_bytes(2, 128, 16)), dtype=t.uint8, device="cuda")
    return {
        "gem_q4_0_gemv_ws": lambda s: g.q4_0_gemv(W, 512, 256, f(2, 256), f(2, 512), stream=s),
        "gem_q4_0_gemv_fused": lambda s: g.q4_0_gemv_fused(W, None, 512, 256, f(2, 256), f(2, 512), stream=s),
        "gem_q4_0_gemm": lambda s: g.q4_0_gemm(W, None, 512, 256, f(16, 256), f(16, 512), stream=s),
        "gem_argmax": lambda s: g.argmax(f(2, 100000), i(2), stream=s),
        "gem_topk": lambda s: g.topk(f(2, 100000), 8, i(2, 8), f(2, 8), stream=s),
        "gem_kv4_attn": lambda s: g.kv4_attn(f(2, 512), 4, 2, 128, i(3), i(2), i(2, 2), pool, 16, 0, 0.1, f(2, 512), stream=s),
    }


@pytest.mark.parametrize("entry", ["gem_q4_0_gemv_ws", "gem_q4_0_gemv_fused", "gem_q4_0_gemm", "gem_argmax", "gem_topk",
                                   "gem_kv4_attn"])
def test_scratch_is_the_memory_of_the_calls_stream(env, monkeypatch, entry):
    g, t = env
    side, seen = t.cuda.Stream(), []

    def fake(*args):
        blocks = [(s["address"], s["total_size"], s["stream"]) for s in t.cuda.memory_snapshot()]
        seen.append({stream for x in args if isinstance(x, int) for at, n, stream in blocks if at <= x < at + n})
        return 0

    call = _calls(g, t)[entry]
    monkeypatch.setattr(g.lib, entry, fake)
    call(side)
    call(None)
    assert len(seen) == 2
    assert side.cuda_stream in seen[0], "the scratch of a call on a side stream is another stream's memory"
    assert side.cuda_stream not in seen[1]
