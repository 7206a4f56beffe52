"""A whole layer of the 8-bit path with attention over the paged 4-bit cache between its products, for prompts and for a
decoding step behind them, up to the scores: each call against the oracle on what the call before it gave."""
import numpy as np
import pytest

from oracle import fp8, kv4
from parity import assert_close
from test_gpu_fp8 import _check_rows, _dev, _tol, _u8, env  # noqa: F401

pytestmark = pytest.mark.gpu

H, NQ, NKV, D, F, V, PAGE = 256, 4, 2, 64, 528, 700, 16
QKV, THETA, SCALE = (NQ + 2 * NKV) * D, 1e4, D ** -0.5


def _weights(t, n, k, seed):
    r = np.random.RandomState(seed)
    w, s = fp8.encode(np.clip(r.randn(n, k) * 60, -448, 448)), np.exp(0.3 * r.randn(-(-n // 128), -(-k // 128))) / (60 * k ** 0.5)
    return w, s.astype(np.float32), _dev(t, w), _dev(t, s.astype(np.float32))


@pytest.mark.parametrize("new", [(17, 3), (150, 61), (1, 200)])
def test_layer_with_attention(env, new):  # noqa: F811
    gem, t = env
    B, pages = len(new), sum(-(-(n + 1) // PAGE) for n in new)
    i32 = dict(dtype=t.int32, device="cuda")
    W = {name: _weights(t, n, k, i) for i, (name, n, k) in enumerate((("qkv", QKV, H), ("o", H, NQ * D), ("gate_up", 2 * F, H), ("down", H, F),
                                                                      ("logits", V, H)))}
    r = np.random.RandomState(9)
    g1, g2, g3 = ((1 + 0.1 * r.randn(H)).astype(np.float32) for _ in range(3))
    pool = t.zeros(pages, gem.kv4_page_bytes(NKV, D, PAGE), dtype=t.uint8, device="cuda")
    table, ring = t.full((B, pages), -1, **i32), t.arange(pages, **i32)
    heads = t.tensor([[0, pages], [0, 0]], device="cuda")
    cached = np.zeros(B, np.int32)
    seen = [np.zeros((0, 2, NKV, D)) for _ in new]               # each request's keys and values, as the cache holds them
    for step, fresh in enumerate((new, (1,) * B)):
        T = sum(fresh)
        kv_len, cu = t.zeros(B, **i32), t.zeros(B + 1, **i32)
        slot, at, seq = (t.zeros(T, **i32) for _ in range(3))
        gem.kv_block_tables(_dev(t, cached), t.tensor(fresh, **i32), PAGE, table, ring, heads[step % 2], heads[(step + 1) % 2], kv_len, cu,
                            slot, at, seq)
        buf = lambda n: t.full((T, n), -7.0, device="cuda")  # noqa: E731
        row = lambda n: (t.empty(T, n, dtype=t.float8_e4m3fn, device="cuda"), t.empty(T, -(-n // 128), device="cuda"))  # noqa: E731

        def product(name, rows, y, residual=None):
            w, s, dw, ds = W[name]
            before = None if residual is None else residual.cpu().numpy()
            gem.fp8_gemm(dw, ds, *rows, y, residual=residual)
            want, most = fp8.gemm(w, s, _u8(rows[0]), rows[1].cpu().numpy(), before)
            assert np.all(np.abs(y.cpu().numpy() - want) <= _tol(w.shape[1], most)), name
            return y

        x, h, qkv, att = _dev(t, r.randn(T, H).astype(np.float32)), buf(H), buf(QKV), buf(NQ * D)
        c = row(H)
        gem.rmsnorm_fp8(x, _dev(t, g1), 1e-6, *c, out=h)
        _check_rows(*c, fp8.rmsnorm(x.cpu().numpy(), None, g1, 1e-6)[1], "first norm")
        product("qkv", c, qkv)

        raw = qkv.cpu().numpy()
        gem.qknorm_mrope(qkv, NQ, NKV, D, None, None, 1e-6, at[None], [D // 2], THETA, qkv)
        got = qkv.cpu().numpy()
        assert_close(got[:, :(NQ + NKV) * D], kv4.qknorm_mrope(raw, NQ, NKV, D, None, None, 1e-6, at.cpu().numpy()[None], [D // 2], THETA), "RoPE")
        gem.kv4_append(qkv[:, NQ * D:(NQ + NKV) * D], qkv[:, (NQ + NKV) * D:], NKV, D, slot, pool, PAGE)
        gem.kv4_attn(qkv, NQ, NKV, D, cu, kv_len, table, pool, PAGE, 0, SCALE, att)
        a = 0
        for b, n in enumerate(fresh):
            rows = got[a:a + n, NQ * D:].reshape(n, 2, NKV, D)
            seen[b] = np.concatenate([seen[b], kv4.values(*kv4.quantise(rows)).reshape(n, 2, NKV, D)])
            assert_close(att[a:a + n].cpu().numpy(), kv4.attention(got[a:a + n, :NQ * D].reshape(n, NQ, D), seen[b][:, 0], seen[b][:, 1],
                                                                   seen[b].shape[0], 0, SCALE).reshape(n, -1), "attention")
            a += n

        c = row(NQ * D)
        gem.quant_fp8(att, *c)
        _check_rows(*c, att.cpu().numpy().astype(np.float64), "attention's rows")
        product("o", c, h, residual=h)

        c, gu = row(H), buf(2 * F)
        gem.rmsnorm_fp8(h, _dev(t, g2), 1e-6, *c)
        _check_rows(*c, fp8.rmsnorm(h.cpu().numpy(), None, g2, 1e-6)[1], "second norm")
        product("gate_up", c, gu)
        c = row(F)
        gem.quant_fp8(gu[:, :F], *c, up=gu[:, F:], act=gem.ACT_GELU_TANH)
        both = gu.cpu().numpy()
        _check_rows(*c, fp8.gated(both[:, :F], both[:, F:], 1), "gate")
        product("down", c, h, residual=h)

        c, logits = row(H), buf(V)
        gem.rmsnorm_fp8(h, _dev(t, g3), 1e-6, *c)
        product("logits", c, logits)
        tokens, lp, rank = t.arange(T, **i32) % V, t.zeros(T, device="cuda"), t.zeros(T, **i32)
        gem.logprobs(logits, tokens, lp, None, rank)
        want = fp8.scores(logits.cpu().numpy(), tokens.cpu().numpy(), 0)
        assert np.array_equal(rank.cpu().numpy(), want["rank"])
        assert np.all(np.abs(lp.cpu().numpy() - want["logp"]) <= 2.0 ** -24 * (132 + 4 * want["spread"]) + 2.0 ** -22 * np.abs(want["logp"]))
        cached = cached + np.array(fresh, np.int32)
    assert gem.device_status(reset=True) == 0
