"""Cases of the 8-bit floating-point path for prompts and batches, and of scoring what the model answers with.

  norm   gem.rmsnorm_fp8   residual addition, RMSNorm and its output in 8 bits (e4m3) with a scale for each 128 values
  quant  gem.quant_fp8     the gated activation, or a plain row, in the same 8-bit form
  gemm   gem.fp8_gemm      product of such rows with weights that have a scale for each block of 128 x 128
  score  gem.logprobs      log probabilities of given tokens, their ranks, the entropy and the top alternatives

One layer of a prompt runs norm, gemm (QKV), attention, quant, gemm (O); norm, gemm (gate and up), quant, gemm
(down); behind the last layer norm, gemm (logits), score.  `run` computes a case with the library's kernels where
`own` is true and with elementary torch operations otherwise.  The scale of an 8-bit row's block is the smallest
power of two that brings its largest magnitude to at most 448; weights have any scales.
"""
import math

import torch

own = False

EPS = 1e-6
TINY = 2.0 ** -100     # a block whose largest magnitude is below this is zeros with a scale of 0

# hidden sizes and FFN sizes of the library's own layer shapes, then generic ones
WIDTHS = [2048, 2560, 5376, 256, 4096, 1008]
FFNS = [6144, 9728, 21504, 512, 8192, 1200]
# (K, N) of the products in those layers: merged QKV, O, merged gate and up, down; then generic ones
PRODUCTS = [(2048, 4096), (2048, 12288), (6144, 2048), (2560, 6144), (2560, 19456), (9728, 2560), (5376, 21504), (21504, 5376),
            (5376, 16384), (256, 512), (4096, 4096), (1008, 1201)]
VOCABS = [262144, 65536, 151669, 32000, 1000]


def listed():
    return [
        # the two norms of a decode step of eight requests
        {"name": "norm decode t8", "op": "norm", "T": 8, "H": 2560, "residual": True},
        # a long prompt of a wide layer
        {"name": "norm prompt t4096", "op": "norm", "T": 4096, "H": 5376, "residual": True},
        # the gated activation of one decoded token, on its way to the down projection
        {"name": "quant decode t1", "op": "quant", "T": 1, "H": 6144, "gate": "silu"},
        # the same of a prompt with an odd number of tokens
        {"name": "quant prompt t4093", "op": "quant", "T": 4093, "H": 9728, "gate": "silu"},
        # QKV projection of one token: the weights are what it reads, and there are few of them
        {"name": "gemm m1 k2048 n4096", "op": "gemm", "M": 1, "K": 2048, "N": 4096, "residual": False},
        # up projection of a decode step of eight requests
        {"name": "gemm m8 k5376 n21504", "op": "gemm", "M": 8, "K": 5376, "N": 21504, "residual": False},
        # down projection of a batch of decoding requests, with the residual's addition
        {"name": "gemm m61 k21504 n5376", "op": "gemm", "M": 61, "K": 21504, "N": 5376, "residual": True},
        # merged gate and up projection of a short prompt
        {"name": "gemm m300 k2560 n19456", "op": "gemm", "M": 300, "K": 2560, "N": 19456, "residual": False},
        # up projection of a long prompt
        {"name": "gemm m4096 k5376 n21504", "op": "gemm", "M": 4096, "K": 5376, "N": 21504, "residual": False},
        # a decode step's sampled token, with the alternatives that an interface shows
        {"name": "score t1 v262144", "op": "score", "T": 1, "N": 262144, "k": 5, "coarse": False, "masked": 0.0},
        # a batch of decoding requests whose grammar bans part of the vocabulary
        {"name": "score t61 v151669 masked", "op": "score", "T": 61, "N": 151669, "k": 20, "coarse": True, "masked": 0.6},
        # scoring a prompt: every token's probability under the tokens before it
        {"name": "score t1021 v262144", "op": "score", "T": 1021, "N": 262144, "k": 1, "coarse": False, "masked": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant", "gemm", "gemm", "gemm", "score"])
    if op == "norm":
        H = rng.choice(WIDTHS)
        return {"op": op, "T": min(_log(rng, 1, 8192), 4096 * 5376 // H), "H": H, "residual": rng.random() < 0.7}
    if op == "quant":
        H = rng.choice(FFNS)
        return {"op": op, "T": min(_log(rng, 1, 8192), 4093 * 9728 // H), "H": H, "gate": rng.choice(["silu", "silu", "gelu", "none"])}
    if op == "gemm":
        K, N = rng.choice(PRODUCTS)
        return {"op": op, "M": min(_log(rng, 1, 8192), 4096 * 5376 * 21504 // (K * N)), "K": K, "N": N, "residual": rng.random() < 0.4}
    N = rng.choice(VOCABS)
    return {"op": op, "T": min(_log(rng, 1, 4096), 1021 * 262144 // N), "N": N, "k": rng.choice([0, 1, 5, 20, 64]),
            "coarse": rng.random() < 0.5, "masked": rng.choice([0.0, 0.0, 0.6])}


# ---- inputs -------------------------------------------------------------------------------------


def _blocks(n):
    return -(-n // 128)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _channels(g, n):
    """Scales of a row's channels: log-normal, a few of them far above the others."""
    return torch.exp(0.5 * _randn(g, n)) * torch.where(torch.rand(n, generator=g, device="cuda") < 0.002, 20.0, 1.0)


def _codes(*shape):
    return torch.zeros(*shape, dtype=torch.float8_e4m3fn, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    if c["op"] in ("norm", "quant"):
        T, H = c["T"], c["H"]
        c.update(codes=_codes(T, H), scales=torch.zeros(T, _blocks(H), device="cuda"))
        x = _randn(g, T, H) * _channels(g, H)
        if c["op"] == "norm":
            # the branch's output, and the residual stream that it is added to
            return dict(c, x=x, res=3 * _randn(g, T, H) if c["residual"] else None, out=torch.zeros(T, H, device="cuda"),
                        gamma=1 + 0.1 * _randn(g, H))
        if c["gate"] == "none":
            return dict(c, x=x, up=None)
        both = torch.cat([2 * _randn(g, T, H), x], 1)      # the merged projection's output: gate, then up
        return dict(c, x=both[:, :H], up=both[:, H:])
    if c["op"] == "gemm":
        M, K, N = c["M"], c["K"], c["N"]
        kb, nb = _blocks(K), _blocks(N)
        w = torch.zeros(nb * 128, kb * 128, device="cuda")
        w[:N, :K] = _randn(g, N, K)
        w *= torch.exp(0.3 * _randn(g, nb * 128, 1)) / math.sqrt(K)
        w = w.view(nb, 128, kb, 128)
        ws = w.abs().amax((1, 3)) / 448
        w = (w / ws[:, None, :, None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(nb * 128, kb * 128)[:N, :K].contiguous()
        x = torch.zeros(M, kb * 128, device="cuda")
        x[:, :K] = _randn(g, M, K) * _channels(g, K)
        x = x.view(M, kb, 128)
        xs = torch.exp2(torch.ceil(torch.log2(x.abs().amax(-1) / 448)))
        x = (x / xs[..., None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(M, -1)[:, :K].contiguous()
        return dict(c, w=w, ws=ws.contiguous(), x=x, xs=xs, y=torch.zeros(M, N, device="cuda"),
                    res=_randn(g, M, N) if c["residual"] else None)
    T, N, k = c["T"], c["N"], c["k"]
    y = _randn(g, T, N) * (1 + 2.5 * torch.rand(T, 1, generator=g, device="cuda"))
    # a few likely tokens in every row, of which the given one mostly is one
    likely = torch.randint(0, N, (T, 8), generator=g, device="cuda")
    y.scatter_add_(1, likely, 12 * torch.rand(T, 8, generator=g, device="cuda"))
    if c["coarse"]:
        y = y.bfloat16().float()                            # a model whose last product rounds to 16 bits: equal logits
    if c["masked"]:
        y.masked_fill_(torch.rand(T, N, generator=g, device="cuda") < c["masked"], -torch.inf)
    tokens = torch.where(torch.rand(T, generator=g, device="cuda") < 0.8, likely[:, 0], torch.randint(0, N, (T,), generator=g, device="cuda"))
    y.scatter_(1, tokens[:, None], y.gather(1, tokens[:, None]).clamp_(min=-20.0))    # a token that was sampled is not banned
    return dict(c, y=y, tokens=tokens.to(torch.int32), logp=torch.zeros(T, device="cuda"), entropy=torch.zeros(T, device="cuda"),
                rank=torch.zeros(T, dtype=torch.int32, device="cuda"), idx=torch.zeros(T, k, dtype=torch.int32, device="cuda"),
                val=torch.zeros(T, k, device="cuda"), scratch=torch.empty(8 << 20, dtype=torch.uint8, device="cuda"))


# ---- the plain form -----------------------------------------------------------------------------


def _to_codes(y):
    """Rows of 64-bit values as (codes, scales).  In 64 bits, because values next to a border fall on either side of it in 32."""
    T, H = y.shape
    kb = _blocks(H)
    y = torch.nn.functional.pad(y, (0, kb * 128 - H)).view(T, kb, 128)
    big = y.abs().amax(-1)
    m, e = torch.frexp(big)
    e = e + torch.where(m > 0.875, -8, -9)                  # 448 is 0.875 * 2^9
    scale = torch.where(big >= TINY, torch.ldexp(torch.ones_like(big), e), 0.0)
    t = torch.where(scale[..., None] > 0, torch.ldexp(y, -e[..., None]), 0.0)
    step = torch.ldexp(torch.ones_like(t), torch.frexp(t)[1].clamp_(min=-5) - 4)
    t = torch.round(t / step) * step
    return t.view(T, -1)[:, :H].float().to(torch.float8_e4m3fn), scale.float()


def _norm_plain(s):
    h = s["x"] if s["res"] is None else s["x"] + s["res"]
    y = h.double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * s["gamma"]
    return [h, *_to_codes(y)]


def _quant_plain(s):
    y = s["x"].double()
    if s["up"] is not None:
        z = y if s["gate"] == "silu" else 2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)
        y = y / (1 + torch.exp(-z)) * s["up"]               # 0.5 (1 + tanh(z / 2)) is 1 / (1 + exp(-z))
    return [*_to_codes(y)]


def _gemm_plain(s):
    K, N = s["K"], s["N"]
    x = s["x"].float() * s["xs"].repeat_interleave(128, 1)[:, :K]
    w = s["w"].float() * s["ws"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    y = torch.matmul(x, w.T)
    return y if s["res"] is None else y + s["res"]


def _score_plain(s):
    y, k = s["y"], s["k"]
    T, N = y.shape
    tok = s["tokens"].long()[:, None]
    given = y.gather(1, tok)
    most = y.amax(1, keepdim=True)
    d = y - most
    e = d.exp()
    total = e.sum(1, keepdim=True)
    log_total = total.log()
    entropy = log_total - torch.where(e > 0, d * e, 0.0).sum(1, keepdim=True) / total
    at = torch.arange(N, device=y.device)
    rank = 1 + ((y > given) | ((y == given) & (at < tok))).sum(1)
    got = [(given - most - log_total)[:, 0], entropy[:, 0], rank.to(torch.int32)]
    if k:
        bits = y.view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 31) - at     # the larger value first, then the lower index
        idx = key.topk(k, 1).indices
        got += [idx.to(torch.int32), y.gather(1, idx) - most - log_total]
    return got


# ---- one pass -----------------------------------------------------------------------------------


def run(s):
    op = s["op"]
    if not own:
        return {"norm": _norm_plain, "quant": _quant_plain, "gemm": _gemm_plain, "score": _score_plain}[op](s)
    import q4_gemv_gqa_gb300 as gem
    if op == "norm":
        gem.rmsnorm_fp8(s["x"], s["gamma"], EPS, s["codes"], s["scales"], residual=s["res"], out=s["out"])
        return [s["out"], s["codes"], s["scales"]]
    if op == "quant":
        gem.quant_fp8(s["x"], s["codes"], s["scales"], up=s["up"], act=gem.ACT_GELU_TANH if s["gate"] == "gelu" else gem.ACT_SILU)
        return [s["codes"], s["scales"]]
    if op == "gemm":
        return gem.fp8_gemm(s["w"], s["ws"], s["x"], s["xs"], s["y"], residual=s["res"])
    gem.logprobs(s["y"], s["tokens"], s["logp"], s["entropy"], s["rank"], s["idx"], s["val"], workspace=s["scratch"])
    return [s["logp"], s["entropy"], s["rank"]] + ([s["idx"], s["val"]] if s["k"] else [])


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        return {"bytes": n * (4 + 4 + (4 if c["residual"] else 0) + 1) + 4 * c["H"] + 4 * c["T"] * _blocks(c["H"]), "flops": 7 * n}
    if c["op"] == "quant":
        n = c["T"] * c["H"]
        return {"bytes": n * ((4 if c["gate"] == "none" else 8) + 1) + 4 * c["T"] * _blocks(c["H"]), "flops": n * (2 if c["gate"] == "none" else 7)}
    if c["op"] == "gemm":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": N * K + M * K + 4 * _blocks(K) * (M + _blocks(N)) + 4 * M * N * (2 if c["residual"] else 1), "flops": 2 * M * N * K}
    return {"bytes": c["T"] * (4 * c["N"] + 16 + 8 * c["k"]), "flops": 5 * c["T"] * c["N"]}


# ---- 64 bits ------------------------------------------------------------------------------------


def _exact_codes(y):
    codes, scales = [], []
    for a in range(0, y.shape[1], 128):
        b = y[:, a:a + 128]
        big = b.abs().max(1).values
        s = torch.exp2(torch.ceil(torch.log2(big / 448)))
        s = torch.where(big > s * 448, s * 2, torch.where(big <= s * 224, s / 2, s))   # where the logarithm's rounding was off
        s = torch.where(big < TINY, 0.0, s)
        v = torch.where(s[:, None] == 0, 0.0, b / s[:, None])
        # the grid: eight steps to each power of two, of 2^-9 below 2^-6
        unit = torch.full_like(v, 2.0 ** -9)
        for p in range(-6, 9):
            unit = torch.where(v.abs() >= 2.0 ** p, 2.0 ** (p - 3), unit)
        low = torch.floor(v / unit)
        part = v / unit - low
        up = (part > 0.5) | ((part == 0.5) & (torch.remainder(low, 2) == 1))
        codes.append((low + up) * unit)
        scales.append(s)
    return torch.cat(codes, 1), torch.stack(scales, 1)


def _exact_norm(s):
    h = s["x"] if s["res"] is None else s["res"] + s["x"]   # the residual stream is held in 32 bits
    y = h.double()
    return [h.double(), *_exact_codes(y * (y.pow(2).sum(1) / s["H"] + EPS).rsqrt()[:, None] * s["gamma"].double()[None])]


def _exact_quant(s):
    x = s["x"].double()
    if s["gate"] == "silu":
        x = x * torch.sigmoid(x) * s["up"].double()
    elif s["gate"] == "gelu":
        x = 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x.pow(3)))) * s["up"].double()
    return [*_exact_codes(x)]


def _exact_gemm(s):
    M, K, N = s["M"], s["K"], s["N"]
    y = torch.zeros(M, N, dtype=torch.float64, device="cuda") if s["res"] is None else s["res"].double()
    for b in range(_blocks(K)):
        a, z = 128 * b, min(K, 128 * b + 128)
        row = s["ws"][:, b].double().repeat_interleave(128)[:N]
        y.addmm_(s["x"][:, a:z].double() * s["xs"][:, b:b + 1].double(), (s["w"][:, a:z].double() * row[:, None]).T)
    return y


def _exact_score(s):
    logp, entropy, rank, idx, val = [], [], [], [], []
    k = s["k"]
    for t, tok in enumerate(s["tokens"].tolist()):
        y = s["y"][t].double()
        lp = y - torch.logsumexp(y, 0)
        p = lp.exp()
        logp.append(lp[tok])
        entropy.append(-(p * torch.where(p > 0, lp, 0.0)).sum())
        rank.append((y > y[tok]).sum() + (y[:tok] == y[tok]).sum() + 1)
        if k:
            order = torch.sort(y, descending=True, stable=True).indices[:k]
            idx.append(order)
            val.append(lp[order])
    got = [torch.stack(logp), torch.stack(entropy), torch.stack(rank).to(torch.int32)]
    return got + ([torch.stack(idx).to(torch.int32), torch.stack(val)] if k else [])


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "quant": _exact_quant, "gemm": _exact_gemm, "score": _exact_score}[s["op"]](s)
