"""Cases of the paged 4-bit KV cache operators: what a serving loop runs between the QKV and the O
projection of a layer, and once per step to place the new tokens.

  tables  gem.kv_block_tables   pages for the new tokens of a batch of requests, and every token's slot
  rope    gem.qknorm_mrope      QK-norm and rotary positions with one or several axes
  append  gem.kv4_append        K and V rows quantised into their slots, and gem.kv4_gather reading them back
  attn    gem.kv4_attn          grouped-query attention over the pages

`run` computes a case with the library's kernels where `own` is true and with elementary torch
operations otherwise.  A page holds `page` tokens of every KV head as [n_kv][page / 16] tiles; a tile
is 16 tokens of one head: K codes [d / 32][16][16 bytes], V codes likewise, K scales [d / 32][16]
binary16, V scales likewise.  16 bytes of codes hold 32 values, byte j element j in its low nibble
and element j + 16 in its high nibble; a value is (code - 8) * scale.
"""
import math

import torch

own = False

EPS = 1e-6
SCRATCH = 32 << 20   # bytes of scratch that a serving loop keeps for its attention calls

# (query heads, KV heads, head dim) of the library's own layer shapes, then generic ones
HEADS = [(16, 8, 128), (32, 8, 128), (32, 16, 256), (32, 4, 512), (4, 2, 64), (6, 2, 128), (8, 1, 128), (8, 8, 64)]


def listed():
    return [
        # one decode step of a small batch: every request places one token
        {"name": "tables decode b8", "op": "tables", "B": 8, "cached": 2048, "fresh": 1, "mixed": False, "page": 16},
        # a busy server: chunks of prompts beside decoding requests, ended and idle ones
        {"name": "tables mixed b1024", "op": "tables", "B": 1024, "cached": 8192, "fresh": 512, "mixed": True, "page": 64},
        # the new tokens of an eight-row decode step
        {"name": "rope decode t8", "op": "rope", "T": 8, "heads": 1, "axes": 1, "interleaved": False, "norm": True},
        # a prompt with images: time, height and width positions on interleaved frequencies
        {"name": "rope image t4093", "op": "rope", "T": 4093, "heads": 1, "axes": 3, "interleaved": True, "norm": True},
        # the same step's rows into the cache
        {"name": "append decode t8", "op": "append", "T": 8, "heads": 1, "page": 16},
        # a prompt's rows of a wide layer, an odd number of them
        {"name": "append prompt t4095", "op": "append", "T": 4095, "heads": 2, "page": 64},
        # single-stream decode at 4096 cached positions
        {"name": "attn b1 4097", "op": "attn", "B": 1, "kv": 4097, "ragged": 0.0, "new": 1, "heads": 0, "page": 16, "window": 0},
        # batched decode, requests of different lengths
        {"name": "attn b8 2049 ragged", "op": "attn", "B": 8, "kv": 2049, "ragged": 0.7, "new": 1, "heads": 1, "page": 32, "window": 0},
        # long contexts: the cache is what the step reads
        {"name": "attn b8 32768", "op": "attn", "B": 8, "kv": 32768, "ragged": 0.3, "new": 1, "heads": 1, "page": 64, "window": 0},
        # wide heads, eight query heads to a KV head, one long sequence
        {"name": "attn b1 32769 d512", "op": "attn", "B": 1, "kv": 32769, "ragged": 0.0, "new": 1, "heads": 3, "page": 64, "window": 0},
        # sliding-window layers
        {"name": "attn b8 window1024", "op": "attn", "B": 8, "kv": 5000, "ragged": 0.9, "new": 1, "heads": 2, "page": 32, "window": 1024},
        # chunks of prompts: 32 new tokens each behind what is cached
        {"name": "attn b4 chunk32", "op": "attn", "B": 4, "kv": 4111, "ragged": 0.5, "new": 32, "heads": 1, "page": 64, "window": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "append", "attn", "attn", "attn"])
    if op == "tables":
        return {"op": op, "B": _log(rng, 1, 1024), "cached": _log(rng, 1, 8192), "fresh": _log(rng, 1, 512),
                "mixed": rng.random() < 0.6, "page": rng.choice([16, 32, 64, 128, 256])}
    heads = rng.randrange(len(HEADS))
    n_q, n_kv, d = HEADS[heads]
    if op == "rope":
        T = max(1, min(_log(rng, 1, 8192), 4093 * 40 * 128 // ((n_q + n_kv) * d)))
        axes = rng.choice([1, 2, 3])
        return {"op": op, "T": T, "heads": heads, "axes": axes, "interleaved": axes > 1 and rng.random() < 0.5, "norm": rng.random() < 0.7}
    if op == "append":
        T = max(1, min(_log(rng, 1, 8192), 4095 * 16 * 256 // (n_kv * d)))
        return {"op": op, "T": T, "heads": heads, "page": rng.choice([16, 32, 64, 128])}
    B = _log(rng, 1, 24)
    new = 1 if rng.random() < 0.6 else _log(rng, 2, 32)
    kv = _log(rng, 1, 40000)
    kv = max(new, min(kv, 6 * 32768 * 8 * 128 // (B * n_kv * d * (1 if new == 1 else 8))))
    window = _log(rng, 8, 2048) if rng.random() < 0.25 else 0
    return {"op": op, "B": B, "kv": kv, "ragged": round(rng.uniform(0.0, 0.95), 2), "new": new, "heads": heads,
            "page": rng.choice([16, 32, 64, 128, 256]), "window": window}


# ---- lengths of a case: the same for every seed, in an order that the seed picks ----------------


def _attn_lengths(c):
    B, kv, new = c["B"], c["kv"], c["new"]
    total = [max(new, round(kv * (1.0 - c["ragged"] * b / max(1, B - 1)))) for b in range(B)]
    # beside full chunks of new tokens some requests bring fewer, and some decode
    fresh = [new if b % 3 == 0 else max(1, new - 5 * (b % 3)) for b in range(B)]
    return total, fresh


def _table_lengths(c):
    got = []
    for b in range(c["B"]):
        cached = c["cached"] * (b % 7 + 1) // 7 + b % 5
        fresh = c["fresh"]
        if c["mixed"]:
            kind = b % 8
            cached = 0 if kind == 1 else cached
            fresh = {0: -1, 1: c["fresh"], 2: max(1, c["fresh"] // 2 + 1), 3: 0}.get(kind, 1)
        got.append((cached, fresh))
    return got


def _pages(n, page):
    return -(-n // page)


def _sections(axes, half):
    if axes == 1:
        return [half]
    rest = half // (axes + 1)
    return [half - rest * (axes - 1)] + [rest] * (axes - 1)


def _axis_of(sections, interleaved):
    n, half = len(sections), sum(sections)
    if not interleaved:
        return [a for a, s in enumerate(sections) for _ in range(s)]
    return [i % n if i % n and i < n * sections[i % n] else 0 for i in range(half)]


# ---- inputs -------------------------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pool(n_pages, page, n_kv, d, g):
    """Pages whose values are normal, with the channels of K and V at scales of their own."""
    bank = 2048
    x = torch.randn(bank, 2, d // 32, 16, 32, generator=g, device="cuda")
    x *= torch.exp(0.4 * torch.randn(2, d // 32, 1, 32, generator=g, device="cuda"))
    at = x.abs().argmax(-1, keepdim=True)
    s = (x.gather(-1, at) / -8).half()
    q = (8 + torch.round(x / s.float())).clamp_(0, 15).to(torch.uint8)
    codes = (q[..., :16] | (q[..., 16:] << 4)).reshape(bank, -1)
    tiles = torch.cat([codes, s.reshape(bank, -1).view(torch.uint8)], 1)
    n = n_pages * n_kv * (page // 16)
    pick = torch.randint(0, bank, (n,), generator=g, device="cuda")
    return tiles[pick].reshape(n_pages, -1)


def prepare(case, seed):
    g = _generator(seed)
    c = dict(case)
    if c["op"] == "tables":
        B, page = c["B"], c["page"]
        lens = _table_lengths(c)
        order = torch.randperm(B, generator=g, device="cuda")
        lens = torch.tensor(lens, dtype=torch.int32, device="cuda")[order]
        cached, fresh = lens[:, 0].contiguous(), lens[:, 1].contiguous()
        held_most = max(_pages(x, page) for x, _ in _table_lengths(c))
        max_pages = max(_pages(x + max(f, 0), page) for x, f in _table_lengths(c)) + 1
        held = sum(_pages(x, page) for x, _ in _table_lengths(c))
        need = sum(_pages(x + f, page) - _pages(x, page) for x, f in _table_lengths(c) if f > 0)
        n_pages = held + need + 7
        T = sum(max(f, 0) for _, f in _table_lengths(c)) + 3
        perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        hp = (cached + page - 1) // page
        start = hp.cumsum(0) - hp
        col = torch.arange(max_pages, device="cuda")
        table = torch.where(col < hp[:, None], perm[(start[:, None] + col).clamp_(max=n_pages - 1)], -1).to(torch.int32)
        ring = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        head = int(seed) % n_pages
        free = n_pages - held
        ring[(head + torch.arange(free, device="cuda")) % n_pages] = perm[held:]
        return dict(c, cached=cached, fresh=fresh, table=table, ring=ring, held_most=held_most,
                    ring_in=torch.tensor([head, head + free], dtype=torch.int64, device="cuda"),
                    ring_out=torch.zeros(2, dtype=torch.int64, device="cuda"),
                    kv_len=torch.zeros(B, dtype=torch.int32, device="cuda"), cu=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
                    slot=torch.zeros(T, dtype=torch.int32, device="cuda"), pos=torch.zeros(T, dtype=torch.int32, device="cuda"),
                    seq=torch.zeros(T, dtype=torch.int32, device="cuda"))
    n_q, n_kv, d = HEADS[c["heads"]]
    c.update(n_q=n_q, n_kv=n_kv, d=d)
    if c["op"] == "rope":
        T = c["T"]
        sections = _sections(c["axes"], d // 2)
        axis = torch.tensor(_axis_of(sections, c["interleaved"]), device="cuda")
        base = int(seed) % 30000
        along = torch.arange(T, device="cuda", dtype=torch.int32)
        # text runs along every axis; inside an image of 64 columns height and width go their own way
        axes = [base + along, base + along // 64, base + along % 64][: c["axes"]]
        gq, gk = (1 + 0.1 * torch.randn(2, d, generator=g, device="cuda")).unbind(0)
        return dict(c, qkv=torch.randn(T, (n_q + 2 * n_kv) * d, generator=g, device="cuda"), pos=torch.stack(axes).contiguous(),
                    gamma_q=gq.contiguous() if c["norm"] else None, gamma_k=gk.contiguous() if c["norm"] else None,
                    sections=sections, axis=axis, theta=1e6, out=torch.zeros(T, (n_q + n_kv) * d, device="cuda"))
    if c["op"] == "append":
        T, page = c["T"], c["page"]
        n_pages = _pages(T, page) + 5
        qkv = torch.randn(T, (n_q + 2 * n_kv) * d, generator=g, device="cuda")
        qkv *= torch.exp(0.4 * torch.randn((n_q + 2 * n_kv) * d, generator=g, device="cuda"))
        pages = torch.randperm(n_pages, generator=g, device="cuda")
        at = torch.arange(T, device="cuda") + int(seed) % page
        slot = (pages[at // page] * page + at % page).to(torch.int32)
        kv = torch.zeros(2, T, n_kv * d, device="cuda")
        return dict(c, k=qkv[:, n_q * d:(n_q + n_kv) * d], v=qkv[:, (n_q + n_kv) * d:], slot=slot,
                    pool=_pool(n_pages, page, n_kv, d, g), out_k=kv[0], out_v=kv[1])
    B, page = c["B"], c["page"]
    lens = torch.tensor(list(zip(*_attn_lengths(c))), dtype=torch.int32, device="cuda")
    lens = lens[torch.randperm(B, generator=g, device="cuda")]
    kv_len, fresh = lens[:, 0].contiguous(), lens[:, 1].contiguous()
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1:] = fresh.cumsum(0)
    total, new = _attn_lengths(c)
    T = sum(new)
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), fresh.long(), output_size=T)
    held = (kv_len + page - 1) // page
    n_pages = sum(_pages(x, page) for x in total) + 9
    max_pages = _pages(max(total), page)
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    start = held.cumsum(0) - held
    col = torch.arange(max_pages, device="cuda")
    table = torch.where(col < held[:, None], perm[(start[:, None] + col).clamp_(max=n_pages - 1)], -1).to(torch.int32)
    return dict(c, kv_len=kv_len, cu=cu, seq=seq, table=table, most=max(new), scale=d ** -0.5,
                q=2 * torch.randn(T, n_q * d, generator=g, device="cuda"), out=torch.zeros(T, n_q * d, device="cuda"),
                pool=_pool(n_pages, page, n_kv, d, g), scratch=torch.empty(SCRATCH, dtype=torch.uint8, device="cuda"))


# ---- the plain form -----------------------------------------------------------------------------


def _tables_plain(s):
    page, table, ring = s["page"], s["table"], s["ring"]
    cached, fresh = s["cached"].long(), s["fresh"].long()
    B, max_pages = table.shape
    n_pages, T = ring.numel(), s["slot"].numel()
    head, tail = s["ring_in"][0], s["ring_in"][1]
    held = (cached + page - 1) // page
    valid = (cached >= 0) & (fresh >= -1) & (cached + fresh.clamp(min=0) <= max_pages * page)
    ends = valid & (fresh == -1)
    wants = torch.where(valid, fresh.clamp(min=0), 0)
    fits = valid & ((wants == 0) | (wants.cumsum(0) <= T))
    need = torch.where(fits & ~ends, (cached + wants + page - 1) // page - held, 0)
    taken = fits & ((need == 0) | (need.cumsum(0) <= tail - head))
    n = torch.where(taken, wants, 0)
    need = torch.where(taken, need, 0)
    first = need.cumsum(0) - need
    col = torch.arange(max_pages, device=table.device)
    k = col - held[:, None]
    new = ring[(head + first[:, None] + k) % n_pages]
    table = torch.where((k >= 0) & (k < need[:, None]), new, table)
    back = torch.where(ends, held, 0)
    at = (tail + (back.cumsum(0) - back)[:, None] + col) % n_pages
    at = torch.where(col < back[:, None], at, n_pages)
    ring = torch.cat([ring, ring[:1]]).scatter(0, at.reshape(-1), table.reshape(-1))[:n_pages]
    cu = torch.zeros(B + 1, dtype=torch.int64, device=table.device)
    cu[1:] = n.cumsum(0)
    t = torch.arange(T, device=table.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    real = seq < B
    b = seq.clamp(max=B - 1)
    pos = cached[b] + t - cu[b]
    slot = table[b, (pos // page).clamp(0, max_pages - 1)] * page + pos % page
    ring_out = torch.stack([head + need.sum(), tail + back.sum()])
    kv_len = torch.where(ends, 0, cached + n)
    minus = torch.full_like(t, -1)
    return [table, ring, ring_out] + [x.to(torch.int32) for x in (kv_len, cu, torch.where(real, slot, minus), torch.where(real, pos, minus),
                                                                 torch.where(real, seq, minus))]


def _rope_plain(s):
    n_q, n_kv, d, half = s["n_q"], s["n_kv"], s["d"], s["d"] // 2
    x = s["qkv"][:, :(n_q + n_kv) * d].reshape(-1, n_q + n_kv, d)
    if s["norm"]:
        gamma = torch.cat([s["gamma_q"].expand(n_q, d), s["gamma_k"].expand(n_kv, d)])
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma
    i = torch.arange(half, device=x.device, dtype=torch.float64)
    angle = s["pos"][s["axis"]].double().T * s["theta"] ** (-i / half)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).reshape(x.shape[0], -1)


def _append_plain(s):
    n_kv, d, page, pool = s["n_kv"], s["d"], s["page"], s["pool"]
    nb = d // 32
    T = s["slot"].numel()
    x = torch.stack([s["k"].reshape(T, n_kv, nb, 32), s["v"].reshape(T, n_kv, nb, 32)], 2)   # [T][n_kv][2][nb][32]
    at = x.abs().argmax(-1, keepdim=True)
    scale = (x.gather(-1, at) * -0.125).clamp(-65504, 65504).half()
    ratio = x.double() / scale.double()                                # next to a border 32 bits decide wrongly
    code = torch.where(scale == 0, 8, (8 + torch.round(ratio)).clamp(0, 15)).to(torch.uint8)
    codes = code[..., :16] | (code[..., 16:] << 4)                     # [T][n_kv][2][nb][16]
    tiles = pool.view(-1, n_kv, page // 16, 18 * d)
    body = tiles[..., :16 * d].unflatten(-1, (2, nb, 16, 16))
    scales = tiles[..., 16 * d:].unflatten(-1, (2, nb, 16, 2))
    slot = s["slot"].long()
    p, tile, row = slot // page, slot % page // 16, slot % 16
    body[p, :, tile, :, :, row] = codes
    scales[p, :, tile, :, :, row] = scale.view(torch.uint8)
    # and back
    got = body[p, :, tile, :, :, row]
    code = torch.cat([got & 15, got >> 4], -1)
    back = (code.float() - 8) * scales[p, :, tile, :, :, row].contiguous().view(torch.float16).float()
    return [back[:, :, 0].reshape(T, n_kv * d), back[:, :, 1].reshape(T, n_kv * d)]


def _attn_plain(s):
    n_q, n_kv, d, page = s["n_q"], s["n_kv"], s["d"], s["page"]
    B, max_pages = s["table"].shape
    G, nb, S = n_q // n_kv, d // 32, max_pages * page
    tiles = s["pool"].view(-1, n_kv, page // 16, 18 * d)[s["table"].clamp(min=0).long()]   # [B][pages][n_kv][page/16][18 d]
    tiles = tiles.transpose(1, 2).reshape(B, n_kv, S // 16, 18 * d)
    body = tiles[..., :16 * d].unflatten(-1, (2, nb, 16, 16))
    scale = tiles[..., 16 * d:].contiguous().view(torch.float16).unflatten(-1, (2, nb, 16, 1)).float()
    x = torch.cat([body & 15, body >> 4], -1).float().sub_(8).mul_(scale)                  # [B][n_kv][S/16][2][nb][16][32]
    x = x.permute(3, 0, 1, 2, 5, 4, 6).reshape(2, B, n_kv, S, d)
    most = s["most"]
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(most, device=n.device)
    row = (s["cu"][:-1].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].view(B, most, n_kv, G, d).transpose(1, 2).reshape(B, n_kv, most * G, d)
    w = torch.matmul(q, x[0].transpose(-1, -2)).mul_(s["scale"]).view(B, n_kv, most, G, S)
    p = (s["kv_len"].long() - n)[:, None] + i
    j = torch.arange(S, device=n.device)
    seen = j <= p[..., None]
    if s["window"]:
        seen &= j > p[..., None] - s["window"]
    w = w.masked_fill_(~seen[:, None, :, None], -torch.inf)
    w = (w - w.amax(-1, keepdim=True)).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(B, n_kv, most * G, S), x[1]).view(B, n_kv, most, G, d) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(B, most, n_q * d)
    t = torch.arange(s["q"].shape[0], device=n.device)
    return o[s["seq"], t - s["cu"][s["seq"]]]


# ---- one pass -----------------------------------------------------------------------------------


def run(s):
    op = s["op"]
    if not own:
        return {"tables": _tables_plain, "rope": _rope_plain, "append": _append_plain, "attn": _attn_plain}[op](s)
    import q4_gemv_gqa_gb300 as gem
    if op == "tables":
        gem.kv_block_tables(s["cached"], s["fresh"], s["page"], s["table"], s["ring"], s["ring_in"], s["ring_out"],
                            s["kv_len"], s["cu"], s["slot"], s["pos"], s["seq"])
        return [s["table"], s["ring"], s["ring_out"], s["kv_len"], s["cu"], s["slot"], s["pos"], s["seq"]]
    if op == "rope":
        return gem.qknorm_mrope(s["qkv"], s["n_q"], s["n_kv"], s["d"], s["gamma_q"], s["gamma_k"], EPS, s["pos"],
                                s["sections"], s["theta"], s["out"], interleaved=s["interleaved"])
    if op == "append":
        gem.kv4_append(s["k"], s["v"], s["n_kv"], s["d"], s["slot"], s["pool"], s["page"])
        gem.kv4_gather(s["pool"], s["page"], s["n_kv"], s["d"], s["slot"], s["out_k"], s["out_v"])
        return [s["out_k"], s["out_v"]]
    return gem.kv4_attn(s["q"], s["n_q"], s["n_kv"], s["d"], s["cu"], s["kv_len"], s["table"], s["pool"], s["page"],
                        s["window"], s["scale"], s["out"], workspace=s["scratch"])


def work(case):
    c = case
    if c["op"] == "tables":
        lens = _table_lengths(c)
        T = sum(max(f, 0) for _, f in lens) + 3
        new = sum(_pages(x + f, c["page"]) - _pages(x, c["page"]) for x, f in lens if f > 0)
        back = sum(_pages(x, c["page"]) for x, f in lens if f < 0)
        return {"bytes": 16 * c["B"] + 12 * T + 8 * (new + back) + 32, "flops": 0}
    n_q, n_kv, d = HEADS[c["heads"]]
    if c["op"] == "rope":
        n = c["T"] * (n_q + n_kv) * d
        return {"bytes": 8 * n + 4 * c["T"] * c["axes"], "flops": n * (7 if c["norm"] else 3)}
    if c["op"] == "append":
        n = 2 * c["T"] * n_kv * d
        # rows in, codes and scales out and in again, values out
        return {"bytes": n * (4 + 2 * 0.5625 + 4) + 8 * c["T"], "flops": 4 * n}
    rows, read, pairs = 0, 0, 0
    for total, new in zip(*_attn_lengths(c)):
        first = max(0, total - new + 1 - c["window"]) if c["window"] else 0
        rows += new
        read += total - first
        pairs += sum(min(total - new + i + 1, c["window"] or total) for i in range(new))
    return {"bytes": read * n_kv * d * 1.125 + 8 * rows * n_q * d, "flops": 4 * pairs * n_q * d}


# ---- 64 bits ------------------------------------------------------------------------------------


def _exact_tables(s):
    page = s["page"]
    cached, fresh, ring, table = (s[k].tolist() for k in ("cached", "fresh", "ring", "table"))
    head, tail = s["ring_in"].tolist()
    n_pages, T, wide = len(ring), s["slot"].numel(), len(table[0])
    popped = pushed = wanted = asked = 0
    given, cu, kv_len = [], [0], []
    for b, (c, f) in enumerate(zip(cached, fresh)):
        ok = c >= 0 and f >= -1 and c + max(f, 0) <= wide * page
        taken = 0
        if ok and f == -1:
            given += table[b][:_pages(c, page)]
        elif ok:
            wanted += f
            if f == 0 or wanted <= T:
                need = _pages(c + f, page) - _pages(c, page)
                asked += need
                if need == 0 or asked <= tail - head:
                    for k in range(need):
                        table[b][_pages(c, page) + k] = ring[(head + popped + k) % n_pages]
                    popped += need
                    taken = f
        cu.append(cu[-1] + taken)
        kv_len.append(0 if ok and f == -1 else c + taken)
    for k, x in enumerate(given):
        ring[(tail + k) % n_pages] = x
    pushed = len(given)
    slot, pos, seq = ([-1] * T for _ in range(3))
    for b, c in enumerate(cached):
        for i in range(cu[b + 1] - cu[b]):
            t, p = cu[b] + i, c + i
            slot[t], pos[t], seq[t] = table[b][p // page] * page + p % page, p, b
    i32 = torch.int32
    return [torch.tensor(table, dtype=i32), torch.tensor(ring, dtype=i32), torch.tensor([head + popped, tail + pushed])] + [
        torch.tensor(x, dtype=i32) for x in (kv_len, cu, slot, pos, seq)]


def _exact_rope(s):
    d, half, T = s["d"], s["d"] // 2, s["T"]
    out = []
    for h in range(s["n_q"] + s["n_kv"]):
        x = s["qkv"][:, h * d:(h + 1) * d].double()
        gamma = s["gamma_q"] if h < s["n_q"] else s["gamma_k"]
        if gamma is not None:
            x = x * (x.pow(2).sum(1) / d + EPS).rsqrt()[:, None] * gamma.double()
        y = torch.empty_like(x)
        for i in range(half):
            a = s["pos"][int(s["axis"][i])].double() * math.pow(s["theta"], -2.0 * i / d)
            y[:, i] = x[:, i] * torch.cos(a) - x[:, i + half] * torch.sin(a)
            y[:, i + half] = x[:, i] * torch.sin(a) + x[:, i + half] * torch.cos(a)
        out.append(y)
    return torch.cat(out, 1).view(T, -1)


def _exact_append(s):
    got = []
    for x in (s["k"], s["v"]):
        x = x.double().reshape(-1, 32)
        big = x.abs().max(1, keepdim=True)
        m = torch.gather(x, 1, big.indices)
        scale = (m / -8).clamp(-65504, 65504).half().double()
        y = torch.where(scale != 0, x / scale, 0.0)
        low = torch.floor(y)
        part = y - low
        up = (part > 0.5) | ((part == 0.5) & (torch.remainder(low, 2) == 1))
        got.append(((low + up).clamp(-8, 7) * scale).view(s["slot"].numel(), -1))
    return got


def _exact_attn(s):
    n_q, n_kv, d, page = s["n_q"], s["n_kv"], s["d"], s["page"]
    G = n_q // n_kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    cu, kv_len = s["cu"].tolist(), s["kv_len"].tolist()
    for b, L in enumerate(kv_len):
        pages = s["table"][b, :_pages(L, page)].long()
        n = cu[b + 1] - cu[b]
        for h in range(n_kv):
            t = s["pool"].view(-1, n_kv, page // 16, 18 * d)[pages, h].reshape(-1, 18 * d)   # tiles in order
            both = []
            for which in range(2):
                c = t[:, which * 8 * d:(which + 1) * 8 * d].reshape(-1, d // 32, 16, 16).int()
                f = t[:, 16 * d + which * d:16 * d + (which + 1) * d].contiguous().view(torch.float16).view(-1, d // 32, 16).double()
                v = torch.empty(t.shape[0], d // 32, 16, 32, dtype=torch.float64, device="cuda")
                v[..., :16] = (c % 16 - 8) * f[..., None]
                v[..., 16:] = (c // 16 - 8) * f[..., None]
                both.append(v.transpose(1, 2).reshape(-1, d)[:L])
            q = s["q"][cu[b]:cu[b + 1], h * G * d:(h + 1) * G * d].double().view(n, G, d)
            w = torch.einsum("ngd,ld->ngl", q, both[0]) * s["scale"]
            p = torch.arange(L - n, L, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")[None]
            hidden = (j > p) | (j <= p - s["window"] if s["window"] else j < 0)
            w = torch.softmax(w.masked_fill(hidden[:, None], -torch.inf), -1)
            out[cu[b]:cu[b + 1], h * G * d:(h + 1) * G * d] = torch.einsum("ngl,ld->ngd", w, both[1]).reshape(n, G * d)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "rope": _exact_rope, "append": _exact_append, "attn": _exact_attn}[s["op"]](s)
