"""Oracle of the paged 4-bit KV cache: numpy in 64 bits, one request, head and token at a time.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

TILE = 16


def page_bytes(n_kv: int, d: int, page: int) -> int:
    return n_kv * page * (d + d // 32 * 4)   # two rows of d / 2 bytes of codes and d / 32 binary16 scales


def quantise(x):
    """Blocks of 32 along the last axis of x (fp32) -> (codes uint8 [..., 32], scales float16 [...])."""
    x = np.asarray(x, np.float32)
    b = x.reshape(-1, 32).astype(np.float64)
    codes = np.full(b.shape, 8, np.uint8)
    scales = np.zeros(len(b), np.float16)
    for i, row in enumerate(b):
        if not np.all(np.isfinite(row)):
            scales[i] = np.float16(np.nan)
            continue
        m = row[np.argmax(np.abs(row))]     # the first of equal ones
        scales[i] = np.float16(np.clip(m / -8.0, -65504.0, 65504.0))
        s = float(scales[i])
        if s != 0.0:
            # a quotient in 64 bits is on a border exactly where the value is (32-bit values, 11-bit scales)
            codes[i] = np.clip(8 + np.rint(row / s), 0, 15).astype(np.uint8)
    shape = x.shape[:-1] + (x.shape[-1] // 32,)
    return codes.reshape(shape + (32,)), scales.reshape(shape)


def values(codes, scales):
    s = scales.astype(np.float64)[..., None]
    v = (codes.astype(np.float64) - 8.0) * s
    return v.reshape(v.shape[:-2] + (-1,))


class Pool:
    """The pool's bytes and where a (slot, head) row lies in them."""

    def __init__(self, n_pages: int, page: int, n_kv: int, d: int, fill: int = 0):
        self.page, self.n_kv, self.d, self.nb = page, n_kv, d, d // 32
        self.bytes = np.full((n_pages, page_bytes(n_kv, d, page)), fill, np.uint8)

    def _at(self, slot, head, which, blk):
        page, row = divmod(int(slot), self.page)
        tile, row = divmod(row, TILE)
        base = (head * (self.page // TILE) + tile) * 18 * self.d
        code = base + (which * self.nb + blk) * TILE * 16 + row * 16
        scale = base + 16 * self.d + ((which * self.nb + blk) * TILE + row) * 2
        return page, code, scale

    def write(self, slot, head, which, codes, scales):
        for blk in range(self.nb):
            p, c, s = self._at(slot, head, which, blk)
            self.bytes[p, c:c + 16] = codes[blk, :16] | (codes[blk, 16:] << 4)
            self.bytes[p, s:s + 2] = scales[blk:blk + 1].view(np.uint8)

    def read(self, slot, head, which):
        out = np.empty((self.nb, 32))
        for blk in range(self.nb):
            p, c, s = self._at(slot, head, which, blk)
            raw = self.bytes[p, c:c + 16]
            scale = float(self.bytes[p, s:s + 2].copy().view(np.float16)[0])
            out[blk] = (np.concatenate([raw & 15, raw >> 4]).astype(np.float64) - 8.0) * scale
        return out.reshape(-1)

    def append(self, k, v, slots):
        for which, x in enumerate((k, v)):
            codes, scales = quantise(np.asarray(x, np.float32).reshape(len(slots), self.n_kv, self.d))
            for t, s in enumerate(slots):
                if 0 <= s < self.bytes.shape[0] * self.page:
                    for h in range(self.n_kv):
                        self.write(s, h, which, codes[t, h], scales[t, h])

    def rows(self, slots, which):
        return np.stack([np.concatenate([self.read(s, h, which) for h in range(self.n_kv)]) for s in slots])


def block_tables(cached, fresh, page, table, ring, ring_in, T_cap):
    """-> dict(table, ring, ring_out, kv_len, cu, slot, pos, seq, refused)."""
    table, ring = np.array(table, np.int32), np.array(ring, np.int32)
    n_pages, wide = len(ring), table.shape[1]
    head, tail = (int(x) for x in ring_in)
    free = tail - head
    bad = head < 0 or not 0 <= free <= n_pages
    room = n_pages - free
    if bad:
        free = room = 0
    ceil = lambda n: -(-n // page)  # noqa: E731
    wants = asked = popped = back_asked = 0
    given, kv_len, cu, refused = [], [], [0], []
    for b in range(len(cached)):
        c, f = int(cached[b]), int(fresh[b])
        ok = c >= 0 and f >= -1 and c + max(f, 0) <= wide * page
        taken = 0
        if ok and f == -1:
            back_asked += ceil(c)
            ok = ceil(c) == 0 or back_asked <= room
            if ok:
                given += list(table[b, :ceil(c)])
        elif ok:
            wants += f
            ok = f == 0 or wants <= T_cap
            if ok:
                need = ceil(c + f) - ceil(c)
                asked += need
                ok = need == 0 or asked <= free
                if ok:
                    for i in range(need):
                        table[b, ceil(c) + i] = ring[(head + popped + i) % n_pages]
                    popped += need
                    taken = f
        if not ok:
            refused.append(b)
        kv_len.append(0 if ok and f == -1 else c + taken)
        cu.append(cu[-1] + taken)
    for i, x in enumerate(given):
        ring[(tail + i) % n_pages] = x
    slot, pos, seq = (np.full(T_cap, -1, np.int32) for _ in range(3))
    for b in range(len(cached)):
        for i in range(cu[b + 1] - cu[b]):
            p = int(cached[b]) + i
            id_ = int(table[b, p // page])
            slot[cu[b] + i] = id_ * page + p % page if 0 <= id_ < n_pages else -2 ** 31
            pos[cu[b] + i], seq[cu[b] + i] = p, b
    return dict(table=table, ring=ring, ring_out=np.array([head + popped, tail + len(given)], np.int64),
                kv_len=np.array(kv_len, np.int32), cu=np.array(cu, np.int32), slot=slot, pos=pos, seq=seq,
                refused=refused, bad_ring=bad)


def axis_of(sections, interleaved):
    n, half = len(sections), sum(sections)
    axis = np.zeros(half, int)
    if interleaved:
        for a in range(1, n):
            axis[a:a + n * sections[a]:n][:sections[a]] = a
    else:
        axis = np.repeat(np.arange(n), sections)
    return axis


def qknorm_mrope(qkv, n_q, n_kv, d, gamma_q, gamma_k, eps, pos, sections, theta, interleaved=False):
    """[T][(n_q + n_kv) * d] in 64 bits."""
    T, half = len(qkv), sum(sections)
    theta = float(np.float32(theta))   # the library takes the base in 32 bits
    freq = theta ** (-np.arange(half) / half)
    ang = np.asarray(pos, np.float64)[axis_of(sections, interleaved)].T * freq     # [T][half]
    c, s = np.cos(ang), np.sin(ang)
    out = np.empty((T, n_q + n_kv, d))
    for h in range(n_q + n_kv):
        x = np.asarray(qkv[:, h * d:(h + 1) * d], np.float64)
        g = gamma_q if h < n_q else gamma_k
        if g is not None:
            x = x / np.sqrt((x * x).mean(1, keepdims=True) + float(np.float32(eps))) * np.asarray(g, np.float64)
        out[:, h] = x
        out[:, h, :half] = x[:, :half] * c - x[:, half:2 * half] * s
        out[:, h, half:2 * half] = x[:, :half] * s + x[:, half:2 * half] * c
    return out.reshape(T, -1)


def attention(q, k, v, kv_len, window, scale):
    """One request: q [n][n_q][d], k, v [kv_len][n_kv][d] -> [n][n_q][d] in 64 bits."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, n_q, d = q.shape
    G = n_q // k.shape[1]
    out = np.zeros((n, n_q, d))
    for i in range(n):
        p = kv_len - n + i
        lo = max(0, p - window + 1) if window else 0
        for h in range(n_q):
            s = float(np.float32(scale)) * (k[lo:p + 1, h // G] @ q[i, h])
            w = np.exp(s - s.max())
            out[i, h] = (w / w.sum()) @ v[lo:p + 1, h // G]
    return out
