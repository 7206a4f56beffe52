"""64-bit reference of the 8-bit floating-point path and of the scores (numpy), written from the formulas in
include/gem.h: e4m3 codes with a power-of-two scale for each 128 values, RMSNorm and the gated activation in
that form, the product with weights scaled by blocks of 128 x 128, and log probabilities of logit rows."""
from __future__ import annotations

import math

import numpy as np


def _table() -> np.ndarray:
    got = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        got[c] = math.nan if c & 127 == 127 else -v if c & 128 else v
    return got


VALUES = _table()                  # value of each code
_GRID = VALUES[:127]               # the positive ones, ascending
_MID = (_GRID[1:] + _GRID[:-1]) / 2


def encode(t: np.ndarray) -> np.ndarray:
    """Codes of finite values of at most 448 (+ half a step), to nearest, ties to the even code."""
    a = np.abs(t)
    low, high = np.searchsorted(_MID, a, "left"), np.searchsorted(_MID, a, "right")   # they differ on a border
    code = np.where((low != high) & (low % 2 == 0), low, high).astype(np.uint8)
    return code | (np.signbit(t).astype(np.uint8) << 7)


def quantise(y: np.ndarray):
    """(codes uint8 [T, H], scales float32 [T, ceil(H / 128)]) of 64-bit rows."""
    T, H = y.shape
    codes, scales = np.zeros((T, H), np.uint8), np.zeros((T, -(-H // 128)), np.float32)
    for b in range(scales.shape[1]):
        v = y[:, 128 * b:128 * b + 128]
        for t in range(T):
            m = np.max(np.abs(v[t]))
            if not m <= np.finfo(np.float32).max:
                scales[t, b] = np.nan
            elif m >= 2.0 ** -100:
                k = math.frexp(m)[1] - 10
                while m > math.ldexp(448.0, k):
                    k += 1
                scales[t, b] = math.ldexp(1.0, k)
                codes[t, 128 * b:128 * b + 128] = encode(v[t] * math.ldexp(1.0, -k))
    return codes, scales


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return VALUES[codes] * np.repeat(scales.astype(np.float64), 128, 1)[:, :codes.shape[1]]


def rmsnorm(x, residual, gamma, eps):
    """(h float32, y float64)"""
    h = x if residual is None else (x + residual).astype(np.float32)
    y = h.astype(np.float64)
    y = y / np.sqrt((y * y).mean(1, keepdims=True) + float(np.float32(eps)))
    return h, y if gamma is None else y * gamma.astype(np.float64)


def gated(x, up, act):
    x, up = x.astype(np.float64), up.astype(np.float64)
    z = x if act == 0 else 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    with np.errstate(over="ignore", invalid="ignore"):
        return np.where(z < -83, 0.0 * x * up, x * up / (1 + np.exp(-z)))


def gemm(W, ws, x, xs, residual=None):
    """(y, sum of the products' magnitudes), both float64 [M, N]."""
    N, K = W.shape
    w = VALUES[W] * np.repeat(np.repeat(ws.astype(np.float64), 128, 0)[:N], 128, 1)[:, :K]
    v = values(x, xs)
    y, most = v @ w.T, np.abs(v) @ np.abs(w).T
    return (y, most) if residual is None else (y + residual, most + np.abs(residual))


def order(row: np.ndarray) -> np.ndarray:
    """Indices of a row, larger values first, equal ones by index, NaN behind every number."""
    return np.lexsort((np.arange(row.size), -np.where(np.isnan(row), 0.0, row.astype(np.float64)), np.isnan(row)))


def scores(y, tokens, k, scale=1.0):
    """dict of logp, entropy, rank, idx, val, and spread = sum p |l - max|, for the rows of y."""
    T, N = y.shape
    got = dict(logp=np.zeros(T), entropy=np.zeros(T), rank=np.zeros(T, np.int32), idx=np.zeros((T, k), np.int32), val=np.zeros((T, k)),
               spread=np.zeros(T))
    for t in range(T):
        row = y[t].astype(np.float64)
        with np.errstate(invalid="ignore"):
            d = (row - row.max()) * scale
            e = np.exp(d)
            s = e.sum()
            lp = d - np.log(s)
            got["entropy"][t] = -np.sum(np.where(e > 0, e / s * np.where(e > 0, lp, 0), 0)) if np.isfinite(s) else np.nan
            got["spread"][t] = np.sum(np.where(e > 0, e / s * -np.where(e > 0, d, 0), 0))
        if not np.isfinite(s):
            lp = np.full(N, np.nan)
        at = order(y[t])
        got["idx"][t], got["val"][t] = at[:k], lp[at[:k]]
        n = int(tokens[t])
        if 0 <= n < N:
            got["logp"][t], got["rank"][t] = lp[n], 1 + int(np.flatnonzero(at == n)[0])
        elif n != -1:
            got["logp"][t] = np.nan
    return got
