"""The 8-bit paged key/value cache in float64: append with rotation, and attention over it.

Written from the definition, one element at a time where that is clearest.  Codes are
e4m3 bytes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN,
there is no infinity.  A block (one page, one kv head) has one scale byte b and a code
c stands for c * 2^(b - 127).
"""
from __future__ import annotations

import numpy as np

MAX = 448.0


def _table():
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = np.nan if c & 127 == 127 else (-mag if c & 128 else mag)
    return t


TABLE = _table()
GRID = TABLE[:127]  # the magnitudes in order; a code is its own index


def encode(x):
    """Codes of x: nearest, ties to the even code, beyond the largest to the largest, NaN to NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), MAX)
    hi = np.clip(np.searchsorted(GRID, a), 1, 126)
    lo = hi - 1
    up, down = a - GRID[lo], GRID[hi] - a
    code = np.where((down < up) | ((down == up) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_byte(amax):
    """The least byte b with amax <= 448 * 2^(b - 127)."""
    b = 0
    while amax > MAX * 2.0 ** (b - 127):
        b += 1
    return b


def rotate(x, pos, cos, sin, interleaved):
    """x [heads, D] at position pos, its first 2 * cos.shape[1] dims rotated."""
    y = np.array(x, dtype=np.float64)
    half = cos.shape[1]
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c, s = float(cos[pos, j]), float(sin[pos, j])
        y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return y


def append(codes, scales, rows, cu, lens, table):
    """Put rows [n, H_kv, D] (float64, rotated) into copies of codes [pages, H_kv, ps, D] and scales."""
    codes, scales = codes.copy(), scales.copy()
    ps = codes.shape[2]
    for s in range(len(lens)):
        n = cu[s + 1] - cu[s]
        start = lens[s] - n
        for j in range(start // ps, -(-lens[s] // ps) if n else 0):
            lo, hi, page = max(start, j * ps), min(lens[s], (j + 1) * ps), table[s][j]
            for h in range(codes.shape[1]):
                new = rows[cu[s] + lo - start:cu[s] + hi - start, h]
                finite = np.abs(new[np.isfinite(new)])
                need = scale_byte(finite.max() if finite.size else 0.0)
                old = int(scales[page, h]) if lo > j * ps else 0
                b = max(old, need)
                older = codes[page, h, :lo - j * ps]
                if b > old:
                    codes[page, h, :lo - j * ps] = encode(TABLE[older] * 2.0 ** (old - b))
                codes[page, h, lo - j * ps:hi - j * ps] = encode(new * 2.0 ** (127 - b))
                scales[page, h] = b
    return codes, scales


def values(codes, scales, table, length):
    """The cache's values of one sequence: [length, H_kv, D]."""
    ps = codes.shape[2]
    out = np.empty((length,) + (codes.shape[1], codes.shape[3]))
    for p in range(length):
        page = table[p // ps]
        scale = np.where(scales[page] == 255, np.nan, 2.0 ** (scales[page].astype(np.float64) - 127))
        out[p] = TABLE[codes[page, :, p % ps]] * scale[:, None]
    return out


def attention(q, k, v, causal, scale):
    """q [n, H, D] of the last n of len(k) tokens over k, v [len, H_kv, D]: (O [n, H, D], lse [H, n])."""
    n, H, D = q.shape
    group = H // k.shape[1]
    out, lse = np.zeros((n, H, D)), np.full((H, n), -np.inf)
    for i in range(n):
        end = max(0, min(len(k), len(k) - n + i + 1)) if causal else len(k)
        if end == 0:
            continue
        for h in range(H):
            s = scale * (k[:end, h // group] @ q[i, h])
            m = s.max()
            w = np.exp(s - m)
            out[i, h] = (w[:, None] * v[:end, h // group]).sum(0) / w.sum()
            lse[h, i] = m + np.log(w.sum())
    return out, lse
