"""The mixture-of-experts layer for a few tokens in float64 (test infrastructure only): selection from the
router's logits, gated experts, combine; and a bound of what fp32 sums may change.

Experts: W1[e] [H, 2 I] (gate columns, then up columns), W2[e] [I, Hd].  h = silu(x W1g) * (x W1u).
"""
from __future__ import annotations

import numpy as np


def select(logits, topk, normalize):
    """(ids [T, topk], gates): largest first, equal logits by index, NaN below every number."""
    T, E = logits.shape
    ids, gates = np.empty((T, topk), np.int32), np.zeros((T, topk))
    for t in range(T):
        rank = sorted(range(E), key=lambda e: (np.isnan(logits[t, e]), -np.nan_to_num(logits[t, e], nan=0.0), e))
        ids[t] = rank[:topk]
        over = logits[t, ids[t]] if normalize else logits[t]
        top = over.max()
        if top == -np.inf:
            continue
        with np.errstate(invalid="ignore"):
            gates[t] = np.exp(logits[t, ids[t]] - top) / np.exp(over - top).sum()
    return ids, gates


def layer(x, logits, W1, W2, topk, normalize):
    """(out [T, Hd], ids, gates, slack [T, Hd]): slack bounds the error of fp32 sums (a step of 2^-23 of the terms'
    magnitudes for each sixteen products and ten more) and of h in two bf16 terms (2^-16 of it)."""
    ids, gates = select(logits, topk, normalize)
    T, H = x.shape
    I, Hd = W2[0].shape
    out, slack = np.zeros((T, Hd)), np.zeros((T, Hd))
    c1, c2 = (H / 16 + 10) * 2.0 ** -23, (2 * I / 16 + topk + 10) * 2.0 ** -23
    for t in range(T):
        for s in range(topk):
            w1, w2 = W1[ids[t, s]], W2[ids[t, s]]
            z, mag = x[t] @ w1, np.abs(x[t]) @ np.abs(w1)
            g, u = z[:I], z[I:]
            silu = g / (1 + np.exp(-g))
            h = silu * u
            # silu's slope is at most 1.1; the exponential and the division are within 2^-20
            dh = np.abs(u) * 1.1 * c1 * mag[:I] + np.abs(silu) * c1 * mag[I:] + (2.0 ** -16 + 2.0 ** -20) * np.abs(h)
            y = h @ w2
            out[t] += gates[t, s] * y
            slack[t] += gates[t, s] * (dh @ np.abs(w2) + c2 * (np.abs(h) @ np.abs(w2)) + 2.0 ** -20 * np.abs(y))
    return out, ids, gates, slack
