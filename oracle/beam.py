"""Beam search's selection in float64: scores of every continuation, and the best of them in order."""
from __future__ import annotations

import numpy as np


def totals(logits, scores, done, eos):
    """(scores of all continuations [B, K, V], -inf where none is offered; lse [B, K], 0 for ended beams) of logits
    [B, K, V] and scores [B, K], float64."""
    x = np.asarray(logits, np.float64)
    with np.errstate(all="ignore"):
        m = x.max(2, keepdims=True)
        finite = np.isfinite(m)
        s = np.log(np.exp(x - np.where(finite, m, 0.0)).sum(2))
        lse = m[..., 0] + s
        lse = np.where(np.isnan(x).any(2), np.nan, np.where(np.isposinf(m[..., 0]), np.inf, lse))
        # x - lse as (x - m) - log s: m + log s has no room for log s where m is the lowest float
        total = scores[..., None] + ((x - m) - s[..., None])
    total = np.where(np.isfinite(lse)[..., None] & np.isfinite(total), total, -np.inf)
    if done is not None:
        ended = np.asarray(done) != 0
        total[ended] = -np.inf
        total[ended, eos] = np.where(np.isfinite(scores[ended]), scores[ended], -np.inf)
        lse = np.where(ended, 0.0, lse)
    return total, lse


def select(total, N):
    """For each user the N best (beam, token, score), equal ones by beam, then token; (-1, -1, -inf) for places left."""
    out = []
    for t in total:
        flat = t.ravel()
        order = np.lexsort((np.arange(flat.size), -flat))[:N]
        best = [(int(i) // t.shape[1], int(i) % t.shape[1], float(flat[i])) for i in order if flat[i] > -np.inf]
        out.append(best + [(-1, -1, -np.inf)] * (N - len(best)))
    return out
