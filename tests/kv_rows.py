"""Attention over the 8-bit cache in float64 with a bound for each row from the keys that this row sees, and from no
others: what a row does not see may be of any size."""
import numpy as np

from oracle import kv_cache as ora


def expected_rows(b, q, kc, ks, vc, vs, causal, scale):
    """(O [n, H, D], lse [H, n], bound of O [n, H, D], bound of lse [H, n]).

    A score is a sum of up to 128 products in fp32, scaled: at most 12 roundings of up to a whole step, 2^-23, of
    S_j = scale * sum |q_d k_jd|; the exponential adds 2^-20 of its result.  So weight p_j is off by
    d_j = 12 * 2^-23 * S_j + 2^-20 of itself, and by 2^-11 more where it is rounded to fp16 for the second product.
    O = sum p_j v_j, numerator and denominator off by as much: 2 sum_j p_j (2^-11 + d_j) (|v_j| + |O|), and by its
    rounding to bf16, 2^-8 |O| (a whole step, for results that fall on the other side of a border).  Weights times the
    scale of their block have a least step of 2^-25 of the largest such product of the row (a block's values are at
    most 448 scales): n steps of it.  lse is off by 2 sum_j p_j d_j and the fp32 roundings of its own magnitude.
    """
    out, lse = np.zeros((b.n, b.H, b.D)), np.full((b.H, b.n), -np.inf)
    tol, tol_lse = np.zeros((b.n, b.H, b.D)), np.zeros((b.H, b.n))
    group = b.H // b.Hkv
    for s in range(len(b.q)):
        if b.q[s] == 0 or b.lens[s] == 0:
            continue
        k, v = ora.values(kc, ks, b.table[s], b.lens[s]), ora.values(vc, vs, b.table[s], b.lens[s])
        page = b.table[s][np.arange(b.lens[s]) // b.ps]
        block = 448.0 * 2.0 ** (vs[page].astype(np.float64) - 127)  # [len, H_kv]
        for i in range(b.q[s]):
            t = b.cu[s] + i
            end = max(0, min(b.lens[s], b.lens[s] - b.q[s] + i + 1)) if causal else b.lens[s]
            if end == 0:
                continue
            for h in range(b.H):
                g = h // group
                x = scale * (k[:end, g] @ q[t, h])
                size = scale * (np.abs(k[:end, g]) @ np.abs(q[t, h]))
                m = x.max()
                w = np.exp(x - m)
                p = w / w.sum()
                o = p @ v[:end, g]
                d = 12 * 2.0 ** -23 * size + 2.0 ** -20
                out[t, h], lse[h, t] = o, m + np.log(w.sum())
                each = p * (2.0 ** -11 + d)
                tol[t, h] = 2.0 ** -8 * np.abs(o) + 2 * (each @ np.abs(v[:end, g]) + each.sum() * np.abs(o)) + \
                    end * 2.0 ** -25 * (p * block[:end, g]).max()
                tol_lse[h, t] = 2 * (p @ d) + 2.0 ** -20 + 2.0 ** -22 * abs(lse[h, t])
    return out, lse, tol, tol_lse


def check_rows(got, lse_got, want, lse_want, tol, tol_lse):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), got[bad][:5], want[bad][:5])
    seen = np.isfinite(lse_want)
    assert np.array_equal(lse_got[~seen], lse_want[~seen])
    bad = ~(np.abs(lse_got[seen] - lse_want[seen]) <= tol_lse[seen])
    assert not bad.any(), (lse_got[seen][bad][:5], lse_want[seen][bad][:5])
