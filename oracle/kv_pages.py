"""Pages of the 8-bit cache shared, copied, compacted, taken and given back: row by row, from the definitions."""
from __future__ import annotations

import numpy as np

from . import kv_cache


def _pages(n, ps):
    return -(-int(n) // ps)


def fork(table, lens, refs, parents, ps, table_out):
    """(table, lengths, refs, copies) after the fork, copies a list of (from, to, slots); None where pages do not suffice."""
    out, refs_out = table_out.copy(), refs.copy()
    free = [p for p in range(len(refs)) if refs[p] == 0]
    new_lens, copies, gone_on = [], [], set()
    for row, n in zip(table, lens):
        for p in row[:_pages(n, ps)]:
            refs_out[p] -= 1
    for o, b in enumerate(parents):
        if b < 0:
            new_lens.append(0)
            continue
        n = lens[b]
        row = list(table[b][:_pages(n, ps)])
        if n % ps and (b in gone_on or refs[row[-1]] != 1):
            if len(copies) == len(free):
                return None
            copies.append((int(row[-1]), free[len(copies)], int(n % ps)))
            row[-1] = copies[-1][1]
        gone_on.add(b)
        for p in row:
            refs_out[p] += 1
        out[o, :len(row)] = row
        new_lens.append(int(n))
    return out, np.array(new_lens, np.int32), refs_out, copies


def resize(table, lens, new_lens, refs, ps):
    """(table, refs) after the change of lengths; None where pages do not suffice."""
    table, out = table.copy(), refs.copy()
    free = [p for p in range(len(refs)) if refs[p] == 0]
    for s, (a, b) in enumerate(zip(lens, new_lens)):
        for i in range(_pages(a, ps), _pages(b, ps)):
            if not free:
                return None
            table[s, i] = free.pop(0)
            out[table[s, i]] += 1
        for i in range(_pages(b, ps), _pages(a, ps)):
            out[table[s, i]] -= 1
    return table, out


def copy_pages(codes, scales, copies):
    codes, scales = codes.copy(), scales.copy()
    for src, dst, n in copies:
        codes[dst, :, :n] = codes[src, :, :n]
        scales[dst] = scales[src]
    return codes, scales


def compact(codes, scales, kept, cu, lens, table):
    """(codes, scales, lengths): each sequence's kept new tokens behind its earlier ones."""
    codes, scales, new = codes.copy(), scales.copy(), []
    ps = codes.shape[2]
    for s, path in enumerate(kept):
        start = lens[s] - (cu[s + 1] - cu[s])
        at = lambda p: (table[s][p // ps], p % ps)
        was = [(codes[at(start + k)[0], :, at(start + k)[1]].copy(), scales[at(start + k)[0]].astype(int)) for k in path]
        new.append(start + len(path))
        for j in range(start // ps, _pages(new[-1], ps)):
            page, lo, hi = table[s][j], max(start, j * ps), min(new[-1], (j + 1) * ps)
            if lo >= hi:
                continue
            for h in range(codes.shape[1]):
                bytes_ = [was[t - start][1][h] for t in range(lo, hi)] + ([int(scales[page, h])] if lo > j * ps else [])
                b = max(bytes_)
                if lo > j * ps:
                    codes[page, h, :lo - j * ps] = _shifted(codes[page, h, :lo - j * ps], int(scales[page, h]), b)
                for t in range(lo, hi):
                    c, old = was[t - start]
                    codes[page, h, t - j * ps] = _shifted(c[h], int(old[h]), b)
                scales[page, h] = b
    return codes, scales, np.array(new, np.int32)


def _shifted(codes, old, new):
    if old == new or new == 255:
        return codes
    return kv_cache.encode(kv_cache.TABLE[codes] * 2.0 ** (old - new))
