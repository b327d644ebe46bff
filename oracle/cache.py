"""Plain 64-bit forms of the paged cache and the attention over it (test
infrastructure only): numpy binary64 from the definitions, one token and one
head at a time.  Nothing is shared with the product.

A cache is held as arrays [pages, page, heads, dim] of values.
"""
from __future__ import annotations

import numpy as np


def places(lengths, queries, pages, page, count):
    """(token row, page, slot) of every token of a step that has a place."""
    out = []
    for b, length in enumerate(lengths):
        for i in range(queries):
            t = int(length) - queries + i
            if t < 0 or t // page >= pages.shape[1]:
                continue
            p = int(pages[b, t // page])
            if 0 <= p < count:
                out.append((b * queries + i, p, t % page))
    return out


def tokens(table, count, page, pages):
    """(page, slot) of the first `count` tokens that lie on a page there is."""
    t = np.arange(min(count, len(table) * page))
    p = np.asarray(table, dtype=np.int64)[t // page] if len(t) else np.zeros(0, np.int64)
    there = (p >= 0) & (p < pages)
    return p[there], (t % page)[there], t[there]


def attention(q, k, v, scale, prefix, prefix_pages, lengths, pages, queries):
    """(out, lse, sum w |v|, most |scale q.k|, sum |q||k| at most) in binary64,
    rows [sequences * queries, heads, ...]; rows of sequences that are not
    there are NaN."""
    count, page, kv, dim = k.shape
    rows, heads, _ = q.shape
    group = heads // kv
    out = np.full((rows, heads, dim), np.nan)
    lse = np.full((rows, heads), np.nan)
    size = np.zeros((rows, heads, dim))
    top = np.zeros((rows, heads))
    mass = np.zeros((rows, heads))
    sp, ss, _ = tokens(prefix_pages, prefix, page, count)
    for b, length in enumerate(lengths):
        if length < 0:
            continue
        op, os_, ot = tokens(pages[b], int(length), page, count)
        for i in range(queries):
            seen = ot < int(length) - queries + 1 + i
            p, s = np.concatenate((sp, op[seen])), np.concatenate((ss, os_[seen]))
            r = b * queries + i
            for h in range(heads):
                kk, vv = k[p, s, h // group], v[p, s, h // group]
                if not len(p):
                    out[r, h], lse[r, h] = 0.0, -np.inf
                    continue
                sc = kk @ q[r, h] * scale
                m = sc.max()
                w = np.exp(sc - m)
                l = w.sum()
                out[r, h], lse[r, h] = w @ vv / l, m + np.log(l)
                size[r, h] = w @ np.abs(vv) / l
                top[r, h] = np.abs(sc).max()
                mass[r, h] = (np.abs(kk) @ np.abs(q[r, h])).max() * scale
    return out, lse, size, top, mass
