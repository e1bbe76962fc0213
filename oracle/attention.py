"""Plain fp64 statements of the cache append and of attention over the cache.

Test infrastructure, as the rest of the oracle: numpy, loops, no code shared
with the CUDA path.  `rows(cache, table, page, s, n)` is the first n tokens of
a sequence in a paged cache; everything else is written from the definitions
of misa_cache_append, misa_attention and misa_attention_selected.
"""
import numpy as np


def rows(cache, table_row, n):
    """[n, heads, dim]: tokens 0..n-1 of the sequence whose page-table row is given."""
    page = cache.shape[1]
    return np.stack([cache[table_row[p // page], p % page] for p in range(n)]) if n else cache[:0, 0]


def rotate(x, cos, sin, interleaved):
    """x [heads, dim] turned by one position's cosines and sines (fp64)."""
    y = np.array(x, np.float64)
    half = len(cos)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        u, v = x[:, a].astype(np.float64), x[:, b].astype(np.float64)
        y[:, a] = u * cos[i] - v * sin[i]
        y[:, b] = v * cos[i] + u * sin[i]
    return y


def attend(q, k, v, pos, token, scale, softcap=0.0, slopes=None):
    """One query over the tokens given: q [Hq, D], k, v [n, Hkv, D], their
    positions token [n] (all <= pos).  Returns out [Hq, D], lse [Hq], and for
    error bounds: spread [Hq, D] = sum p |v|, reach [Hq] = max_s sum_d |q k|,
    top [Hq] = max |x|."""
    hq, d = q.shape
    grp = hq // k.shape[1]
    out, spread = np.zeros((hq, d)), np.zeros((hq, d))
    lse, reach, top = np.full(hq, -np.inf), np.zeros(hq), np.zeros(hq)
    if len(token) == 0:
        return out, lse, spread, reach, top
    q, k, v = q.astype(np.float64), k.astype(np.float64), v.astype(np.float64)
    for h in range(hq):
        kh, vh = k[:, h // grp], v[:, h // grp]
        x = kh @ q[h] * scale
        if softcap:
            x = softcap * np.tanh(x / softcap)
        if slopes is not None:
            x = x - slopes[h] * (pos - np.asarray(token, np.float64))
        m = x.max()
        e = np.exp(x - m)
        p = e / e.sum()
        out[h], lse[h] = p @ vh, m + np.log(e.sum())
        spread[h] = p @ np.abs(vh)
        reach[h] = (np.abs(kh) @ np.abs(q[h])).max() * abs(scale)
        top[h] = np.abs(x).max()
    return out, lse, spread, reach, top
