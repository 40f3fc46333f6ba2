"""fp64 reference of the paged key-value cache's operators, one row and one position at a time.

Written from the definitions in include/lora_attn.h alone: inputs are plain float64 arrays (the values that
the stored types stand for), the loops follow the text, and nothing is shared with the GPU path.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def gather(pool, table, i, n):
    """The first n positions of sequence i, (n, heads, dim); a page number outside the pool gives NaN."""
    page_size = pool.shape[1]
    out = np.full((n,) + pool.shape[2:], np.nan)
    for p in range(n):
        page = int(table[i][p // page_size])
        if 0 <= page < pool.shape[0]:
            out[p] = pool[page, p % page_size]
    return out


def visible(t, length, window, sinks):
    """Positions that the row at position t sees, as a truth value each."""
    p = np.arange(length)
    seen = p <= t
    if window >= 0:
        seen &= (p > t - window) | (p < sinks)
    return seen


def attn(q, q_starts, kv_len, k_pool, v_pool, table, scale, window=-1, sinks=0):
    """dict of out (rows, heads, dim); mass (n_seq, kv_heads, max len), the weight each position got; and, for
    error bounds, absv = sum w |v|, sumv = sum |v| over seen positions, smax = the largest |q| . |k| * scale
    seen by a row, seen = how many positions it sees (rows, heads)."""
    rows, heads, dim = q.shape
    hk = k_pool.shape[2]
    group = heads // hk
    n_seq = len(kv_len)
    out = np.zeros((rows, heads, dim))
    absv, sumv = np.zeros_like(out), np.zeros_like(out)
    smax, seen_n = np.zeros((rows, heads)), np.zeros((rows, heads))
    mass = np.zeros((n_seq, hk, max(list(kv_len) + [0])))
    for i in range(n_seq):
        length, n = int(kv_len[i]), int(q_starts[i + 1] - q_starts[i])
        k, v = gather(k_pool, table, i, length), gather(v_pool, table, i, length)
        for j in range(n):
            r = q_starts[i] + j
            seen = np.flatnonzero(visible(length - n + j, length, window, sinks))
            if len(seen) == 0:
                continue
            for c in range(heads):
                h = c // group
                ks, vs = k[seen, h], v[seen, h]
                s = ks @ q[r, c] * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[r, c] = w @ vs
                absv[r, c] = w @ np.abs(vs)
                sumv[r, c] = np.abs(vs).sum(axis=0)
                smax[r, c] = (np.abs(ks) @ np.abs(q[r, c])).max() * abs(scale)
                seen_n[r, c] = len(seen)
                mass[i, h, seen] += w
    return dict(out=out, mass=mass, absv=absv, sumv=sumv, smax=smax, seen=seen_n)


def e4m3_grid():
    """The 256 values of the e4m3 codes (NaN at 0x7f and 0xff)."""
    vals = np.zeros(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        mag = np.nan if (e == 15 and m == 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        vals[code] = -mag if code & 128 else mag
    return vals


def to_e4m3(x):
    """Codes nearest to x, ties to the even code, clamped to the largest value; NaN keeps the NaN code."""
    pos = e4m3_grid()[:127]
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=E4M3_MAX, neginf=-E4M3_MAX)), E4M3_MAX)
    hi = np.clip(np.searchsorted(pos, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - pos[lo], pos[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def append(pool, new, q_starts, kv_len, table):
    """pool with the batch's rows stored (any element type: a copy); rows of invalid pages are skipped."""
    pool = pool.copy()
    page_size = pool.shape[1]
    for i in range(len(kv_len)):
        n = int(q_starts[i + 1] - q_starts[i])
        for j in range(n):
            p = int(kv_len[i]) - n + j
            page = int(table[i][p // page_size])
            if 0 <= page < pool.shape[0]:
                pool[page, p % page_size] = new[q_starts[i] + j]
    return pool


def evict_keep(mass, length, budget, sinks, recent):
    """Positions of one head that stay, ascending."""
    if length <= budget:
        return list(range(length))
    forced = [p for p in range(length) if p < sinks or p >= length - recent]
    free = [p for p in range(length) if not (p < sinks or p >= length - recent)]
    free.sort(key=lambda p: (np.isnan(mass[p]), -mass[p] if not np.isnan(mass[p]) else 0.0, p))
    return sorted(forced + free[:budget - sinks - recent])
