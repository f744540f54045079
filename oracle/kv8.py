"""CPU oracle for the paged 8-bit K/V cache.

TEST INFRASTRUCTURE, like the rest of ``oracle/``.  Plain numpy in float64,
one page or one query row at a time; it shares nothing with the CUDA path.

A pool holds e4m3 codes [pages][page][Hkv][d] and one scale per page and head;
an element stands for value(code) * scale.  Appending to a page sets, for each
head, need = the smallest power of two (2^-120 at least) with
max |new finite elements| <= 448 need; the scale becomes need on an empty
page, else the larger of the two, and the older codes are rounded again under
a scale that grew.
"""
from __future__ import annotations

import numpy as np


def _values() -> np.ndarray:
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


VALUES = _values()


def decode(codes) -> np.ndarray:
    return VALUES[np.asarray(codes, np.uint8)]


def encode(x) -> np.ndarray:
    """Nearest code, ties to the even one; at most 448; NaN and infinities
    become the positive NaN code."""
    x = np.asarray(x, np.float64)
    pos = VALUES[:127]                     # 0 ... 448, ascending
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    up, down = pos[hi] - a, a - pos[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    c = np.where(np.signbit(x), c + 128, c)
    return np.where(np.isfinite(x), c, 127).astype(np.uint8)


def need(x) -> float:
    """The scale that a page's new elements of one head ask for."""
    x = np.abs(np.asarray(x, np.float64))
    x = x[np.isfinite(x)]
    top = x.max() if x.size else 0.0
    e = -120
    while top > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, codes, scales, table, lens, new_off) -> None:
    """Stores rows x [T][Hkv][d] (float64) behind lens[b] tokens of each
    sequence, in place; table entries outside the pool leave their page out."""
    pages, page, Hkv, _ = codes.shape
    for b in range(len(lens)):
        if lens[b] < 0:
            continue
        rows = x[new_off[b]:new_off[b + 1]]
        n = int(lens[b])
        for col in range(n // page, -(-(n + len(rows)) // page) if len(rows) else 0):
            lo, hi = max(n, col * page), min(n + len(rows), (col + 1) * page)
            if col >= table.shape[1] or not 0 <= table[b, col] < pages:
                continue
            p, first, last = table[b, col], lo - col * page, hi - col * page
            for h in range(Hkv):
                part = rows[lo - n:hi - n, h]
                s = need(part)
                if first:
                    s = max(s, float(scales[p, h]))
                    if s != scales[p, h]:
                        old = decode(codes[p, :first, h]) * float(scales[p, h])
                        codes[p, :first, h] = encode(old / s)
                codes[p, first:last, h] = encode(part / s)
                scales[p, h] = s


def gather(codes, scales, table, b, keys) -> np.ndarray:
    """Stored rows [len(keys)][Hkv][d] of sequence b."""
    page = codes.shape[1]
    keys = np.asarray(keys, np.int64)
    p = table[b, keys // page]
    return decode(codes[p, keys % page]) * np.asarray(scales, np.float64)[p][..., None]


def attention(Q, k8, v8, k_scale, v_scale, table, seq, keys, scale):
    """Rows Q [T][Hq][d] (float64) of sequences seq[t] over their keys[t]
    (lists of positions).  Returns O, lse and what the error bounds need: per
    (t, h), the sum of p |v| as an array like O, the largest scale * sum_c
    |q_c k_c| and the largest weight * v scale."""
    T, Hq, d = Q.shape
    Hkv, page = k8.shape[2], k8.shape[1]
    G = Hq // Hkv
    O, mag = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    lse = np.full((T, Hq), -np.inf)
    big, top = np.zeros((T, Hq)), np.zeros((T, Hq))
    for t in range(T):
        ks = np.asarray(keys[t], np.int64)
        if len(ks) == 0:
            continue
        K = gather(k8, k_scale, table, seq[t], ks)
        V = gather(v8, v_scale, table, seq[t], ks)
        vs = np.asarray(v_scale, np.float64)[table[seq[t], ks // page]]
        for h in range(Hq):
            g = h // G
            x = K[:, g] @ Q[t, h] * scale
            e = np.exp(x - x.max())
            p = e / e.sum()
            O[t, h], mag[t, h] = p @ V[:, g], p @ np.abs(V[:, g])
            lse[t, h] = x.max() + np.log(e.sum())
            big[t, h] = (np.abs(K[:, g]) @ np.abs(Q[t, h])).max() * scale
            top[t, h] = (p * vs[:, g]).max()
    return O, lse, mag, big, top
