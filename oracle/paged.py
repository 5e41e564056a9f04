"""Serving operators in fp64: norm and position rotation of rows, the append
of a chunk to a paged cache, attention of the chunk over it (definitions in
include/vark.h, "Serving: a paged cache").

Pools are [pages][H][page_size][D] with table [B][max_pages] and lengths [B],
or, head-specific, [pages][page_size][D] with [B][H][max_pages] and [B][H]."""
from __future__ import annotations

import math

import numpy as np

NORM_NONE, NORM_RMS, NORM_L2 = 0, 1, 2


def norm_rotate(x, norm, weight, eps, rope, positions, pairs):
    """x [tokens][H][D]; rope [P][2][R / 2] or None; positions [tokens].
    Returns (y, mag): mag[...] = |a cos| + |b sin| of the sums that gave y."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    ss = (x * x).sum(-1, keepdims=True)
    if norm == NORM_RMS:
        x = x / np.sqrt(ss / D + eps)
    elif norm == NORM_L2:
        x = x / np.maximum(np.sqrt(ss), eps)
    if weight is not None:
        x = x * np.asarray(weight, dtype=np.float64)
    y, mag = x.copy(), np.abs(x)
    if rope is None:
        return y, mag
    half = rope.shape[2]
    for n, p in enumerate(positions):
        if p < 0:
            continue
        for j in range(half):
            ia, ib = (2 * j, 2 * j + 1) if pairs else (j, j + half)
            c, s = float(rope[p, 0, j]), float(rope[p, 1, j])
            a, b = x[n, :, ia], x[n, :, ib]
            y[n, :, ia], y[n, :, ib] = a * c - b * s, a * s + b * c
            mag[n, :, ia], mag[n, :, ib] = abs(a * c) + abs(b * s), abs(a * s) + abs(b * c)
    return y, mag


def paged_row(table, lens, cu, page_size, b, h, i):
    """(page, row in page) of token i of sequence b for head h, or None where
    the cache does not hold it.  h is ignored for shared tables."""
    n = int(cu[b + 1]) - int(cu[b])
    length = int(lens[b, h]) if np.ndim(lens) == 2 else int(lens[b])
    row = length - n + i
    if row < 0:
        return None
    t = table[b, h] if np.ndim(table) == 3 else table[b]
    return int(t[row // page_size]), row % page_size


def gather_rows(pool, table, lens, b, h):
    """The cache rows of (b, h): [len][D]."""
    head = np.ndim(lens) == 2
    ps = pool.shape[-2]
    length = int(lens[b, h]) if head else int(lens[b])
    t = table[b, h] if head else table[b]
    out = np.empty((length, pool.shape[-1]), dtype=pool.dtype)
    for r in range(length):
        page = int(t[r // ps])
        out[r] = pool[page, r % ps] if head else pool[page, h, r % ps]
    return out


def paged_attention(q, cu, k_pages, v_pages, table, lens, tau, causal):
    """q [tokens][Hq][D]; tau [Hq].  Returns (out, lse, mean_abs, logit_abs):
    mean_abs [tokens][Hq][D] is the attention-weighted mean of |v| and
    logit_abs [tokens][Hq] the largest sum |q_d k_d| tau / sqrt(D) of a row --
    the magnitudes that rounding errors scale with.  Tokens of no sequence are
    left at zero."""
    q = np.asarray(q, dtype=np.float64)
    N, Hq, D = q.shape
    H = table.shape[1] if np.ndim(table) == 3 else k_pages.shape[1]
    G = Hq // H
    out = np.zeros((N, Hq, D))
    lse = np.zeros((N, Hq))
    mean_abs = np.zeros((N, Hq, D))
    logit_abs = np.zeros((N, Hq))
    for b in range(len(cu) - 1):
        n = int(cu[b + 1]) - int(cu[b])
        for h in range(H):
            K = gather_rows(k_pages, table, lens, b, h).astype(np.float64)
            V = gather_rows(v_pages, table, lens, b, h).astype(np.float64)
            for i in range(n):
                lim = len(K) - n + i + 1 if causal else len(K)
                t = int(cu[b]) + i
                for hq in range(h * G, (h + 1) * G):
                    if lim <= 0:
                        lse[t, hq] = -math.inf
                        continue
                    f = float(tau[hq]) / math.sqrt(D)
                    x = (K[:lim] @ q[t, hq]) * f
                    m = x.max()
                    p = np.exp(x - m)
                    l = p.sum()
                    out[t, hq] = (p @ V[:lim]) / l
                    lse[t, hq] = m + math.log(l)
                    mean_abs[t, hq] = (p @ np.abs(V[:lim])) / l
                    logit_abs[t, hq] = (np.abs(K[:lim]) @ np.abs(q[t, hq])).max() * abs(f)
    return out, lse, mean_abs, logit_abs
