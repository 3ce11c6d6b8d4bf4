"""fp64 CPU oracle for the paged single-plane cache (test infrastructure only).

The cache of sequence i is what its page table says: position p lies in slot
p % page of page table[i][p // page].  The attention of a new token at position t
sees positions p <= t with no window, or p > t - window, or p < sinks.
"""
from __future__ import annotations

import numpy as np


def append(K, V, k_pages, v_pages, table, ctx, row0):
    """Writes row row0[i] + j at position ctx[i] + j; pages [npages][Hkv][page][d]."""
    page = k_pages.shape[2]
    for i in range(len(ctx)):
        for j in range(row0[i + 1] - row0[i]):
            pos = ctx[i] + j
            k_pages[table[i][pos // page], :, pos % page] = K[row0[i] + j]
            v_pages[table[i][pos // page], :, pos % page] = V[row0[i] + j]


def gather(pages, table_row, n):
    """Positions 0..n-1 of a sequence: [Hkv][n][d]."""
    page = pages.shape[2]
    ids = np.asarray(table_row[: -(-n // page)], dtype=np.int64)
    rows = pages[ids].transpose(1, 0, 2, 3).reshape(pages.shape[1], -1, pages.shape[3])
    return rows[:, :n]


def seen(pos, n, window, sinks):
    key = np.arange(n)
    ok = key <= pos
    if window:
        ok &= (key > pos - window) | (key < sinks)
    return ok


def attn(Q, k_pages, v_pages, table, ctx, row0, window=0, sinks=0, scale=0.0):
    """O [nrows][H][d] and lse [nrows][H] in 64 bits; rows of no sequence are NaN.  Hidden
    keys and values are left out by indexing, so what they hold cannot matter."""
    nrows, H, d = Q.shape
    G = H // k_pages.shape[1]
    scale = scale or 1.0 / np.sqrt(d)
    O = np.full((nrows, H, d), np.nan)
    lse = np.full((nrows, H), np.nan)
    for i in range(len(ctx)):
        n = row0[i + 1] - row0[i]
        if n <= 0:
            continue
        K = gather(k_pages, table[i], ctx[i] + n).astype(np.float64)
        V = gather(v_pages, table[i], ctx[i] + n).astype(np.float64)
        for j in range(n):
            ok = seen(ctx[i] + j, ctx[i] + n, window, sinks)
            r = row0[i] + j
            q = Q[r].astype(np.float64).reshape(-1, G, d)
            s = np.einsum("hgd,hkd->hgk", q, K[:, ok]) * scale
            with np.errstate(invalid="ignore", over="ignore"):
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                lse[r] = (m[..., 0] + np.log(e.sum(-1))).reshape(H)
                p = e / e.sum(-1, keepdims=True)
                O[r] = np.einsum("hgk,hkd->hgd", p, V[:, ok]).reshape(H, d)
    return O, lse
