"""fp64 CPU oracle for the token draw (test infrastructure only).

Tokens in the order (logit descending, index ascending); w = exp((z - max) / T).  Kept:
the first k, of them while the mass before is below p times the mass of the first k, of
them those with w >= min_p, and always the first.  The draw is the smallest index whose
running sum of kept w exceeds u times the kept mass.
"""
from __future__ import annotations

import numpy as np


def kept(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(indices kept, weights of all tokens); temperature <= 0 keeps the first token."""
    z = np.where(np.isnan(z), -np.inf, np.asarray(z, dtype=np.float64))
    order = np.argsort(-z, kind="stable")
    m = z[order[0]]
    if m == -np.inf:
        return order[:0], np.zeros(len(z))
    if not temperature > 0:
        w = np.zeros(len(z))
        w[order[0]] = 1.0
        return order[:1], w
    with np.errstate(invalid="ignore"):
        w = np.where(z == m, 1.0, np.exp((z - m) / temperature))
    sel = order if top_k <= 0 else order[:top_k]
    if top_p < 1:
        ahead = np.concatenate([[0.0], np.cumsum(w[sel])[:-1]])
        sel = sel[(ahead < top_p * w[sel].sum()) | (np.arange(len(sel)) == 0)]
    if min_p > 0:
        sel = sel[(w[sel] >= min_p) | (np.arange(len(sel)) == 0)]
    return sel, w


def draw(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log probability, distance of u * mass from the nearest running sum, as a
    share of the mass)."""
    sel, w = kept(z, temperature, top_k, top_p, min_p)
    if len(sel) == 0:
        return -1, -np.inf, 1.0
    idx = np.sort(sel)
    c = np.cumsum(w[idx])
    at = int(np.searchsorted(c, u * c[-1], side="right"))
    margin = np.min(np.abs(c[:-1] / c[-1] - u)) if len(c) > 1 else 1.0
    return int(idx[at]), float(np.log(w[idx[at]] / c[-1])), float(margin)
