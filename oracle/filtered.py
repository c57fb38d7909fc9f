"""Oracle: top-k, top-p and min-p before the exponential race, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The visual atlas (diomchen.github.io/reference/visual-atlas.html), fig. 23, names
top-k and top-p as extensions of the engine's temperature sampler without fixing
their details; the reading here: tokens are ordered by logit, equal logits by
column; top-k keeps the first k; top-p keeps, of those, every token before which
the probabilities (renormalised over them) sum to less than p; min-p keeps, of
those, the tokens at least min_p times as likely as the likeliest; the race of
fig. 23 then runs among the kept tokens on the noise of ``oracle/sampler.py``.
"""
from __future__ import annotations

import numpy as np

from .sampler import exponential_noise


def kept(logits, T, k, p, min_p):
    """Columns one row keeps, in order."""
    l = np.asarray(logits, dtype=np.float64)
    order = np.argsort(-l, kind="stable")
    order = np.array([v for v in order if l[v] > -np.inf], dtype=np.int64)        # neither -inf nor NaN
    if len(order) == 0:
        return order
    z = (l[order] - l[order[0]]) / T
    if k > 0:
        order, z = order[:k], z[:k]
    w = np.exp(z)
    if p < 1:
        before = np.cumsum(w) - w
        n = int(np.searchsorted(before, p * w.sum(), side="left"))
        order, z = order[:n], z[:n]
    if min_p > 0:
        order = order[z >= np.log(min_p)]
    return order


def sample(logits, temperatures, top_k, top_p, min_p, seed, offset=0):
    """(ids, margin): the winners and the race's log-margin (inf with one kept token).
    A row with an infinite logit: the first of them.  A row with nothing above -inf: -1."""
    logits = np.asarray(logits)
    B, V = logits.shape
    e = exponential_noise(seed, offset, range(B), V)
    ids, margin = np.full(B, -1, np.int64), np.full(B, np.inf)
    for b in range(B):
        inf = np.nonzero(logits[b] == np.inf)[0]
        if len(inf):
            ids[b] = inf[0]
            continue
        T = float(temperatures[b])
        cols = kept(logits[b], T, int(top_k[b]), float(top_p[b]), float(min_p[b]))
        if len(cols) == 0:
            continue
        key = logits[b, cols].astype(np.float64) / T - np.log(e[b, cols])
        best = np.lexsort((cols, -key))
        ids[b] = cols[best[0]]
        if len(cols) > 1:
            margin[b] = key[best[0]] - key[best[1]]
    return ids, margin


def decided(logits, temperatures, top_k, top_p, min_p, seed, offset=0, p_slack=1e-6):
    """(ids, clear): the winners, and which rows are decided by more than rounding: a race margin
    above 1e-9 and the same winner with top_p moved by p_slack of itself either way."""
    p = np.asarray(top_p, dtype=np.float64)
    ids, margin = sample(logits, temperatures, top_k, p, min_p, seed, offset)
    clear = margin > 1e-9
    for f in (1 - p_slack, 1 + p_slack):
        clear &= sample(logits, temperatures, top_k, np.where(p < 1, p * f, p), min_p, seed, offset)[0] == ids
    return ids, clear
