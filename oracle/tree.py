"""Oracle: a step of decoding along a tree of drafted tokens, in float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages decode one token per step; a tree of drafts is the step of speculative
decoding that verifies many guesses at once.  Node 0 is certain, every other node a
guess at what follows its parent; the nodes' rows are the last of the sequence.
"""
from __future__ import annotations

import numpy as np


def sees_of(words: np.ndarray, n: int) -> np.ndarray:
    """Boolean [n, n] of a tree's mask words (uint64 [n, words]): row i, column j for bit j of node i."""
    out = np.zeros((n, n), bool)
    for i in range(n):
        for j in range(n):
            out[i, j] = bool((int(words[i, j // 64]) >> (j % 64)) & 1)
    return out


def words_of(sees: np.ndarray, width: int) -> np.ndarray:
    """The mask words (uint64 [n, width]) of a boolean [n, n]."""
    n = sees.shape[0]
    out = np.zeros((n, width), np.uint64)
    for i in range(n):
        for j in np.flatnonzero(sees[i]):
            out[i, j // 64] |= np.uint64(1 << (int(j) % 64))
    return out


def attention(q, k, v, sees, scale):
    """q [n, hq, D], k and v [L, hkv, D] (the last n rows the nodes'), sees [n, n] -> (out, A), A = sum p |v|.

    Keys a node does not see are not looked at; a node that sees nothing gets zeros."""
    n, hq, d = q.shape
    length, hkv, _ = k.shape
    out, weight = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    for i in range(n):
        keys = np.concatenate([np.arange(length - n), length - n + np.flatnonzero(sees[i])])
        if keys.size == 0:
            continue
        for h in range(hq):
            g = h // (hq // hkv)
            with np.errstate(invalid="ignore"):
                s = k[keys, g] @ q[i, h] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[i, h] = p @ v[keys, g]
                weight[i, h] = p @ np.abs(v[keys, g])
    return out, weight


def accept(target, draft, sees, limit):
    """The path from node 0 along children whose draft is the target at their parent, and the token that follows."""
    n = len(target)
    if n == 0:
        return [], -1
    parent = [max([j for j in range(i) if sees[i, j]], default=-1) for i in range(n)]
    path = [0]
    while len(path) < limit:
        here = path[-1]
        children = [i for i in range(n) if parent[i] == here and draft[i] == target[here]]
        if not children:
            break
        path.append(children[0])
    return path, int(target[path[-1]])
