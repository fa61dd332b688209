"""Eviction from a cache by accumulated attention weight (oracle; test infrastructure).

Of the n = lens[b] keys of a (batch, head) all stay when n <= budget; otherwise
the last `recent` ones and, of the others, the budget - recent of the largest
weight, of equal ones the one of the lower index first (NaN counts as -inf).
The kept rows, ascending, move to the front of the cache.
"""
from __future__ import annotations

import math

import numpy as np


def select(weights, lens, budget: int, recent: int):
    """(keep int32 [B, H, budget], -1 behind the last; new_lens int32 [B])."""
    w = np.asarray(weights, dtype=np.float64)
    B, H, N = w.shape
    keep = np.full((B, H, budget), -1, dtype=np.int32)
    new = np.zeros(B, dtype=np.int32)
    for b in range(B):
        n = min(max(int(lens[b]), 0), N)
        new[b] = min(n, budget)
        for h in range(H):
            rows = list(range(n))
            if n > budget:
                def rank(j):
                    x = float(w[b, h, j])
                    return (math.inf if math.isnan(x) else -x, j)
                best = sorted(range(n - recent), key=rank)[:budget - recent]
                rows = sorted(best) + list(range(n - recent, n))
            keep[b, h, :len(rows)] = rows
    return keep, new


def compact(arrays, outs, idx, count, start=None, zero_end=None, in_place=False):
    """Row s + t of every out <- row s + idx[b, h, t] of its array, t < count[b]; arrays and
    outs [B, H, N, ...]. The last out, when zero_end is given, is zeroed in
    [s + count, zero_end). Returns new outs."""
    src = [np.array(a) for a in arrays]
    res = [np.array(o) for o in outs]
    idx = np.asarray(idx)
    for b in range(src[0].shape[0]):
        s = 0 if start is None else int(start[b])
        c = min(max(int(count[b]), 0), idx.shape[2])
        for h in range(src[0].shape[1]):
            for t in range(c):
                x = int(idx[b, 0 if idx.shape[1] == 1 else h, t])
                for a, r in zip(src, res):
                    if x < 0 or not 0 <= s + x < a.shape[2] or not 0 <= s + t < r.shape[2] or (in_place and x < t):
                        continue
                    r[b, h, s + t] = a[b, h, s + x]
            if zero_end is not None:
                res[-1][b, h, max(s + c, 0):max(int(zero_end[b]), 0)] = 0
    return res
