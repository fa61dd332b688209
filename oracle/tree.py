"""Drafted tokens over a cache, float64 (oracle; test infrastructure).

Batch b's cache holds lens[b] keys; T drafted tokens lie behind them, node t in
cache row lens[b] + t. parents[b, t] is the node's parent, -1 when it follows
the sequence itself, -2 when the place is empty (parents None: a chain). Row t
sees every key before lens[b], itself and its ancestors; an empty place sees
nothing and is seen by nobody. Nodes whose cache row would lie past the cache
are seen by nobody.

    out, lse    attention.attention_rows over the keys seen
    weight_j    sum over rows and the group's heads of row_scale * exp(s_j - lse)
"""
from __future__ import annotations

import math

import numpy as np

from .attention import _f64, attention_rows


def ancestors(parents) -> list:
    """For each place the set of nodes it sees, itself included (empty for an empty place)."""
    seen = []
    for t, p in enumerate(parents):
        p = int(p)
        if p == -2:
            seen.append(set())
        else:
            seen.append({t} | (seen[p] if 0 <= p < t else set()))
    return seen


def visible(length: int, parents, T: int, N: int) -> np.ndarray:
    """Boolean [T, N]: the cache rows each drafted token sees."""
    length = min(max(int(length), 0), N)
    parents = list(range(-1, T - 1)) if parents is None else parents
    vis = np.zeros((T, N), dtype=bool)
    for t, nodes in enumerate(ancestors(parents)):
        if int(parents[t]) == -2:
            continue
        vis[t, :length] = True
        for n in nodes:
            if length + n < N:
                vis[t, length + n] = True
    return vis


def _inputs(q, k, lens, parents):
    q, k = _f64(q), _f64(k)
    lens = np.asarray(lens)
    parents = [None] * q.shape[0] if parents is None else np.asarray(parents)
    return q, k, lens, parents, q.shape[1] // k.shape[1]


def tree_attention(q, k, v, lens, parents=None):
    """q [B, Hq, T, d], k/v [B, Hkv, N, d] -> (out [B, Hq, T, d], lse [B, Hq, T]).
    Cache rows no drafted token sees may hold anything."""
    q, k, lens, parents, G = _inputs(q, k, lens, parents)
    v = _f64(v)
    B, Hq, T, d = q.shape
    out, lse = np.zeros((B, Hq, T, d)), np.full((B, Hq, T), -np.inf)
    for b in range(B):
        vis = visible(lens[b], parents[b], T, k.shape[2])
        seen = vis.any(axis=0)
        live = vis.any(axis=1)
        for h in range(Hq):
            o, s = attention_rows(q[b, h, live], k[b, h // G][seen], v[b, h // G][seen], vis[live][:, seen])
            out[b, h, live], lse[b, h, live] = o, s
    return out, lse


def key_weights(q, k, lse, lens, parents=None, row_scale=None, weights_in=None, decay=1.0, weights_out=None):
    """weights_out [B, Hkv, N] with the held keys' entries replaced (None: zeros elsewhere)."""
    q, k, lens, parents, G = _inputs(q, k, lens, parents)
    lse = _f64(lse)
    B, Hq, T, d = q.shape
    Hkv, N = k.shape[1], k.shape[2]
    w = np.zeros((B, Hkv, N)) if weights_out is None else _f64(weights_out).copy()
    scale = np.ones((B, T)) if row_scale is None else _f64(row_scale)
    for b in range(B):
        vis = visible(lens[b], parents[b], T, N)
        held = min(max(int(lens[b]), 0) + T, N)
        for g in range(Hkv):
            total = np.zeros(held)
            if weights_in is not None and decay != 0:
                total = decay * _f64(weights_in)[b, g, :held]
            for t in range(T):
                if scale[b, t] == 0:
                    continue
                at = np.flatnonzero(vis[t])
                for h in range(g * G, (g + 1) * G):
                    if np.isneginf(lse[b, h, t]):
                        continue
                    total[at] += scale[b, t] * np.exp(k[b, g, at] @ q[b, h, t] / math.sqrt(d) - lse[b, h, t])
            w[b, g, :held] = total
    return w


__all__ = ["ancestors", "visible", "tree_attention", "key_weights"]
