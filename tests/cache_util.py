"""Inputs and tolerances shared by the tests of the cache operators."""
import math

import numpy as np
import torch

from oracle import tree as OT

HALF_BF16 = 2.0 ** -8   # half a step of bf16, relative to the value
ULP = 2.0 ** -23        # a full step of fp32: bounds a rounding or a truncation


def make(seed, B, Hq, Hkv, T, N, D, lens, tree=None, token_major=False, scale=1.0):
    """q, k, v (bf16, on the CPU), lens and parents as tensors. tree: None for a
    chain, "random" for random trees, or a list of lists."""
    g = torch.Generator().manual_seed(seed)
    q = (scale * torch.randn(B, Hq, T, D, generator=g)).to(torch.bfloat16)
    if token_major:
        k = torch.randn(B, N, Hkv, D, generator=g).to(torch.bfloat16).transpose(1, 2)
        v = torch.randn(B, N, Hkv, D, generator=g).to(torch.bfloat16).transpose(1, 2)
    else:
        k = torch.randn(B, Hkv, N, D, generator=g).to(torch.bfloat16)
        v = torch.randn(B, Hkv, N, D, generator=g).to(torch.bfloat16)
    parents = random_trees(seed, B, T) if tree == "random" else tree
    parents = None if parents is None else torch.tensor(parents, dtype=torch.int32)
    return q, k, v, torch.tensor(lens, dtype=torch.int32), parents


def random_trees(seed, B, T, empty=True):
    """Parents of random trees; from the second batch on the last places are empty."""
    rng = np.random.default_rng(seed)
    trees = []
    for b in range(B):
        size = T if b == 0 or not empty else int(rng.integers(1, T + 1))
        trees.append([-2 if t >= size else (-1 if t == 0 else int(rng.integers(-1, t))) for t in range(T)])
    return trees


def to_gpu(t):
    """The tensor on the GPU with the strides it has."""
    if t is None:
        return None
    if t.is_contiguous():
        return t.cuda()
    return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)


def score_error(q, k):
    """Bound on the error of a fp32 score q.k / sqrt(D) against the exact one:
    D products (exact in fp32 for bf16 inputs) summed with at most a full step
    of the running sum lost per addition, then two roundings of the scaled
    value; in the unit of the natural exponent. [B, Hq, T]"""
    q, k = OT._f64(q), OT._f64(k)
    B, Hq, T, D = q.shape
    G = Hq // k.shape[1]
    size = np.zeros((B, Hq, T))
    for b in range(B):
        for h in range(Hq):
            kk = np.abs(np.nan_to_num(k[b, h // G], nan=0.0, posinf=0.0, neginf=0.0))
            size[b, h] = (np.abs(np.nan_to_num(q[b, h])) @ kk.T).max(axis=-1) / math.sqrt(D)
    return (D + 4) * ULP * size


def attention_tolerance(q, k, v, lens, parents, out, lse):
    """How far out and lse may be off, from the roundings the kernel makes:
    out: weights rounded to bf16 (half a step each), the output rounded to bf16
        (half a step), and in fp32: the scores (a relative error of twice their
        absolute one in a normalised weight), exp2 (2 steps), sums over the keys
        (a step each).
    lse: the scores' error, the sum's, exp2's, and 4 steps at its own size."""
    n = int(np.max(np.asarray(lens))) + q.shape[2]
    ds = score_error(q, k)
    rel = 2 * ds + (n + 8) * ULP
    mass, _ = OT.tree_attention(q, k, np.abs(np.nan_to_num(OT._f64(v), nan=0.0, posinf=0.0, neginf=0.0)), lens, parents)
    # sum of p |v|: an upper bound on what the weights' relative errors can move
    err = mass * (HALF_BF16 + rel[..., None]) * (1 + HALF_BF16)
    tol_out = err + HALF_BF16 * np.abs(out) + 1e-30
    tol_lse = ds + (n + 8) * ULP + 4 * ULP * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return tol_out, tol_lse


def check_attention(out, lse, q, k, v, lens, parents=None):
    """GPU results against the oracle within attention_tolerance; empty rows exact."""
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ref_out, ref_lse = OT.tree_attention(q, k, v, lens, parents)
    tol_out, tol_lse = attention_tolerance(q, k, v, lens, parents, ref_out, ref_lse)
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), empty), "rows that see no key differ"
    assert (out[empty] == 0).all(), "rows that see no key must output 0"
    assert np.isfinite(out).all()
    worst = np.max(np.abs(out - ref_out) / tol_out, initial=0.0)
    assert worst <= 1.0, f"out is {worst} times its tolerance off"
    fin = ~empty
    if fin.any():
        worst = np.max(np.abs(lse[fin] - ref_lse[fin]) / tol_lse[fin])
        assert worst <= 1.0, f"lse is {worst} times its tolerance off"


def weights_tolerance(q, k, lse, lens, parents, row_scale, weights_in, decay, ref):
    """A weight r * exp(s - lse): the score's error, the roundings of lse in base 2 and
    of the exponent (a step at the size of |lse| + 64: smaller weights are below
    e^-64), exp2's two steps; then a sum over R rows, a step each, and the old
    value's product and sum."""
    B, Hq, T, _ = q.shape
    R = T * (Hq // k.shape[1])
    l = np.abs(np.where(np.isfinite(OT._f64(lse)), OT._f64(lse), 0.0)).max(initial=0.0)
    rel = score_error(q, k).max(initial=0.0) + 2 * ULP * (l + 64) + (R + 4) * ULP
    mag = OT.key_weights(q, k, lse, lens, parents, None if row_scale is None else np.abs(OT._f64(row_scale)),
                         None if weights_in is None else np.abs(OT._f64(weights_in)), abs(decay))
    return mag * (rel + 4 * ULP) + R * math.exp(-64)
