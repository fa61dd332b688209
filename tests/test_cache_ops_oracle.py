"""Pins of the cache operators' oracle (oracle/tree.py, oracle/evict.py), on the CPU."""
import math

import numpy as np
import pytest
import torch

from oracle import decode as OD
from oracle import evict as OE
from oracle import tree as OT

from .cache_util import make, random_trees


@pytest.mark.parametrize("T", [1, 2, 7, 20])
def test_ancestors_equal_the_closure_of_the_parent_relation(T):
    for parents in random_trees(T, 4, T):
        step = np.zeros((T, T), dtype=bool)
        for t, p in enumerate(parents):
            step[t, t] = p != -2
            if p >= 0:
                step[t, p] = True
        closure = np.linalg.matrix_power(step.astype(float), max(T, 1)) > 0
        seen = OT.ancestors(parents)
        for t in range(T):
            assert seen[t] == set(np.flatnonzero(closure[t])), (parents, t)


def test_chain_equals_decode_over_every_block():
    """A chain of T tokens at the end of the cache is the decode rule with every block listed."""
    q, k, v, lens, _ = make(3, 2, 4, 2, 5, 200, 16, [195, 195])
    sel = np.broadcast_to(np.arange(4), (2, 2, 5, 4))
    ref = OD.decode_attention(q, k, v, sel)
    for parents in (None, [[-1, 0, 1, 2, 3]] * 2):
        got = OT.tree_attention(q, k, v, lens, parents)
        np.testing.assert_allclose(got[0], ref[0], atol=1e-12)
        np.testing.assert_allclose(got[1], ref[1], atol=1e-12)


def test_tree_equals_dense_masked_attention():
    q, k, v, lens, parents = make(4, 2, 4, 4, 6, 60, 16, [31, 0], [[-1, 0, 0, 2, -1, 4], [-1, -1, 0, 1, 3, -2]])
    bias = torch.full((2, 1, 6, 60), -math.inf, dtype=torch.float64)
    for b, rows in enumerate([[{0}, {0, 1}, {0, 2}, {0, 2, 3}, {4}, {4, 5}], [{0}, {1}, {0, 2}, {1, 3}, {1, 3, 4}, set()]]):
        for t, nodes in enumerate(rows):
            if nodes:
                bias[b, 0, t, :int(lens[b])] = 0
            for n in nodes:
                bias[b, 0, t, int(lens[b]) + n] = 0
    ref = torch.nn.functional.scaled_dot_product_attention(q.double(), k.double(), v.double(), attn_mask=bias)
    out, lse = OT.tree_attention(q, k, v, lens, parents)
    empty = np.isneginf(lse)
    assert empty.sum() == 4 and empty[1, :, 5].all() and (out[empty] == 0).all()
    np.testing.assert_allclose(out[~empty], ref.numpy()[~empty], atol=1e-12)


def test_rows_not_seen_may_hold_anything():
    q, k, v, lens, parents = make(5, 1, 2, 1, 4, 40, 16, [20], [[-1, 0, 1, -2]])
    ref = OT.tree_attention(q, k, v, lens, parents)
    k[0, 0, 23:] = math.nan
    v[0, 0, 23:] = math.inf
    got = OT.tree_attention(q, k, v, lens, parents)
    np.testing.assert_array_equal(got[0], ref[0])


def test_weights_of_a_row_sum_to_one_and_follow_the_softmax():
    q, k, v, lens, parents = make(6, 2, 6, 2, 5, 50, 16, [30, 0], "random")
    _, lse = OT.tree_attention(q, k, v, lens, parents)
    live = np.isfinite(lse).reshape(2, 2, 3, 5).sum(axis=(2, 3))
    w = OT.key_weights(q, k, lse, lens, parents)
    np.testing.assert_allclose(w.sum(-1), live, atol=1e-12)
    # one row alone, times its scale, on top of a decayed sum
    row = np.zeros((2, 5))
    row[:, 0] = 2.0
    old = np.random.default_rng(0).random((2, 2, 50))
    w = OT.key_weights(q, k, lse, lens, parents, row, old, 0.5)
    s = (q[0, :3, 0].double() @ k[0, 0, :31].double().T / 4.0).softmax(-1).sum(0).numpy()
    np.testing.assert_allclose(w[0, 0, :31], 2 * s + 0.5 * old[0, 0, :31], atol=1e-12)
    assert (w[0, :, 35:] == 0).all()


def test_select_equals_a_stable_sort():
    rng = np.random.default_rng(1)
    w = np.round(rng.random((2, 3, 64)), 1)  # many ties
    keep, new = OE.select(w, [64, 40], 16, 4)
    assert new.tolist() == [16, 16]
    for b, n in enumerate([64, 40]):
        for h in range(3):
            order = np.argsort(-w[b, h, :n - 4], kind="stable")[:12]
            assert keep[b, h].tolist() == sorted(order.tolist()) + list(range(n - 4, n))
    keep, new = OE.select(w, [10, 0], 16, 4)
    assert new.tolist() == [10, 0] and keep[0, 0].tolist() == list(range(10)) + [-1] * 6 and (keep[1] == -1).all()
    w[0, 0, :4] = [math.nan, math.inf, -math.inf, -0.0]
    keep, _ = OE.select(w, [64, 64], 63, 0)
    assert keep[0, 0].tolist() == [j for j in range(64) if j != 2] or keep[0, 0].tolist() == [j for j in range(64) if j != 0]


def test_compact_equals_indexing():
    a = np.arange(2 * 2 * 10).reshape(2, 2, 10)
    idx = np.array([[[1, 3, 7]], [[0, 1, 9]]])
    r, = OE.compact([a], [a], idx, [3, 2], in_place=True)
    assert r[0, 1].tolist() == [11, 13, 17] + list(range(13, 20))
    assert r[1, 0].tolist() == list(range(20, 30))
    r, = OE.compact([a], [np.zeros((2, 2, 4), int)], idx, [3, 3], start=[2, 0], zero_end=[0, 0])
    assert r[0, 0].tolist() == [0, 0, 3, 5] and r[1, 1].tolist() == [30, 31, 39, 0]
