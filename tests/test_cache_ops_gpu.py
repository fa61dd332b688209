"""Drafted tokens over a cache, key weights and eviction on the GPU, against the oracle.

mfa_tree_decode, mfa_key_weights, mfa_evict_select and mfa_cache_compact
through the C ABI, every row and key of every case compared with
oracle/tree.py and oracle/evict.py on the same bf16 inputs (tolerances:
tests/cache_util.py). Moves and selections are exact.
"""
import math

import numpy as np
import pytest
import torch

from mask_aware_block_mfa_b200 import binding as B
from oracle import evict as OE
from oracle import tree as OT

from .cache_util import HALF_BF16, ULP, check_attention, make, random_trees, to_gpu, weights_tolerance

pytestmark = pytest.mark.gpu


def decode(q, k, v, lens, parents=None, op=None, **kw):
    op = B.TreeDecode() if op is None else op
    out, lse = op(to_gpu(q), to_gpu(k), to_gpu(v), to_gpu(lens), to_gpu(parents), **kw)
    err = op.status()
    op.clear()
    return out.cpu(), lse.cpu(), err


# D, Hkv, G, T, N, lens, tree, token_major
CASES = [
    (128, 2, 4, 1, 300, [299, 0, 128], None, False),        # one token; no key before it; a tile's end
    (64, 1, 1, 1, 1, [0], None, False),                     # the smallest call
    (128, 2, 2, 1, 130, [127, 126, 129, 1, 64], None, True),
    (64, 5, 3, 13, 700, [0, 687, 300], "random", True),     # groups of three
    (256, 2, 4, 4, 600, [596, 77], None, False),
    (256, 1, 16, 9, 500, [250, 491, 0], "random", True),    # 144 rows
    (128, 1, 4, 26, 1500, [1400], "random", False),
    (128, 2, 4, 32, 900, [868, 400], "random", False),      # 128 rows
    (128, 1, 4, 33, 900, [800], "random", False),           # 132 rows
    (64, 1, 8, 64, 700, [636, 3], "random", True),          # 512 rows
    (128, 1, 1, 256, 400, [144, 100], "random", False),     # the largest tree
    (128, 1, 2, 300, 700, [400, 10], None, False),          # a chain longer than any tree
    (64, 2, 1, 500, 500, [0], None, False),                 # plain causal attention
    (256, 3, 1, 17, 2000, [1983, 900, 130, 128, 127], "random", False),
    (128, 16, 1, 2, 260, [258] + [7 * i for i in range(30)], "random", True),
    (128, 1, 16, 1, 4000, [3999], None, False),             # one sequence over every SM
    (64, 1, 32, 1, 9000, [8999], None, True),
    (64, 1, 150, 3, 700, [697, 200], "random", True),       # a group larger than a row tile
    (256, 2, 70, 2, 300, [290, 0], None, False),
    (128, 1, 7, 20, 900, [850, 3], "random", True),         # 140 rows, 126 in the first tile
    (128, 2, 5, 3, 400, [390], "random", False),            # 15 rows of 16
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "d%d_h%d_g%d_t%d_n%d_b%d_%s" % (c[:5] + (len(c[5]), c[6])))
def test_tree_decode_matches_the_oracle(case):
    D, Hkv, G, T, N, lens, tree, major = case
    q, k, v, lens, parents = make(D + T + N, len(lens), Hkv * G, Hkv, T, N, D, lens, tree, major)
    out, lse, err = decode(q, k, v, lens, parents)
    assert err == 0
    check_attention(out, lse, q, k, v, lens, parents)


@pytest.mark.parametrize("D,G,T,tree", [(64, 2, 2, None), (64, 3, 10, "random"), (64, 4, 13, "random"), (64, 4, 32, "random"), (128, 2, 1, None),
                                        (128, 4, 7, "random"), (128, 5, 10, "random"), (128, 4, 30, "random"), (256, 2, 3, None),
                                        (256, 4, 8, "random"), (256, 6, 10, "random"), (256, 4, 30, "random")])
def test_tree_decode_with_many_tiles_and_pairs_per_block(D, G, T, tree):
    """Over 1500 tiles of 128 keys, so that every block walks ten or more, most of
    them long pairs and some of them many short ones."""
    lens = [9000, 40, 0, 5117, 300, 9728 - T, 128]
    q, k, v, lens, parents = make(D + T, len(lens), 8 * G, 8, T, 9728, D, lens, tree, True)
    op = B.TreeDecode()
    args = [to_gpu(x) for x in (q, k, v, lens, parents)]
    runs = [op(*args) for _ in range(3)]
    assert op.status() == 0
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
    out, lse = (x.cpu() for x in runs[0])
    ref_out, ref_lse = reference(args, D)
    mass, _ = reference(args[:2] + [args[2].abs()] + args[3:], D)
    tol_out, tol_lse = large_tolerance(args, mass, ref_out, ref_lse)
    assert ((out.cuda().double() - ref_out).abs() <= tol_out).all()
    empty = torch.isneginf(ref_lse)
    assert torch.equal(torch.isneginf(lse.cuda()), empty)
    assert ((lse.cuda().double() - ref_lse).abs() <= tol_lse)[~empty].all()


def reference(args, D):
    """The definition in 64 bits on the GPU, one batch at a time (large cases)."""
    q, k, v, lens, parents = args
    Bz, Hq, T, _ = q.shape
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full((Bz, Hq, T), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(Bz):
        end = int(lens[b]) + T
        vis = torch.from_numpy(OT.visible(int(lens[b]), None if parents is None else parents[b].tolist(), T, k.shape[2])[:, :end]).cuda()
        G = Hq // k.shape[1]
        kk, vv = (x[b, :, :end].double().repeat_interleave(G, 0) for x in (k, v))
        s = (q[b].double() @ kk.transpose(1, 2) / math.sqrt(D)).masked_fill(~vis, -math.inf)
        lse[b] = s.logsumexp(-1)
        out[b] = torch.where(vis.any(-1)[None, :, None], torch.nan_to_num((s - lse[b][..., None]).exp()) @ vv, 0.0)
    return out, lse


def large_tolerance(args, mass, out, lse):
    """attention_tolerance with |q . k| bounded by |q| |k|, on the GPU; mass: sum of p |v|."""
    q, k, _, lens, _ = args
    n, D = int(lens.max()) + q.shape[2], q.shape[3]
    ds = float((D + 4) * ULP * q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max() / math.sqrt(D))
    rel = 2 * ds + (n + 8) * ULP
    return mass * (HALF_BF16 + rel) * (1 + HALF_BF16) + HALF_BF16 * out.abs() + 1e-30, ds + (n + 8) * ULP + 4 * ULP * lse.abs()


@pytest.mark.parametrize("T,G", [(1, 4), (8, 4), (60, 2)])
def test_tree_decode_follows_a_maximum_that_grows(T, G):
    """Scores rise along the cache by far more than an exponent's range, so that the
    running maximum moves on in almost every tile; then they fall again."""
    q, k, v, lens, parents = make(11, 2, G, 1, T, 1200, 128, [1100, 700], "random" if T > 1 else None)
    ramp = torch.cat([torch.linspace(0, 6, 600), torch.linspace(6, 0, 600)])
    k = (k.float() * ramp[None, None, :, None]).to(torch.bfloat16)
    q = (q.float() * 3).to(torch.bfloat16)
    out, lse, err = decode(q, k, v, lens, parents)
    assert err == 0
    check_attention(out, lse, q, k, v, lens, parents)


def test_tree_decode_equal_keys_and_large_scores():
    """Every score equal and large (the weights are 1 / n), then one key that takes all."""
    q, k, v, lens, _ = make(12, 1, 4, 2, 1, 500, 128, [499])
    q.fill_(8.0)
    k.fill_(8.0)
    out, lse, err = decode(q, k, v, lens)
    assert err == 0
    check_attention(out, lse, q, k, v, lens)
    k[:, :, 333] = 16.0
    out, lse, err = decode(q, k, v, lens)
    check_attention(out, lse, q, k, v, lens)


@pytest.mark.parametrize("D,T,G", [(128, 6, 4), (64, 6, 3), (256, 40, 4)])
def test_what_no_row_sees_may_hold_anything(D, T, G):
    """Infinities and NaN behind the last node, in padding nodes' keys and rows, and, for
    the rows that do not see them, in other nodes' keys."""
    trees = [[-1] + [0] * (T - 2) + [-2], [-1, 0] + [-2] * (T - 2)]
    q, k, v, lens, parents = make(13, 2, G, 1, T, 400, D, [260, 380 - T], trees)
    ref = decode(q, k, v, lens, parents)
    check_attention(ref[0], ref[1], q, k, v, lens, parents)
    for fill in (math.nan, math.inf, -math.inf):
        for b in range(2):
            n = int(lens[b])
            first = n + (T - 1 if b == 0 else 2)
            k[b, :, first:] = fill
            v[b, :, first:] = fill
            q[b, :, first - n:] = fill
        out, lse, err = decode(q, k, v, lens, parents)
        assert err == 0
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    # node 2's key and value: only its own row sees them
    k[0, :, 262], v[0, :, 262] = math.nan, math.nan
    out, lse, err = decode(q, k, v, lens, parents)
    assert err == 0 and torch.isnan(out[0, :, 2]).all() and torch.isnan(lse[0, :, 2]).all()
    rest = [t for t in range(T) if t != 2]
    assert torch.equal(out[0, :, rest], ref[0][0, :, rest]) and torch.equal(lse[0, :, rest], ref[1][0, :, rest])
    # an infinity in one column of a seen value row: the row's whole output is NaN
    q, k, v, lens, parents = make(13, 2, G, 1, T, 400, D, [260, 380 - T], trees)
    v[0, 0, 262, 5] = math.inf
    out, lse, err = decode(q, k, v, lens, parents)
    assert err == 0 and torch.isnan(out[0, :, 2]).all()
    assert torch.equal(out[0, :, rest], ref[0][0, :, rest]) and torch.equal(lse, ref[1])


def test_nan_in_a_query_row_stays_in_that_row():
    q, k, v, lens, parents = make(14, 1, 4, 1, 5, 300, 128, [290], "random")
    ref = decode(q, k, v, lens, parents)
    q[0, 2, 3, 7] = math.nan
    out, lse, err = decode(q, k, v, lens, parents)
    assert err == 0 and torch.isnan(out[0, 2, 3]).all() and torch.isnan(lse[0, 2, 3])
    out[0, 2, 3], lse[0, 2, 3] = ref[0][0, 2, 3], ref[1][0, 2, 3]
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("D,G,T", [(64, 1, 1), (128, 4, 1), (128, 4, 8), (256, 2, 3), (256, 4, 16), (64, 4, 32), (128, 4, 25)])
def test_leading_keys_that_score_minus_infinity(D, G, T):
    """A row's first tiles give it no maximum; the later scores are far below 0, so that weights
    relative to 0 would vanish. Blocks of one tile and of several."""
    for Bz, Hkv in ((1, 1), (40, 8)):
        n, skip = 900, 300
        q, k, v, lens, _ = make(D + T, Bz, G * Hkv, Hkv, T, n + T, D, [n] * Bz)
        q[..., 3], k[..., 3] = -64.0, 60.0
        part = k[:, :, skip:].clone(), v[:, :, skip:].clone()
        k[:, :, :skip, 3] = math.inf
        out, lse, err = decode(q, k, v, lens)
        assert err == 0
        few = slice(0, 3)
        check_attention(out[few], lse[few], q[few], part[0][few], part[1][few], lens[few] - skip)
        assert torch.isfinite(lse).all() and torch.isfinite(out).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 40, 90])
def test_pairs_cut_into_many_parts(D, T):
    """32, 1280 and 2880 rows in all: the merge with eight, four and one warp per row."""
    q, k, v, lens, parents = make(D + T, 1, 32, 8, T, 1600, D, [1500], "random")
    out, lse, err = decode(q, k, v, lens, parents)
    assert err == 0
    check_attention(out, lse, q, k, v, lens, parents)


def test_empty_trees_and_a_full_cache():
    q, k, v, lens, parents = make(15, 2, 2, 1, 3, 64, 128, [61, 0], [[-2, -2, -2], [-1, -1, -2]])
    out, lse, err = decode(q, k, v, lens, parents)
    assert err == 0
    check_attention(out, lse, q, k, v, lens, parents)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()


def test_bad_lengths_and_parents_are_flagged_and_bounded():
    """Every clamped call still gives what the documented clamping says."""
    q, k, v, _, _ = make(16, 1, 2, 1, 4, 64, 128, [0])
    for lens, parents in (([-5], None), ([62], None), ([1 << 30], None), ([-(1 << 31)], None), ([10], [[-1, 1, 0, 1]]),
                          ([10], [[-1, 0, 77, -9]]), ([10], [[-2, 0, 1, -1]])):
        lens = torch.tensor(lens, dtype=torch.int32)
        parents = None if parents is None else torch.tensor(parents, dtype=torch.int32)
        out, lse, err = decode(q, k, v, lens, parents)
        assert err == B.DEVERR_BOUNDS, (lens, parents)
        fixed = parents
        if parents is not None:
            # an entry that is out of range or leads to a padding row ends the way up
            row = parents[0].tolist()
            fixed = torch.tensor([[p if p == -2 else (-1 if p < 0 or p >= t or row[p] == -2 else p) for t, p in enumerate(row)]],
                                 dtype=torch.int32)
        check_attention(out, lse, q, k, v, lens, fixed)
        kw = B.KeyWeights()
        w = kw(q.cuda(), k.cuda(), lse.cuda(), lens.cuda(), to_gpu(parents)).cpu().double().numpy()
        assert kw.status() == B.DEVERR_BOUNDS
        ref = OT.key_weights(q, k, lse, lens, fixed)
        tol = weights_tolerance(q, k, lse, lens, fixed, None, None, 1.0, ref)
        assert (np.abs(w - ref) <= tol).all()


def test_strided_views():
    """Caches that are slices of larger ones, rows of q from a packed projection, out in a
    token-major buffer; what lies between the rows of out stays as it was."""
    Bz, Hkv, G, T, D, N = 2, 3, 4, 5, 128, 200
    q, k, v, lens, parents = make(17, Bz, Hkv * G, Hkv, T, N, D, [100, 195], "random")
    packed = torch.zeros(Bz, T, Hkv * (G + 2), D, dtype=torch.bfloat16, device="cuda")
    qv = packed[:, :, :Hkv * G].transpose(1, 2)
    qv.copy_(q)
    kv = torch.full((Bz, N + 9, 2, Hkv, D), math.nan, dtype=torch.bfloat16, device="cuda")
    kk, vv = kv[:, 5:5 + N, 0].transpose(1, 2), kv[:, 5:5 + N, 1].transpose(1, 2)
    kk.copy_(k)
    vv.copy_(v)
    wide = torch.full((Bz, T, Hkv * G, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    op = B.TreeDecode()
    out, lse = op(qv, kk, vv, lens.cuda(), parents.cuda(), out=wide[..., D:].transpose(1, 2))
    assert op.status() == 0
    check_attention(out.cpu(), lse.cpu(), q, k, v, lens, parents)
    assert (wide[..., :D] == 7.0).all()
    w = B.KeyWeights()(qv, kk, lse, lens.cuda(), parents.cuda())
    w2 = B.KeyWeights()(q.cuda(), k.cuda(), lse, lens.cuda(), parents.cuda())
    assert torch.equal(w, w2)


def test_offsets_past_2_to_31():
    """The last sequence of a cache of 3.2e9 elements, against a copy of that sequence alone."""
    Bz, N, D = 25, 1000000, 128
    k = torch.empty(Bz, 1, N, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    n = 70000
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = torch.zeros(Bz, dtype=torch.int32, device="cuda")
    lens[-1] = n - 2
    for t in (k, v):
        t[:, :, :2] = 0
        t[-1, 0, :n] = torch.randn(n, D, generator=g, device="cuda", dtype=torch.bfloat16)
    q = torch.randn(Bz, 4, 2, D, generator=g, device="cuda", dtype=torch.bfloat16)
    out, lse = B.TreeDecode()(q, k, v, lens)
    s = torch.einsum("htd,jd->htj", q[-1].double(), k[-1, 0, :n].double()) / math.sqrt(D)
    s[:, 0, n - 1] = -math.inf
    assert torch.allclose(lse[-1].double(), s.logsumexp(-1), atol=1e-3, rtol=0)
    assert torch.allclose(out[-1].double(), s.softmax(-1) @ v[-1, 0, :n].double(), atol=2e-3, rtol=0)
    w = B.KeyWeights()(q, k, lse, lens)
    p = s.softmax(-1).sum((0, 1))
    assert ((w[-1, 0, :n].double() - p).abs() <= 1e-3 * p).all() and (w[-1, 0, n:] == 0).all()
    # rows moved within the last sequence
    op = B.CacheCompact()
    idx = torch.zeros(Bz, 1, 3, dtype=torch.int32, device="cuda")
    idx[-1, 0] = torch.tensor([5, 60000, 69999])
    count = torch.zeros(Bz, dtype=torch.int32, device="cuda")
    count[-1] = 3
    want = k[-1, 0, idx[-1, 0].long()].clone()
    op(k, v, idx, count)
    assert op.status() == 0 and torch.equal(k[-1, 0, :3], want)


def test_results_do_not_change_from_run_to_run():
    q, k, v, lens, parents = make(18, 3, 8, 2, 11, 3000, 128, [2900, 1000, 5], "random")
    ref = decode(q, k, v, lens, parents)
    op = B.TreeDecode()
    for _ in range(3):
        out, lse, _ = decode(q, k, v, lens, parents, op)
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_captured_calls_follow_growing_sequences():
    """A captured decode, weights and commit, replayed as the lengths (device data) grow."""
    q, k, v, lens, _ = make(19, 2, 4, 2, 2, 400, 128, [100, 3])
    gq, gk, gv, gl = q.cuda(), k.cuda(), v.cuda(), lens.cuda()
    op, kw = B.TreeDecode(), B.KeyWeights()
    out, lse = torch.empty_like(gq), torch.empty(2, 4, 2, device="cuda")
    w = torch.zeros(2, 2, 400, device="cuda")
    op(gq, gk, gv, gl, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(gq, gk, gv, gl, out=out, lse=lse)
        kw(gq, gk, lse, gl, weights_out=w)
    for n in ([100, 3], [101, 127], [300, 398], [5, 0]):
        lens = torch.tensor(n, dtype=torch.int32)
        gl.copy_(lens)
        w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check_attention(out.cpu(), lse.cpu(), q, k, v, lens)
        ref = OT.key_weights(q, k, lse.cpu(), lens)
        assert (np.abs(w.cpu().double().numpy() - ref) <= weights_tolerance(q, k, lse.cpu(), lens, None, None, None, 1.0, ref)).all()
    assert op.status() == 0 and kw.status() == 0


def test_calls_on_other_streams_and_two_at_once():
    """Two objects on two streams at the same time; memory made for a call belongs to its stream."""
    a = make(20, 2, 8, 2, 7, 2000, 128, [1900, 1200], "random")
    b = make(21, 2, 8, 2, 7, 2000, 128, [1000, 1993], "random")
    ref = [decode(*x) for x in (a, b)]
    ga, gb = [to_gpu(t) for t in a], [to_gpu(t) for t in b]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2 = B.TreeDecode(), B.TreeDecode()
    torch.cuda.synchronize()
    for _ in range(10):
        r1 = o1(*ga, stream=s1)
        r2 = o2(*gb, stream=s2)
    torch.cuda.synchronize()
    for got, want in ((r1, ref[0]), (r2, ref[1])):
        assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


def test_a_step_on_a_named_stream_with_tensors_that_are_dropped_at_once():
    """Every operator on a stream given by name; the inputs' last references go before the
    work is done, and new tensors are made meanwhile on the current stream."""
    side = torch.cuda.Stream()
    q, k, v, lens, parents = make(22, 2, 8, 2, 7, 2000, 128, [1900, 1200], "random")
    ref_out, ref_lse, _ = decode(q, k, v, lens, parents)
    w_ref = B.KeyWeights()(to_gpu(q), to_gpu(k), ref_lse.cuda(), lens.cuda(), parents.cuda()).cpu()
    keep_ref, new_ref = B.Evictor(500, 20).select(w_ref.cuda(), lens.cuda())
    tree, kw, ev = B.TreeDecode(), B.KeyWeights(), B.Evictor(500, 20)
    for _ in range(5):
        args = [to_gpu(x) for x in (q, k, v, lens, parents)]
        side.wait_stream(torch.cuda.current_stream())
        out, lse = tree(*args, stream=side)
        with torch.cuda.stream(side):
            w = torch.zeros(2, 2, 2000, device="cuda")
        kw(args[0], args[1], lse, args[3], args[4], weights_out=w, stream=side)
        keep, new = ev(args[1], args[2], w, args[3], stream=side)
        kept = [args[1], args[2]]
        del args
        junk = [torch.full((4, 2, 2000, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        side.synchronize()
        assert torch.equal(out.cpu(), ref_out) and torch.equal(lse.cpu(), ref_lse)
        assert torch.equal(keep, keep_ref) and torch.equal(new, new_ref)
        rows = keep.clamp_min(0).long().cpu()[..., None].expand(2, 2, 500, 128)
        for moved, whole in zip(kept, (k, v)):
            assert torch.equal(moved[:, :, :500].cpu(), torch.gather(whole, 2, rows))
        del junk
    assert tree.status() == 0 and kw.status() == 0 and ev.status() == 0


def test_two_graphs_with_an_object_each_replayed_in_turn():
    q, k, v, lens, parents = make(23, 2, 8, 2, 5, 900, 128, [800, 300], "random")
    g = [to_gpu(x) for x in (q, k, v, lens, parents)]
    graphs = []
    for T in (5, 2):  # the second with a smaller workspace need, from the same inputs' first rows
        op = B.TreeDecode()
        qq, par = g[0][:, :, :T].contiguous(), g[4][:, :T].contiguous()
        out, lse = torch.empty_like(qq), torch.empty(2, 8, T, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op(qq, g[1], g[2], g[3], par, out=out, lse=lse)
        graphs.append((graph, op, out, lse, decode(q[:, :, :T], k, v, lens, parents[:, :T].contiguous())))
    for _ in range(3):
        for graph, op, out, lse, ref in graphs:
            out.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out.cpu(), ref[0]) and torch.equal(lse.cpu(), ref[1]) and op.status() == 0


def test_an_empty_batch_launches_nothing():
    q, k, v = (torch.empty(0, h, n, 64, dtype=torch.bfloat16, device="cuda") for h, n in ((4, 1), (2, 9), (2, 9)))
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    out, lse = B.TreeDecode()(q, k, v, lens)
    assert out.shape == q.shape and lse.shape == (0, 4, 1)
    assert B.KeyWeights()(q, k, lse, lens).shape == (0, 2, 9)


# ---- key weights ----

# D, Hkv, G, T, N, lens, tree, token_major, scaled, decay
WEIGHT_CASES = [
    (128, 2, 4, 1, 300, [299, 0, 128], None, False, False, 1.0),
    (64, 1, 1, 1, 1, [0], None, False, False, 0.0),
    (64, 5, 3, 13, 700, [0, 687, 300], "random", True, True, 0.9),
    (256, 2, 4, 4, 600, [596, 77], None, False, False, 0.0),
    (256, 1, 16, 9, 500, [250, 491, 0], "random", True, True, 0.5),     # 144 rows
    (128, 1, 4, 32, 900, [868], None, False, False, 0.0),               # 128 rows
    (128, 2, 4, 33, 900, [800, 2], "random", False, True, 1.0),         # 132 rows
    (64, 1, 8, 64, 700, [636, 3], "random", True, False, 1.0),          # 512 rows
    (128, 1, 1, 256, 400, [144, 100], "random", False, True, 0.25),
    (128, 1, 2, 300, 700, [400, 10], None, False, True, 1.0),
    (256, 1, 3, 100, 700, [600], None, False, False, -1.5),
    (128, 16, 1, 2, 260, [258] + [7 * i for i in range(30)], "random", True, False, 1.0),
]


@pytest.mark.parametrize("case", WEIGHT_CASES, ids=lambda c: "d%d_h%d_g%d_t%d_n%d_b%d_%s" % (c[:5] + (len(c[5]), c[6])))
def test_key_weights_match_the_oracle(case):
    D, Hkv, G, T, N, lens, tree, major, scaled, decay = case
    q, k, v, lens, parents = make(D + T + N, len(lens), Hkv * G, Hkv, T, N, D, lens, tree, major)
    lse = torch.from_numpy(OT.tree_attention(q, k, v, lens, parents)[1]).float()
    g = torch.Generator().manual_seed(3)
    row = None
    if scaled:
        row = torch.where(torch.rand(len(lens), T, generator=g) < 0.5, torch.zeros(()), torch.randn(len(lens), T, generator=g))
    old = torch.rand(len(lens), Hkv, N, generator=g) if decay != 0 else None
    ref = OT.key_weights(q, k, lse, lens, parents, row, old, decay)
    tol = weights_tolerance(q, k, lse, lens, parents, row, old, decay, ref)
    kw = B.KeyWeights()
    args = (to_gpu(q), to_gpu(k), lse.cuda(), lens.cuda(), to_gpu(parents), to_gpu(row))
    w = kw(*args, weights_in=to_gpu(old), decay=decay)
    assert kw.status() == 0
    assert (np.abs(w.cpu().double().numpy() - ref) <= tol).all()
    # in place: the same values, entries past the keys held left as they were
    if old is not None:
        acc = old.cuda()
        kw(*args, weights_in=acc, decay=decay, weights_out=acc)
        held = torch.arange(N)[None, :] < (lens + T)[:, None]
        want = torch.where(held[:, None], w.cpu(), old)
        assert torch.equal(acc.cpu(), want)


@pytest.mark.parametrize("D,G,T,tree", [(64, 2, 2, None), (64, 4, 32, "random"), (64, 4, 100, "random"), (128, 2, 1, None), (128, 4, 7, "random"),
                                        (128, 5, 10, "random"), (128, 4, 30, "random"), (128, 4, 50, "random"), (128, 4, 80, "random"),
                                        (128, 4, 120, "random"), (128, 16, 40, "random"), (256, 2, 3, None), (256, 4, 8, "random"),
                                        (256, 4, 30, "random"), (256, 8, 30, "random")])
def test_key_weights_with_many_tiles_and_pairs_per_block(D, G, T, tree):
    """As for tree decode; 2 to 640 rows: one to four row tiles at once, one or two passes."""
    lens = [9000, 40, 0, 5117, 300, 9728 - T, 128]
    q, k, v, lens, parents = make(D + T, len(lens), 8 * G, 8, T, 9728, D, lens, tree, True)
    args = [to_gpu(x) for x in (q, k, k, lens, parents)]
    _, lse = reference(args, D)
    lse = lse.float()
    gen = torch.Generator().manual_seed(3)
    old = torch.rand(len(lens), 8, 9728, generator=gen).cuda()
    row = (torch.rand(len(lens), T, generator=gen) < 0.6).float().cuda()
    kw = B.KeyWeights()
    runs = [kw(args[0], args[1], lse, args[3], args[4], row, old, 0.5, torch.full_like(old, 7.0)) for _ in range(3)]
    assert kw.status() == 0 and torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])
    want = torch.full_like(old, 7.0).double()
    for b in range(len(lens)):
        end = int(lens[b]) + T
        vis = torch.from_numpy(OT.visible(int(lens[b]), None if parents is None else parents[b].tolist(), T, 9728)[:, :end]).cuda()
        s = args[0][b].double() @ args[1][b, :, :end].double().repeat_interleave(G, 0).transpose(1, 2) / math.sqrt(D)
        p = torch.where(vis, (s - lse[b].double()[..., None]).exp(), 0.0) * row[b].double()[None, :, None]
        want[b, :, :end] = p.view(8, G * T, end).sum(1) + 0.5 * old[b, :, :end].double()
    # every term is positive: the roundings of weights_tolerance, with |q . k| bounded by |q| |k|
    rows = T * G
    ds = float((D + 4) * ULP * args[0].double().norm(dim=-1).max() * args[1].double().norm(dim=-1).max() / math.sqrt(D))
    top = float(lse[torch.isfinite(lse)].abs().max())
    tol = want.abs() * (ds + 2 * ULP * (top + 64) + (rows + 8) * ULP) + rows * math.exp(-64)
    assert ((runs[0].double() - want).abs() <= tol).all()


def test_key_weights_leave_out_what_rows_of_scale_zero_hold():
    q, k, v, lens, parents = make(30, 1, 4, 2, 6, 300, 128, [280], [[-1, 0, 0, 1, 2, -2]])
    _, lse, _ = decode(q, k, v, lens, parents)
    row = torch.tensor([[1.0, 0.0, 1.0, 0.0, 2.0, 1.0]])
    kw = B.KeyWeights()
    ref = kw(q.cuda(), k.cuda(), lse.cuda(), lens.cuda(), parents.cuda(), row.cuda())
    for t in (1, 3, 5):
        q[:, :, t], lse[:, :, t] = math.nan, math.nan
        k[:, :, 280 + t] = math.nan
    w = kw(q.cuda(), k.cuda(), lse.cuda(), lens.cuda(), parents.cuda(), row.cuda(), weights_out=torch.zeros(1, 2, 300, device="cuda"))
    assert torch.equal(w, ref) and kw.status() == 0
    # decay 0 does not read the old weights
    old = torch.full((1, 2, 300), math.nan, device="cuda")
    assert torch.equal(kw(q.cuda(), k.cuda(), lse.cuda(), lens.cuda(), parents.cuda(), row.cuda(), old, 0.0), ref)


@pytest.mark.parametrize("D,T", [(64, 3), (128, 5), (256, 20)])
def test_key_weights_with_scales_of_both_signs_over_many_short_pairs(D, T):
    """Several pairs of one or two tiles for each block, every second batch's with a negative scale."""
    Bz, Hkv, N = 160, 6, 200
    lens = [(37 * b) % (N - T + 1) for b in range(Bz)]
    q, k, v, lens, _ = make(D, Bz, Hkv, Hkv, T, N, D, lens)
    lse = torch.from_numpy(OT.tree_attention(q, k, v, lens)[1]).float()
    row = torch.rand(Bz, T, generator=torch.Generator().manual_seed(5)) + 0.5
    row[::2, T // 2] *= -1.0
    ref = OT.key_weights(q, k, lse, lens, None, row)
    tol = weights_tolerance(q, k, lse, lens, None, row, None, 1.0, ref)
    kw = B.KeyWeights()
    runs = [kw(q.cuda(), k.cuda(), lse.cuda(), lens.cuda(), None, row.cuda()) for _ in range(10)]
    assert kw.status() == 0
    assert (np.abs(runs[0].cpu().double().numpy() - ref) <= tol).all()
    assert all(torch.equal(r, runs[0]) for r in runs)


@pytest.mark.parametrize("D,G,T", [(64, 1, 1), (128, 2, 3), (64, 4, 10), (128, 4, 40), (256, 4, 30)])
@pytest.mark.parametrize("scaled", [False, True])
def test_key_weights_of_keys_that_score_minus_infinity(D, G, T, scaled):
    """An infinite key that every row scores -inf gets no weight, whatever rows are left out."""
    q, k, v, lens, _ = make(D + T, 1, 2 * G, 2, T, 400, D, [330])
    q[..., 3] = -1.0 - q[..., 3].abs()
    lse = torch.from_numpy(OT.tree_attention(q, k, v, lens)[1]).float()
    row = None
    if scaled:
        row = torch.ones(1, T)
        row[:, ::2] = 0.0
    at = [0, 5, 130, 255, 300, 329]
    plain = k.clone()
    k[:, :, at, 3] = math.inf
    ref = OT.key_weights(q, plain, lse, lens, None, row)
    tol = weights_tolerance(q, plain, lse, lens, None, row, None, 1.0, ref)
    ref[:, :, at], tol[:, :, at] = 0.0, 0.0
    kw = B.KeyWeights()
    w = kw(q.cuda(), k.cuda(), lse.cuda(), lens.cuda(), None, None if row is None else row.cuda())
    assert kw.status() == 0
    assert (np.abs(w.cpu().double().numpy() - ref) <= tol).all()


# ---- eviction ----

def weights_like(g, *shape):
    """Accumulated weights: skewed, many of them zero, with ties."""
    w = torch.exp(2 * torch.randn(*shape, generator=g))
    w = torch.where(torch.rand(*shape, generator=g) < 0.3, torch.zeros(()), w)
    return torch.where(torch.rand(*shape, generator=g) < 0.2, torch.round(w), w)


@pytest.mark.parametrize("Hkv,N,lens,budget,recent", [
    (2, 300, [300, 299, 101, 100, 99, 0, 1], 100, 7),
    (1, 1, [1, 0], 1, 0),
    (3, 5000, [5000, 4097, 17], 1024, 64),
    (1, 20011, [20011], 3001, 100),
    (2, 70000, [70000, 64001], 2000, 0),
    (1, 200000, [199999], 50000, 1000),
    (2, 900, [900], 899, 0), (2, 900, [900], 899, 899), (2, 900, [900], 1, 1), (2, 900, [900, 1], 1, 0), (2, 900, [900], 2000, 10),
])
def test_select_equals_the_oracle(Hkv, N, lens, budget, recent):
    g = torch.Generator().manual_seed(N)
    w = weights_like(g, len(lens), Hkv, N)
    op = B.Evictor(budget, recent)
    keep, new = op.select(w.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"))
    ref_keep, ref_new = OE.select(w, lens, budget, recent)
    assert op.status() == 0
    assert np.array_equal(new.cpu().numpy(), ref_new) and np.array_equal(keep.cpu().numpy(), ref_keep)


@pytest.mark.parametrize("values", ["equal", "zeros", "special", "negative", "close"])
@pytest.mark.parametrize("N", [700, 60000])
def test_select_ties_and_special_values(values, N):
    g = torch.Generator().manual_seed(8)
    if values == "equal":
        w = torch.full((1, 1, N), 0.125)
    elif values == "zeros":
        w = torch.where(torch.rand(1, 1, N, generator=g) < 0.5, torch.zeros(()), -torch.zeros(()))
    elif values == "special":
        pool = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1.0, 1e-45, -1e-45, 3.4e38, -3.4e38])
        w = pool[torch.randint(0, 10, (1, 1, N), generator=g)]
    elif values == "negative":
        w = torch.randn(1, 1, N, generator=g)
    else:  # differ in the last bits only
        w = (1.0 + torch.randint(0, 40, (1, 1, N), generator=g) * 2.0 ** -23).float()
    op = B.Evictor(N // 3, 5)
    keep, new = op.select(w.cuda(), torch.tensor([N], dtype=torch.int32, device="cuda"))
    ref_keep, ref_new = OE.select(w, [N], N // 3, 5)
    assert np.array_equal(keep.cpu().numpy(), ref_keep) and np.array_equal(new.cpu().numpy(), ref_new)


def test_select_flags_lengths_outside_the_cache():
    w = torch.rand(3, 1, 50)
    op = B.Evictor(10, 2)
    keep, new = op.select(w.cuda(), torch.tensor([-1, 51, 50], dtype=torch.int32, device="cuda"))
    assert op.status() == B.DEVERR_BOUNDS
    ref = OE.select(w, [0, 50, 50], 10, 2)
    assert np.array_equal(keep.cpu().numpy(), ref[0]) and np.array_equal(new.cpu().numpy(), ref[1])


def cache_and_lists(seed, Bz, H, N, D, n_idx, heads, major, ascending=True):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(Bz, N, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    k, v = (t.transpose(1, 2) if major else t.transpose(1, 2).contiguous() for t in (k, v))
    w = torch.rand(Bz, H, N, generator=g)
    idx = torch.stack([torch.randperm(N, generator=g)[:n_idx] for _ in range(Bz * heads)]).view(Bz, heads, n_idx)
    return k, v, w, (idx.sort(-1).values if ascending else idx).int()


@pytest.mark.parametrize("Bz,H,N,D,n_idx,count,heads,major,in_place", [
    (2, 3, 1000, 64, 300, [300, 17], 3, True, True),
    (2, 3, 1000, 64, 300, [300, 0], 3, True, False),
    (1, 2, 5000, 128, 4999, [4999], 2, False, True),
    (1, 2, 5000, 128, 2500, [2500], 1, False, False),
    (3, 1, 700, 256, 500, [500, 499, 1], 1, True, True),
    (1, 1, 1, 8, 1, [1], 1, False, True),
    (2, 2, 130, 72, 65, [65, 64], 2, True, True),
    (2, 2, 130, 512, 129, [129, 128], 1, False, True),
    (1, 4, 300, 96, 256, [256], 4, False, False),
])
def test_compact_equals_the_oracle(Bz, H, N, D, n_idx, count, heads, major, in_place):
    k, v, w, idx = cache_and_lists(N + D, Bz, H, N, D, n_idx, heads, major)
    if not in_place and n_idx < N:  # any order, rows named twice
        idx = idx.flip(-1)
        idx[..., 0] = idx[..., -1]
    zero_end = torch.tensor([N - 1 - b for b in range(Bz)], dtype=torch.int32)
    gk, gv, gw = to_gpu(k), to_gpu(v), w.cuda()
    op = B.CacheCompact()
    dev = dict(weights=gw, zero_end=zero_end.cuda())
    cnt = torch.tensor(count, dtype=torch.int32)
    if in_place:
        op(gk, gv, idx.cuda(), cnt.cuda(), **dev)
        got, outs = (gk, gv, gw), (k, v, w)
    else:
        outs = (torch.full((Bz, H, n_idx + 5, D), 3.0).bfloat16(), torch.full((Bz, H, n_idx + 5, D), 4.0).bfloat16(),
                torch.full((Bz, H, n_idx + 5), 5.0))
        got = [t.cuda() for t in outs]
        op(gk, gv, idx.cuda(), cnt.cuda(), k_out=got[0], v_out=got[1], weights_out=got[2], **dev)
        assert torch.equal(gk.cpu(), k) and torch.equal(gv.cpu(), v) and torch.equal(gw.cpu(), w)
    assert op.status() == 0
    ref = OE.compact([t.float().numpy() for t in (k, v, w)], [t.float().numpy() for t in outs], idx.numpy(), count,
                     zero_end=zero_end, in_place=in_place)
    for a, b in zip(got, ref):
        assert np.array_equal(a.float().cpu().numpy(), b)


def test_compact_flags_and_skips_bad_entries():
    k, v, w, _ = cache_and_lists(5, 1, 2, 100, 64, 1, 1, False)
    idx = torch.tensor([[[3, 0, 200, -1, 50, 2147483647, -2147483648, 7]]], dtype=torch.int32)
    for in_place in (True, False):
        gk, gv, gw = k.cuda(), v.cuda(), w.cuda()
        outs = (gk, gv, gw) if in_place else tuple(torch.zeros_like(t) for t in (gk, gv, gw))
        op = B.CacheCompact()
        kw = {} if in_place else dict(k_out=outs[0], v_out=outs[1], weights_out=outs[2])
        before = [t.cpu().float().numpy() for t in outs]
        op(gk, gv, idx.cuda(), torch.tensor([8], dtype=torch.int32, device="cuda"), weights=gw, **kw)
        assert op.status() == B.DEVERR_SEL
        ref = OE.compact([t.float().numpy() for t in (k, v, w)], before, idx.numpy(), [8], in_place=in_place)
        for a, b in zip(outs, ref):
            assert np.array_equal(a.float().cpu().numpy(), b)
    # a start that puts rows outside the cache; counts outside the list are clamped
    for start, count in (([98], [8]), ([-3], [8]), ([0], [100]), ([5], [-4]), ([2147483647], [8]), ([-2147483648], [8])):
        idx = torch.arange(8, dtype=torch.int32).view(1, 1, 8) + 2
        gk, gv, gw = k.cuda(), v.cuda(), w.cuda()
        op = B.CacheCompact()
        op(gk, gv, idx.cuda(), torch.tensor(count, dtype=torch.int32, device="cuda"), weights=gw,
           start=torch.tensor(start, dtype=torch.int32, device="cuda"))
        assert op.status() == (B.DEVERR_SEL if start[0] not in (0, 5) else 0), start
        ref = OE.compact([t.float().numpy() for t in (k, v, w)], [t.float().numpy() for t in (k, v, w)], idx.numpy(), count,
                         start=start, in_place=True)
        for a, b in zip((gk, gv, gw), ref):
            assert np.array_equal(a.float().cpu().numpy(), b)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("Hkv,N,D,lens,budget,recent", [
    (2, 3000, 128, [3000, 1500, 700, 0], 1000, 50),
    (3, 20011, 64, [20011, 5], 3001, 100),
    (1, 9000, 256, [8999], 8000, 8000),
])
def test_evictor_keeps_what_the_oracle_keeps(in_place, Hkv, N, D, lens, budget, recent):
    Bz = len(lens)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(Bz, N, Hkv, D, generator=g).to(torch.bfloat16).transpose(1, 2) for _ in range(2))
    w = weights_like(g, Bz, Hkv, N)
    gk, gv, gw = to_gpu(k), to_gpu(v), w.cuda()
    op = B.Evictor(budget, recent)
    gl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if in_place:
        outs, kw, before = (gk, gv, gw), {}, (k, v, w)
    else:
        before = (torch.ones(Bz, Hkv, budget, D).bfloat16(), torch.ones(Bz, Hkv, budget, D).bfloat16(), torch.ones(Bz, Hkv, budget))
        outs = tuple(t.cuda() for t in before)
        kw = dict(k_out=outs[0], v_out=outs[1], weights_out=outs[2])
    keep, new = op(gk, gv, gw, gl, zero_end=gl if in_place else None, **kw)
    assert op.status() == 0
    ref_keep, ref_new = OE.select(w, lens, budget, recent)
    assert np.array_equal(keep.cpu().numpy(), ref_keep) and np.array_equal(new.cpu().numpy(), ref_new)
    ref = OE.compact([t.float().numpy() for t in (k, v, w)], [t.float().numpy() for t in before], ref_keep, ref_new,
                     zero_end=lens if in_place else None, in_place=in_place)
    for a, b in zip(outs, ref):
        assert np.array_equal(a.float().cpu().numpy(), b)


# ---- together ----

@pytest.mark.parametrize("captured", [False, True])
def test_a_serving_loop(captured):
    """Draft a tree, attend, add the accepted branch's weights, commit the branch, evict:
    rounds of it against the oracle, eager and as one replayed graph."""
    Bz, Hkv, G, T, D, N, budget, recent = 2, 2, 4, 6, 128, 160, 100, 20
    rng = np.random.default_rng(9)
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(Bz, Hkv, N, D, generator=g).to(torch.bfloat16) for _ in range(2))
    w = torch.zeros(Bz, Hkv, N)
    lens = torch.tensor([90, 40], dtype=torch.int32)
    gk, gv, gw, gl = k.cuda(), v.cuda(), w.cuda(), lens.cuda()
    gq = torch.empty(Bz, Hkv * G, T, D, dtype=torch.bfloat16, device="cuda")
    gpar = torch.empty(Bz, T, dtype=torch.int32, device="cuda")
    grow = torch.empty(Bz, T, device="cuda")
    gidx = torch.empty(Bz, 1, T, dtype=torch.int32, device="cuda")
    gcnt = torch.empty(Bz, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(gq), torch.empty(Bz, Hkv * G, T, device="cuda")
    keep = torch.empty(Bz, Hkv, budget, dtype=torch.int32, device="cuda")
    new = torch.empty(Bz, dtype=torch.int32, device="cuda")
    tree, kw, ev = B.TreeDecode(), B.KeyWeights(), B.Evictor(budget, recent)

    def step():
        tree(gq, gk, gv, gl, gpar, out=out, lse=lse)
        kw(gq, gk, lse, gl, gpar, grow, gw, 0.9, gw)
        ev.compact(gk, gv, gidx, gcnt, gw, start=gl, zero_end=gl + T)
        gl.add_(gcnt)
        ev.select(gw, gl, keep, new)
        ev.compact(gk, gv, keep, new, gw, zero_end=gl + T)
        gl.copy_(new)

    graph = None
    for it in range(8):
        trees = random_trees(it, Bz, T)
        q = torch.randn(Bz, Hkv * G, T, D, generator=g).to(torch.bfloat16)
        accepted = []
        for tr in trees:
            live = [t for t in range(T) if tr[t] != -2]
            accepted.append(sorted(OT.ancestors(tr)[live[int(rng.integers(len(live)))]]))
        row = torch.zeros(Bz, T)
        idx = torch.zeros(Bz, 1, T, dtype=torch.int32)
        for b, nodes in enumerate(accepted):
            row[b, nodes] = 1.0
            idx[b, 0, :len(nodes)] = torch.tensor(nodes, dtype=torch.int32)
        cnt = torch.tensor([len(n) for n in accepted], dtype=torch.int32)
        parents = torch.tensor(trees, dtype=torch.int32)
        # the draft model writes its keys and values behind the sequence
        for b in range(Bz):
            n = int(lens[b])
            for host, dev in ((k, gk), (v, gv)):
                host[b, :, n:n + T] = torch.randn(Hkv, T, D, generator=g).to(torch.bfloat16)
                dev[b, :, n:n + T] = host[b, :, n:n + T].cuda()
        for dev, host in ((gq, q), (gpar, parents), (grow, row), (gidx, idx), (gcnt, cnt)):
            dev.copy_(host)
        if captured and it == 1:
            graph = torch.cuda.CUDAGraph()
            state = [t.clone() for t in (gk, gv, gw, gl)]
            with torch.cuda.graph(graph):
                step()
            for t, s in zip((gk, gv, gw, gl), state):
                t.copy_(s)
        if graph is not None:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        check_attention(out.cpu(), lse.cpu(), q, k, v, lens, parents)
        ref = OT.key_weights(q, k, lse.cpu(), lens, parents, row, w, 0.9, w)
        # the weights of this step, checked through the rows that moved: the kernel's own
        # sums decide what is kept, so that the host follows them from here
        tol = weights_tolerance(q, k, lse.cpu(), lens, parents, row, w, 0.9, ref)
        kn, vn = k.float().numpy(), v.float().numpy()
        kn, vn, wn, tn = OE.compact([kn, vn, ref, tol], [kn, vn, ref, tol], idx.numpy(), cnt, start=lens, in_place=True)
        mid = lens + cnt
        ref_keep = keep.cpu().numpy()
        for b in range(Bz):
            n = int(mid[b])
            for h in range(Hkv):
                rows = ref_keep[b, h][:min(n, budget)]
                assert list(rows) == sorted(set(rows.tolist())) and (ref_keep[b, h][len(rows):] == -1).all()
                if n > budget:
                    assert list(rows[budget - recent:]) == list(range(n - recent, n))
                    gone = np.setdiff1d(np.arange(n - recent), rows)
                    best = rows[:budget - recent]
                    assert (wn[b, h, gone] - tn[b, h, gone]).max() <= (wn[b, h, best] + tn[b, h, best]).min()
        kn, vn, wn, tn = OE.compact([kn, vn, wn, tn], [kn, vn, wn, tn], ref_keep, np.minimum(mid.numpy(), budget), in_place=True)
        lens = torch.minimum(mid, torch.tensor(budget)).int()
        assert torch.equal(gl.cpu(), lens)
        k, v = torch.from_numpy(kn).to(torch.bfloat16), torch.from_numpy(vn).to(torch.bfloat16)
        for b in range(Bz):
            n = int(lens[b])
            assert torch.equal(gk[b, :, :n].cpu(), k[b, :, :n]) and torch.equal(gv[b, :, :n].cpu(), v[b, :, :n])
            got = gw[b, :, :n].cpu().double().numpy()
            assert (np.abs(got - wn[b, :, :n]) <= tn[b, :, :n]).all()
            assert (gw[b, :, n:int(mid[b]) + T].cpu() == 0).all()
        w = gw.cpu()
        k, v = gk.cpu(), gv.cpu()
    assert tree.status() == 0 and kw.status() == 0 and ev.status() == 0
