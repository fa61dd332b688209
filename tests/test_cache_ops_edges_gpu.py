"""Cache operators on the GPU where tiles, parts and calls meet: chains over several tiles of
drafted keys, the documented serving step run as a loop, K and V between one another. Against the definition in 64 bits (the tolerances of test_cache_ops_gpu.py)."""
import math
import os

import pytest
import torch

from mask_aware_block_mfa_b200 import binding as B

from .cache_util import make, to_gpu
from .test_cache_ops_gpu import large_tolerance, reference

pytestmark = pytest.mark.gpu


def check_large(args, runs):
    """Equal runs, the first within the tolerance of the definition."""
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
    out, lse = runs[0]
    D = args[0].shape[3]
    ref_out, ref_lse = reference(args, D)
    mass, _ = reference(args[:2] + [args[2].abs()] + args[3:], D)
    tol_out, tol_lse = large_tolerance(args, mass, ref_out, ref_lse)
    assert ((out.double() - ref_out).abs() <= tol_out).all()
    assert ((lse.double() - ref_lse).abs() <= tol_lse).all()


@pytest.mark.parametrize("D,G,T", [(64, 1, 1), (64, 4, 1), (128, 1, 1), (128, 4, 1), (128, 16, 1), (128, 8, 4), (128, 40, 1), (256, 4, 1),
                                   (256, 16, 4)])
def test_a_maximum_that_moves_before_and_in_a_tile_of_drafts_only(D, G, T):
    """Lengths of whole tiles, so that the drafted keys have a tile of their own, and scores that rise
    by more than the lazy maximum's slack in the last tile before it and again in it. Blocks of several
    tiles, with many pairs."""
    Bz, Hkv, N = 40, 8, 640
    lens = [128 * (1 + b % 4) for b in range(Bz)]
    q, k, v, lens, _ = make(D + G, Bz, Hkv * G, Hkv, T, N, D, lens)
    q[..., 3], k[..., 3] = 8.0, 0.0
    step = 2.0 * math.sqrt(D)  # 16 in the scores, 23 in powers of two
    for b in range(Bz):
        n = int(lens[b])
        k[b, :, n - 20 + b % 7, 3] = step
        k[b, :, n + T - 1, 3] = 2 * step
    args = [to_gpu(x) for x in (q, k, v, lens)] + [None]
    op = B.TreeDecode()
    runs = [op(*args) for _ in range(20)]
    assert op.status() == 0
    check_large(args, runs)


@pytest.mark.parametrize("T,G", [(300, 1), (300, 3), (520, 1)])
def test_chains_over_several_tiles_of_drafts_in_wide_heads(T, G):
    """Scores that rise from tile to tile through the drafted keys: every tile moves its rows' maxima."""
    Bz, Hkv, N, D = 6, 4, 1200, 256
    q, k, v, lens, _ = make(T + G, Bz, Hkv * G, Hkv, T, N, D, [0, 128, 500, 256, 37, N - T])
    q[..., 3] = 8.0
    k[..., 3] = (torch.arange(N) // 64).float() * math.sqrt(D)  # 8 in the scores for every 64 keys
    args = [to_gpu(x) for x in (q, k, v, lens)] + [None]
    op = B.TreeDecode()
    runs = [op(*args) for _ in range(10)]
    assert op.status() == 0
    check_large(args, runs)


def readme_serving_step():
    """The README's lines from the comment on serving to the end of their block."""
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        block = next(b for b in f.read().split("```") if "# serving from a cache" in b)
    return block[block.index("# serving from a cache"):]


def test_the_readme_step_run_as_a_loop_keeps_no_sums_of_keys_that_left():
    """Round after round of the documented step: what is behind the keys held has no weight left that
    the next drafts would begin with, lens follows the eviction, and the sums are those of the keys held."""
    step = compile(readme_serving_step(), "README.md", "exec")
    g = torch.Generator(device="cuda").manual_seed(31)
    Bz, Hkv, G, T, D, N, budget = 2, 2, 2, 6, 64, 8300, 8192

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    k, v = rand(Bz, Hkv, N, D), rand(Bz, Hkv, N, D)
    held = torch.tensor([budget - 3, 100], dtype=torch.int32)
    names = {"B": B, "k_cache": k, "v_cache": v, "lens": held.cuda(), "T": T, "w": torch.zeros(Bz, Hkv, N, device="cuda"),
             "parents": torch.tensor([[-1, 0, 0, 1, 2, -1]] * Bz, dtype=torch.int32, device="cuda")}
    nodes = torch.tensor([[[0, 2, 4]], [[0, 1, 0]]], dtype=torch.int32)
    count = torch.tensor([3, 2], dtype=torch.int32)
    rows = torch.zeros(Bz, T)
    for b in range(Bz):
        rows[b, nodes[b, 0, :count[b]].long()] = 1.0
    names |= {"accepted_nodes": nodes.cuda(), "n_accepted": count.cuda(), "accepted": rows.cuda()}
    for it in range(4):
        names["q_drafts"] = rand(Bz, Hkv * G, T, D)
        for b in range(Bz):  # the drafts' keys and values
            n = int(held[b])
            k[b, :, n:n + T], v[b, :, n:n + T] = rand(Hkv, T, D), rand(Hkv, T, D)
        exec(step, names)
        held = (held + count).clamp_max(budget)
        for b in range(Bz):
            assert (names["w"][b, :, int(held[b]):] == 0).all(), it
        assert torch.equal(names["lens"].cpu(), held), it
        # An accepted row sees accepted nodes only, so its weights add up to 1 over the keys that stay; an eviction
        # takes sums away. (Weights are off by the scores' and the lse's error: 2 (D + 4) 2^-23 |q| |k| / sqrt(D),
        # below 4e-4 for |q|, |k| < 13, and the sums of 8200 keys by 1e-3 / 2.)
        total = names["w"].double().sum(-1).cpu()
        want = (it + 1) * G * count.double()[:, None]
        assert (total <= want * (1 + 1e-3)).all() and (total[1] >= want[1] * (1 - 1e-3)).all()


LAYOUTS = {  # a buffer's shape from B, H, N, D, and its K and V as [B, H, N, D]
    "tokens": (lambda b, h, n, d: (b, n, 2, h, d), lambda x: (x[:, :, 0].transpose(1, 2), x[:, :, 1].transpose(1, 2))),
    "columns": (lambda b, h, n, d: (b, h, n, 2 * d), lambda x: x.chunk(2, -1)),
    "heads": (lambda b, h, n, d: (b, 2 * h, n, d), lambda x: (x[:, ::2], x[:, 1::2])),
    "batches": (lambda b, h, n, d: (b, 2, h * n, d),  # K head by head, V token by token
                lambda x: (x[:, 0].unflatten(1, (3, -1)), x[:, 1].unflatten(1, (-1, 3)).transpose(1, 2))),
}


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_rows_move_where_k_and_v_lie_between_one_another(layout, in_place):
    shape, views = LAYOUTS[layout]
    Bz, H, N, D, n = 2, 3, 500, 64, 200
    g = torch.Generator(device="cuda").manual_seed(7)
    buf = torch.randn(shape(Bz, H, N, D), generator=g, device="cuda", dtype=torch.bfloat16)
    out = buf if in_place else torch.zeros(shape(Bz, H, n, D), dtype=torch.bfloat16, device="cuda")
    (k, v), (ko, vo) = views(buf), views(out)
    idx = torch.stack([torch.randperm(N, generator=g, device="cuda")[:n].sort().values for _ in range(Bz * H)]).view(Bz, H, n).int()
    want_k, want_v = (torch.gather(x, 2, idx.long()[..., None].expand(Bz, H, n, D)) for x in (k, v))
    rest = [x[:, :, n:].clone() for x in (k, v)]
    op = B.CacheCompact()
    op(k, v, idx, torch.full((Bz,), n, dtype=torch.int32, device="cuda"), **({} if in_place else dict(k_out=ko, v_out=vo)))
    assert op.status() == 0
    assert torch.equal(ko[:, :, :n], want_k) and torch.equal(vo[:, :, :n], want_v)
    if in_place:
        assert torch.equal(k[:, :, n:], rest[0]) and torch.equal(v[:, :, n:], rest[1])


@pytest.mark.parametrize("D,G,T,tree", [(64, 2, 1, False), (128, 4, 1, False), (256, 2, 3, False), (128, 2, 6, True), (64, 2, 40, False),
                                        (128, 4, 30, True)])
def test_a_broken_value_reaches_its_rows_whatever_the_key_scores(D, G, T, tree):
    """Node 0's value holds an infinity and its key scores -inf: rows that see it are NaN in all columns, whether
    a pair is cut in front of the drafted keys' tile (few pairs) or not (many). A padding node changes nothing."""
    for Bz, Hkv in ((1, 1), (40, 8)):
        n = 256
        parents = None
        if tree:  # every second node follows node 0, the others the sequence; the last place is empty
            parents = [[-2 if t == T - 1 else (0 if t % 2 == 0 and t > 0 else -1) for t in range(T)]] * Bz
        q, k, v, lens, parents = make(D + T, Bz, G * Hkv, Hkv, T, n + T, D, [n] * Bz, parents)
        q[..., 3] = -1.0 - q[..., 3].abs()
        clean = [to_gpu(x) for x in (q, k, v, lens, parents)]
        k[:, :, n, 3], v[:, :, n, 5] = math.inf, math.inf
        if tree:
            v[:, :, n + T - 1] = math.inf
        op = B.TreeDecode()
        ref, _ = op(*clean)
        out, lse = op(*[to_gpu(x) for x in (q, k, v, lens, parents)])
        assert op.status() == 0
        for t in range(T):
            if tree and t == T - 1:
                assert (out[:, :, t] == 0).all() and torch.isneginf(lse[:, :, t]).all()
            elif tree and t % 2 == 1:
                assert torch.equal(out[:, :, t], ref[:, :, t])
            else:
                assert torch.isnan(out[:, :, t]).all() and torch.isfinite(lse[:, :, t]).all(), t
