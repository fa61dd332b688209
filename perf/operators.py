"""Serving operators over a key/value cache, as they are measured.

Three operators work on one contiguous cache, k and v ``[B, Hkv, N, D]`` in
bf16, of which batch b holds ``lens[b]`` keys:

* ``tree``: attention of T drafted tokens per sequence, a tree given by its
  parents (or a chain, or one token), over the cache. The drafted tokens'
  keys lie behind the sequence's own, at ``lens[b] + t``; node t sees every key
  before ``lens[b]``, itself and its ancestors.
* ``weights``: the attention weight that every key got from those rows, summed
  over rows and the query heads of its group, added to a decayed older sum.
* ``evict``: the keys to keep (the most recent ones, and of the others the ones
  of the largest accumulated weight), and their rows of k, v and the weights
  moved together.

With ``own`` false `run` computes them in elementary torch operations.
"""
from __future__ import annotations

import math
import random

import torch

own = False


def listed():
    return [
        # One token of one sequence over a short cache: the smallest call, where latency counts.
        {"name": "tree_one_token_1k", "op": "tree", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "N": 1024, "T": 1, "low": 1000, "high": 1000, "tree": 0,
         "token_major": False},
        # Plain decoding of a batch of sequences of different lengths.
        {"name": "tree_batch_8k", "op": "tree", "B": 16, "Hq": 32, "Hkv": 8, "D": 128, "N": 8192, "T": 1, "low": 500, "high": 8191, "tree": 0,
         "token_major": True},
        # One sequence of a long context, a tree of 26 drafts.
        {"name": "tree_long_64k", "op": "tree", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "N": 65536, "T": 26, "low": 65000, "high": 65000, "tree": 3,
         "token_major": False},
        # A batch with wide trees: 256 query rows for each key/value head.
        {"name": "tree_wide_32k", "op": "tree", "B": 8, "Hq": 32, "Hkv": 8, "D": 128, "N": 32768, "T": 64, "low": 16000, "high": 32704, "tree": 5,
         "token_major": False},
        # Wide heads, a chain of four drafts, a full cache.
        {"name": "tree_chain_d256", "op": "tree", "B": 8, "Hq": 32, "Hkv": 8, "D": 256, "N": 32768, "T": 4, "low": 30000, "high": 32764, "tree": 0,
         "token_major": False},
        # Narrow heads in groups of three, odd sizes, a sequence without any key yet.
        {"name": "tree_odd_d64", "op": "tree", "B": 3, "Hq": 15, "Hkv": 5, "D": 64, "N": 5003, "T": 13, "low": 0, "high": 4990, "tree": 9,
         "token_major": True},
        # The weights of one decoded token over a short cache.
        {"name": "weights_one_token_4k", "op": "weights", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "N": 4096, "T": 1, "low": 4000, "high": 4000, "tree": 0,
         "decay": 1.0, "scaled": False, "token_major": False},
        # The last 32 rows of each prompt, as the window that judges the prompt's keys.
        {"name": "weights_window_32k", "op": "weights", "B": 4, "Hq": 32, "Hkv": 8, "D": 128, "N": 32768, "T": 32, "low": 32736, "high": 32736, "tree": 0,
         "decay": 0.0, "scaled": False, "token_major": False},
        # A step of a batch with trees, of which only the accepted rows count.
        {"name": "weights_tree_32k", "op": "weights", "B": 8, "Hq": 32, "Hkv": 8, "D": 128, "N": 32768, "T": 16, "low": 9000, "high": 32700, "tree": 4,
         "decay": 0.95, "scaled": True, "token_major": True},
        # A short cache cut to half.
        {"name": "evict_1k", "op": "evict", "B": 1, "Hkv": 8, "D": 128, "N": 2048, "low": 2048, "high": 2048, "budget": 1024, "recent": 64,
         "token_major": False},
        # Prompts cut to a quarter before decoding begins.
        {"name": "evict_32k", "op": "evict", "B": 8, "Hkv": 8, "D": 128, "N": 32768, "low": 20000, "high": 32768, "budget": 8192, "recent": 512,
         "token_major": False},
        # Odd sizes, some sequences shorter than the budget.
        {"name": "evict_odd_d64", "op": "evict", "B": 5, "Hkv": 3, "D": 64, "N": 20011, "low": 1, "high": 20011, "budget": 3001, "recent": 100,
         "token_major": True},
    ]


def _log(rng, low, high):
    """A whole number, spread over the logarithm of [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["tree", "weights", "evict"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    N = _log(rng, 300, 65536)
    # keys over all sequences: at most what the largest listed case holds
    B = _log(rng, 1, max(1, min(64, (8 * 8 * 32768 * 128) // (N * Hkv * D))))
    low, high = (N, N) if rng.random() < 0.3 else (rng.randrange(0, N // 2), N)
    case = {"op": op, "B": B, "Hkv": Hkv, "D": D, "N": N, "low": low, "high": high, "token_major": rng.random() < 0.5}
    if op == "evict":
        case["budget"] = _log(rng, max(1, N // 32), N)
        case["recent"] = rng.randrange(0, case["budget"] // 2 + 1)
        return case
    G = rng.choice([1, 2, 3, 4, 4, 6, 8, 16])
    # query rows for each key/value head, so that the pairs stay below the largest listed case's
    rows = max(G, min(512, (8 * 8 * 32768 * 256 * 128) // (B * Hkv * N * D)))
    T = _log(rng, 1, max(1, min(128, rows // G, N // 2)))
    case |= {"Hq": Hkv * G, "T": T, "tree": rng.choice([0, 1 + rng.randrange(1000)])}
    case["low"], case["high"] = min(low, N - T), N - T
    if op == "weights":
        case |= {"decay": rng.choice([0.0, 0.9, 1.0]), "scaled": rng.random() < 0.5}
    return case


def _lens(case):
    """The sequences' lengths: the shortest and the longest first, the others spread between."""
    rng = random.Random("%d %d %d" % (case["B"], case["low"], case["high"]))
    lens = [case["high"], case["low"]] + [rng.randint(case["low"], case["high"]) for _ in range(case["B"])]
    return lens[: case["B"]]


def _parents(case):
    """The trees, one list of parents for each sequence: -1 follows the sequence's last token, -2 is no node (sequences draft
    different numbers of tokens). The first sequence has a node in every place."""
    rng = random.Random("%d %d" % (case["tree"], case["T"]))
    trees = []
    for b in range(case["B"]):
        size = case["T"] if b == 0 else rng.randint(max(1, case["T"] // 2), case["T"])
        trees.append([(-1 if t == 0 or rng.random() < 1.5 / case["T"] else rng.randrange(max(0, t - 8), t)) if t < size else -2
                      for t in range(case["T"])])
    return trees


def _cache(case, g):
    """A [B, Hkv, N, D] cache, in this order in memory or token by token."""
    B, H, N, D = case["B"], case["Hkv"], case["N"], case["D"]
    if case["token_major"]:
        return torch.randn(B, N, H, D, generator=g, device="cuda", dtype=torch.bfloat16).transpose(1, 2)
    return torch.randn(B, H, N, D, generator=g, device="cuda", dtype=torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    B, Hkv, N, D = case["B"], case["Hkv"], case["N"], case["D"]
    s = {"case": dict(case), "k": _cache(case, g), "lens": torch.tensor(_lens(case), dtype=torch.int32, device="cuda")}
    if case["op"] == "evict":
        s["v"] = _cache(case, g)
        # accumulated weights: a few keys hold most, and some were never attended
        w = torch.exp(2.0 * torch.randn(B, Hkv, N, generator=g, device="cuda"))
        s["weights"] = torch.where(torch.rand(B, Hkv, N, generator=g, device="cuda") < 0.3, torch.zeros_like(w), w)
        R = case["budget"]
        s["k_out"] = torch.zeros(B, Hkv, R, D, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros(B, Hkv, R, D, dtype=torch.bfloat16, device="cuda")
        s["weights_out"] = torch.zeros(B, Hkv, R, device="cuda")
        return s
    s["q"] = torch.randn(B, case["Hq"], case["T"], D, generator=g, device="cuda", dtype=torch.bfloat16)
    s["parents"] = torch.tensor(_parents(case), dtype=torch.int32, device="cuda") if case["tree"] else None
    if case["op"] == "tree":
        s["v"] = _cache(case, g)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, case["Hq"], case["T"], device="cuda")
        return s
    s["lse"] = _lse(s)
    s["row_scale"] = (torch.rand(B, case["T"], generator=g, device="cuda") < 0.4).float() if case["scaled"] else None
    s["weights_in"] = torch.rand(B, Hkv, N, generator=g, device="cuda") if case["decay"] != 0.0 else None
    s["weights_out"] = torch.zeros(B, Hkv, N, device="cuda")
    return s


# ---- the plain forms ----

def _visible(s):
    """[B, T, N]: which keys each row sees."""
    case, lens = s["case"], s["lens"].long()
    B, T, N = case["B"], case["T"], case["N"]
    if s["parents"] is None:
        parents = (torch.arange(T, device="cuda") - 1).expand(B, T)
    else:
        parents = s["parents"].long()
    nodes = torch.arange(T, device="cuda")
    step = (parents[:, :, None] == nodes) | (nodes[:, None] == nodes)
    # (1 + step to the parent)^T is positive at a node's ancestors and itself
    above = torch.linalg.matrix_power(step.double(), T) > 0
    at = torch.arange(N, device="cuda")[None, :] - lens[:, None]
    inside = torch.gather(above, 2, at.clamp(0, T - 1)[:, None, :].expand(B, T, N)) & (at < T)[:, None, :]
    return (inside | (at < 0)[:, None, :]) & (parents != -2)[:, :, None]


def _scores(s):
    """[B, Hkv, G, T, N] in 32 bits, -inf where a row does not see a key."""
    case = s["case"]
    B, Hkv, T, D = case["B"], case["Hkv"], case["T"], case["D"]
    q = s["q"].float().reshape(B, Hkv, -1, D)
    x = torch.matmul(q, s["k"].float().transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, -1, T, case["N"])
    return x.masked_fill_(~_visible(s)[:, None, None], -math.inf)


def _lse(s):
    x = _scores(s)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    return (torch.log(x.sub_(m).exp_().sum(-1)) + m.squeeze(-1)).reshape(s["q"].shape[:3])


def _plain_tree(s):
    B, Hq, T, D = s["q"].shape
    x = _scores(s)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, s["k"].shape[1], -1, s["k"].shape[2]), s["v"].float()).view(*p.shape[:-1], D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (torch.log(total) + m).squeeze(-1)
    return out.reshape(B, Hq, T, D).to(torch.bfloat16), lse.reshape(B, Hq, T)


def _plain_weights(s):
    case = s["case"]
    B, Hkv, T, N = case["B"], case["Hkv"], case["T"], case["N"]
    lse = s["lse"].view(B, Hkv, -1, T, 1)
    p = _scores(s).sub_(torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))).exp_()
    if s["row_scale"] is not None:
        p = p * s["row_scale"][:, None, None, :, None]
    w = p.sum((2, 3))
    if s["weights_in"] is not None:
        w = w + case["decay"] * s["weights_in"]
    held = torch.arange(N, device="cuda")[None, :] < (s["lens"].long() + T)[:, None]
    return torch.where(held[:, None], w, s["weights_out"])


def _plain_evict(s):
    case, w = s["case"], s["weights"]
    B, Hkv, N, D = s["k"].shape
    R, lens = case["budget"], s["lens"].long()
    at = torch.arange(N, device="cuda")
    last = (at[None, :] >= (lens - case["recent"])[:, None])[:, None]
    held = (at[None, :] < lens[:, None])[:, None]
    rank = torch.where(held, torch.where(last, math.inf, w), -math.inf)
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :R]
    new = lens.clamp_max(R)
    slot = torch.arange(R, device="cuda")[None, None, :]
    filled = slot < new[:, None, None]
    keep = torch.sort(torch.where(filled, best, N), dim=-1).values
    row = keep.clamp_max(N - 1)
    k = torch.where(filled[..., None], torch.gather(s["k"], 2, row[..., None].expand(B, Hkv, R, D)), s["k_out"])
    v = torch.where(filled[..., None], torch.gather(s["v"], 2, row[..., None].expand(B, Hkv, R, D)), s["v_out"])
    weights = torch.where(filled, torch.gather(w, 2, row), s["weights_out"])
    return torch.where(filled, keep, -1).int(), new.int(), k, v, weights


def run(s):
    case = s["case"]
    if own:
        from mask_aware_block_mfa_b200 import binding
        # what a serving loop keeps between calls: the workspace and the error word
        if "op" not in s:
            s["op"] = {"tree": binding.TreeDecode, "weights": binding.KeyWeights}[case["op"]]() if case["op"] != "evict" else \
                binding.Evictor(case["budget"], case["recent"])
        if case["op"] == "tree":
            return s["op"](s["q"], s["k"], s["v"], s["lens"], s["parents"], out=s["out"], lse=s["lse"])
        if case["op"] == "weights":
            return s["op"](s["q"], s["k"], s["lse"], s["lens"], s["parents"], row_scale=s["row_scale"], weights_in=s["weights_in"],
                           decay=case["decay"], weights_out=s["weights_out"])
        keep, new = s["op"](s["k"], s["v"], s["weights"], s["lens"], k_out=s["k_out"], v_out=s["v_out"], weights_out=s["weights_out"])
        return keep, new, s["k_out"], s["v_out"], s["weights_out"]
    return {"tree": _plain_tree, "weights": _plain_weights, "evict": _plain_evict}[case["op"]](s)


def work(case):
    B, Hkv, N, D = case["B"], case["Hkv"], case["N"], case["D"]
    lens = _lens(case)
    if case["op"] == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        # weights read once; kept rows of k, v and the weights read and written, the list written
        return {"bytes": Hkv * (4 * sum(lens) + kept * (2 * 2 * 2 * D + 4 + 4)) + 8 * B, "flops": 0}
    T, Hq = case["T"], case["Hq"]
    trees = _parents(case) if case["tree"] else [[t - 1 for t in range(T)]] * B
    pairs = 0
    for n, tree in zip(lens, trees):
        depth = []
        for p in tree:
            depth.append(0 if p == -2 else 1 + (depth[p] if p >= 0 else 0))
            pairs += n + depth[-1] if p != -2 else 0
    keys = sum(n + sum(p != -2 for p in tree) for n, tree in zip(lens, trees))
    small = 4 * B + (4 * B * T if case["tree"] else 0) + B * Hq * T * (2 * D + 4)  # lens, parents, q and lse
    if case["op"] == "tree":
        return {"bytes": small + Hkv * keys * 2 * 2 * D + B * Hq * T * 2 * D, "flops": 4 * D * Hq * pairs}
    sums = Hkv * 4 * (sum(lens) + B * T) * (2 if case["decay"] != 0.0 else 1)
    return {"bytes": small + Hkv * keys * 2 * D + sums + (4 * B * T if case["scaled"] else 0), "flops": 2 * D * Hq * pairs}


# ---- from the definitions, in 64 bits ----

def _rows_seen(n, tree):
    """For each node its keys, as the list of nodes on the way up (None: no node)."""
    seen = []
    for t, p in enumerate(tree):
        seen.append(None if p == -2 else ([] if p < 0 else seen[p]) + [t])
    return seen


def exact(case, seed):
    s = prepare(case, seed)
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    lens = s["lens"].tolist()
    if case["op"] == "evict":
        R, recent = case["budget"], case["recent"]
        k, v, weights = (s[n].double() for n in ("k_out", "v_out", "weights_out"))
        for b, n in enumerate(lens):
            first = max(0, n - recent)
            for g in range(Hkv):
                w = s["weights"][b, g, :first].double()
                if n <= R:
                    rows = torch.arange(n, device="cuda")
                else:
                    order = torch.argsort(-w, stable=True)[: R - min(recent, n)]
                    rows = torch.cat([torch.sort(order).values, torch.arange(first, n, device="cuda")])
                k[b, g, : len(rows)] = s["k"][b, g, rows].double()
                v[b, g, : len(rows)] = s["v"][b, g, rows].double()
                weights[b, g, : len(rows)] = s["weights"][b, g, rows].double()
        return None, None, k, v, weights
    T, G = case["T"], case["Hq"] // Hkv
    trees = s["parents"].tolist() if s["parents"] is not None else [list(range(-1, T - 1))] * B
    out = torch.zeros(B, case["Hq"], T, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, case["Hq"], T), -math.inf, dtype=torch.float64, device="cuda")
    sums = None if case["op"] == "tree" else s["weights_out"].double()
    for b, n in enumerate(lens):
        blocked = torch.ones(T, n + T, dtype=torch.bool)
        live = []
        for t, nodes in enumerate(_rows_seen(n, trees[b])):
            if nodes is not None:
                live.append(t)
                blocked[t, :n] = False
                blocked[t, [n + x for x in nodes]] = False
        live = torch.tensor(live, device="cuda")
        blocked = blocked.to("cuda")[live]
        for g in range(Hkv):
            heads = slice(g * G, (g + 1) * G)
            x = torch.einsum("htd,jd->htj", s["q"][b, heads][:, live].double(), s["k"][b, g, : n + T].double()) / math.sqrt(D)
            x = x.masked_fill(blocked, -math.inf)
            if sums is None:
                lse[b, heads.start:heads.stop, live] = torch.logsumexp(x, -1)
                out[b, heads.start:heads.stop, live] = torch.einsum("htj,jd->htd", torch.softmax(x, -1), s["v"][b, g, : n + T].double())
                continue
            p = torch.exp(x - s["lse"][b, heads][:, live].double()[..., None])
            if s["row_scale"] is not None:
                p = p * s["row_scale"][b, live].double()[None, :, None]
            old = 0.0 if s["weights_in"] is None else case["decay"] * s["weights_in"][b, g, : n + T].double()
            sums[b, g, : n + T] = p.sum((0, 1)) + old
    return (out, lse) if sums is None else sums
