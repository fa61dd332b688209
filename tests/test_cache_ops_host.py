"""What the cache operators refuse, on the host: no call here gets past its checks,
so none touches a GPU."""
import ctypes

import pytest
import torch

from mask_aware_block_mfa_b200 import binding as B
from mask_aware_block_mfa_b200 import build as BUILD

PTR = 1 << 20  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    BUILD.build()
    return B.load()


def tensor(shape, data=PTR, dtype=B.MFA_BF16, stride=None):
    t = B.MfaTensor()
    t.data, t.dtype = data, dtype
    t.B, t.H, t.N, t.D = shape
    s, acc = [], 1
    for n in reversed(shape):
        s.insert(0, acc)
        acc *= max(n, 1)
    for a, x in enumerate(stride or s):
        t.stride[a] = x
    return t


def tree_call(lib, **kw):
    a = dict(q=tensor((2, 8, 3, 128)), k=tensor((2, 2, 100, 128)), v=tensor((2, 2, 100, 128)), lens=PTR, parents=PTR,
             out=tensor((2, 8, 3, 128)), lse=PTR, ws=PTR, ws_bytes=1 << 40, err=PTR)
    a.update(kw)
    return lib.mfa_tree_decode(*(a[n] for n in ("q", "k", "v", "lens", "parents", "out", "lse", "ws", "ws_bytes", "err")), None)


def weights_call(lib, **kw):
    a = dict(q=tensor((2, 8, 3, 128)), k=tensor((2, 2, 100, 128)), lse=PTR, lens=PTR, parents=None, row=None, w_in=None,
             decay=1.0, w_out=PTR, err=PTR)
    a.update(kw)
    return lib.mfa_key_weights(*(a[n] for n in ("q", "k", "lse", "lens", "parents", "row", "w_in", "decay", "w_out", "err")), None)


Q = (2, 8, 3, 128)
K = (2, 2, 100, 128)
# what is changed, and the answer of both calls
SHARED = [
    (dict(lens=None), B.MFA_ERR_INVALID_ARG),
    (dict(lse=None), B.MFA_ERR_INVALID_ARG),
    (dict(err=None), B.MFA_ERR_INVALID_ARG),
    (dict(q=None), B.MFA_ERR_INVALID_ARG),
    (dict(k=None), B.MFA_ERR_INVALID_ARG),
    (dict(q=tensor(Q, data=None)), B.MFA_ERR_INVALID_ARG),
    (dict(q=tensor(Q, dtype=B.MFA_F32)), B.MFA_ERR_UNSUPPORTED),
    (dict(q=tensor(Q, data=PTR + 8)), B.MFA_ERR_UNSUPPORTED),
    (dict(k=tensor(K, stride=(25600, 12800, 132, 1))), B.MFA_ERR_UNSUPPORTED),
    (dict(k=tensor(K, stride=(25600, 12800, 128, 2))), B.MFA_ERR_UNSUPPORTED),
    (dict(k=tensor(K, stride=(25600, 0, 128, 1))), B.MFA_ERR_UNSUPPORTED),
    (dict(k=tensor((3, 2, 100, 128))), B.MFA_ERR_SHAPE_MISMATCH),
    (dict(k=tensor((2, 3, 100, 128))), B.MFA_ERR_SHAPE_MISMATCH),
    (dict(k=tensor((2, 2, 100, 64))), B.MFA_ERR_SHAPE_MISMATCH),
]


@pytest.mark.parametrize("case", range(len(SHARED)))
def test_tree_decode_and_key_weights_refuse(lib, case):
    change, want = SHARED[case]
    assert tree_call(lib, **change) == want
    assert weights_call(lib, **change) == want


@pytest.mark.parametrize("D", [8, 32, 96, 192, 512])
def test_head_sizes_not_served(lib, D):
    q, k = tensor((1, 2, 1, D)), tensor((1, 1, 9, D))
    assert tree_call(lib, q=q, k=k, v=k, out=q) == B.MFA_ERR_UNSUPPORTED
    assert weights_call(lib, q=q, k=k) == B.MFA_ERR_UNSUPPORTED
    assert lib.mfa_tree_decode_workspace_bytes(1, 2, 1, 1, D) == 0


def test_sizes_not_served(lib):
    big = tensor((1, 2, B.TREE_MAX_NODES + 1, 64))
    k = tensor((1, 1, 900, 64))
    assert tree_call(lib, q=big, k=k, v=k, out=big) == B.MFA_ERR_UNSUPPORTED          # a tree of too many nodes
    assert weights_call(lib, q=big, k=k, parents=PTR) == B.MFA_ERR_UNSUPPORTED
    q = tensor((1, 2, 1, 64))
    for n in (0, 1 << 30):
        k = tensor((1, 1, n, 64))
        assert tree_call(lib, q=q, k=k, v=k, out=q) == B.MFA_ERR_UNSUPPORTED
        assert weights_call(lib, q=q, k=k) == B.MFA_ERR_UNSUPPORTED
    assert weights_call(lib, q=tensor((1, 2, 0, 64)), k=tensor((1, 1, 9, 64))) == B.MFA_ERR_UNSUPPORTED
    assert weights_call(lib, w_out=None) == B.MFA_ERR_INVALID_ARG


def test_tree_decode_workspace(lib):
    need = lib.mfa_tree_decode_workspace_bytes(2, 8, 2, 3, 128)
    assert need > 0
    assert tree_call(lib, ws=None) == B.MFA_ERR_INVALID_ARG
    assert tree_call(lib, ws=PTR + 16) == B.MFA_ERR_INVALID_ARG
    assert tree_call(lib, ws_bytes=need - 1) == B.MFA_ERR_INVALID_ARG
    assert lib.mfa_tree_decode_workspace_bytes(2, 7, 2, 3, 128) == 0
    assert lib.mfa_tree_decode_workspace_bytes(2, 0, 2, 3, 128) == 0
    assert lib.mfa_tree_decode_workspace_bytes(-1, 8, 2, 3, 128) == 0


def test_tree_decode_shapes(lib):
    assert tree_call(lib, v=tensor((2, 2, 99, 128))) == B.MFA_ERR_SHAPE_MISMATCH
    assert tree_call(lib, out=tensor((2, 8, 4, 128))) == B.MFA_ERR_SHAPE_MISMATCH
    assert tree_call(lib, v=tensor(K, dtype=B.MFA_F32)) == B.MFA_ERR_UNSUPPORTED


def test_nothing_to_do_succeeds_without_a_launch(lib):
    q, k = tensor((0, 8, 3, 128)), tensor((0, 2, 100, 128))
    assert tree_call(lib, q=q, k=k, v=k, out=q) == B.MFA_OK
    assert weights_call(lib, q=q, k=k) == B.MFA_OK
    q = tensor((2, 8, 0, 128))
    assert tree_call(lib, q=q, out=q) == B.MFA_OK
    assert lib.mfa_evict_select(None, None, 0, 2, 10, 5, 1, None, None, PTR, None) == B.MFA_OK
    k = tensor((0, 2, 100, 128))
    assert lib.mfa_cache_compact(k, k, None, None, None, 1, 0, None, None, k, k, None, PTR, None) == B.MFA_OK


@pytest.mark.parametrize("args,want", [
    ((PTR, PTR, 1, 0, 10, 5, 1, PTR, PTR * 2, PTR), B.MFA_ERR_INVALID_ARG),
    ((PTR, PTR, 1, 2, 0, 5, 1, PTR, PTR * 2, PTR), B.MFA_ERR_INVALID_ARG),
    ((PTR, PTR, 1, 2, 10, 0, 0, PTR, PTR * 2, PTR), B.MFA_ERR_INVALID_ARG),
    ((PTR, PTR, 1, 2, 10, 5, 6, PTR, PTR * 2, PTR), B.MFA_ERR_INVALID_ARG),
    ((PTR, PTR, 1, 2, 10, 5, -1, PTR, PTR * 2, PTR), B.MFA_ERR_INVALID_ARG),
    ((None, PTR, 1, 2, 10, 5, 1, PTR, PTR * 2, PTR), B.MFA_ERR_INVALID_ARG),
    ((PTR, None, 1, 2, 10, 5, 1, PTR, PTR * 2, PTR), B.MFA_ERR_INVALID_ARG),
    ((PTR, PTR, 1, 2, 10, 5, 1, None, PTR * 2, PTR), B.MFA_ERR_INVALID_ARG),
    ((PTR, PTR, 1, 2, 10, 5, 1, PTR, PTR, PTR), B.MFA_ERR_INVALID_ARG),        # new_lens is lens
    ((PTR, PTR, 1, 2, 10, 5, 1, PTR, PTR * 2, None), B.MFA_ERR_INVALID_ARG),
    ((PTR, PTR, 1, 2, 1 << 30, 5, 1, PTR, PTR * 2, PTR), B.MFA_ERR_UNSUPPORTED),
    ((PTR, PTR, 65536, 2, 10, 5, 1, PTR, PTR * 2, PTR), B.MFA_ERR_UNSUPPORTED),
])
def test_select_refuses(lib, args, want):
    assert lib.mfa_evict_select(*args, None) == want


def compact_call(lib, **kw):
    far = 1 << 32
    a = dict(k=tensor((1, 2, 50, 64)), v=tensor((1, 2, 50, 64), PTR * 2), w=None, start=None, idx=PTR, heads=1, n=4, count=PTR,
             zero=None, ko=tensor((1, 2, 20, 64), far), vo=tensor((1, 2, 20, 64), far * 2), wo=None, err=PTR)
    a.update(kw)
    return lib.mfa_cache_compact(*(a[n] for n in ("k", "v", "w", "start", "idx", "heads", "n", "count", "zero", "ko", "vo", "wo", "err")), None)


def test_compact_refuses(lib):
    k, v = tensor((1, 2, 50, 64)), tensor((1, 2, 50, 64), PTR * 2)
    inv, shape, uns = B.MFA_ERR_INVALID_ARG, B.MFA_ERR_SHAPE_MISMATCH, B.MFA_ERR_UNSUPPORTED
    for change, want in (
            (dict(err=None), inv), (dict(count=None), inv), (dict(idx=None), inv), (dict(heads=0), inv), (dict(n=-1), inv),
            (dict(w=PTR * 8), inv), (dict(wo=PTR * 8), inv), (dict(zero=PTR), inv),
            (dict(heads=3), shape), (dict(v=tensor((1, 2, 49, 64), PTR * 2)), shape), (dict(ko=tensor((1, 2, 20, 128), 1 << 32)), shape),
            (dict(vo=tensor((1, 2, 21, 64), 1 << 33)), shape),
            (dict(k=tensor((1, 2, 50, 64), dtype=B.MFA_F32)), uns), (dict(k=tensor((1, 2, 50, 64), PTR + 2)), uns),
            # outputs that share bytes with the inputs, or with one another
            (dict(ko=tensor((1, 2, 20, 64), PTR + 1024)), inv), (dict(ko=tensor((1, 2, 20, 64), PTR * 2)), inv),
            (dict(vo=tensor((1, 2, 20, 64), 1 << 32)), inv), (dict(ko=k, vo=tensor((1, 2, 50, 64), 1 << 33)), inv),
            (dict(ko=tensor((1, 2, 50, 64), 1 << 32), vo=v), inv),
            (dict(ko=tensor((1, 2, 50, 64), PTR + 128), vo=v), inv),
            # in place with another weights_out; apart with the same
            (dict(ko=k, vo=v, w=PTR * 8, wo=PTR * 9), inv), (dict(w=PTR * 8, wo=PTR * 8), inv),
            (dict(k=k, v=k, ko=k, vo=k), inv)):
        assert compact_call(lib, **change) == want, change
    for D in (4, 12, 520, 1024):
        t = [tensor((1, 2, 50, D), PTR << i, stride=(16384 * 8, 8192 * 8, 1024, 1)) for i in range(4)]
        assert compact_call(lib, k=t[0], v=t[1], ko=t[2], vo=t[3]) == uns


def test_compact_refuses_long_lists_and_tensors_whose_rows_share_bytes(lib):
    assert compact_call(lib, n=1 << 30) == B.MFA_ERR_UNSUPPORTED
    k, v = tensor((1, 2, 50, 64)), tensor((1, 2, 50, 64), PTR + 64)
    assert compact_call(lib, k=k, v=v, ko=k, vo=v) == B.MFA_ERR_INVALID_ARG
    assert compact_call(lib, vo=tensor((1, 2, 20, 64), (1 << 32) + 112)) == B.MFA_ERR_INVALID_ARG


def test_null_and_misuse_through_ctypes(lib):
    assert lib.mfa_tree_decode(None, None, None, None, None, None, None, None, 0, None, None) == B.MFA_ERR_INVALID_ARG
    assert lib.mfa_key_weights(None, None, None, None, None, None, None, ctypes.c_float(0), None, None, None) == B.MFA_ERR_INVALID_ARG
    assert lib.mfa_cache_compact(*[None] * 5, 1, 1, *[None] * 7) == B.MFA_ERR_INVALID_ARG


def test_the_wrappers_run_on_cuda_only():
    for make in (B.TreeDecode, B.KeyWeights, B.CacheCompact, lambda d: B.Evictor(4, 1, d)):
        with pytest.raises(ValueError, match="CUDA"):
            make("cpu")


def test_the_wrappers_refuse_host_tensors_and_wrong_types():
    dev = torch.device("cuda", 0)
    t = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        B._cache_desc("q", t, dev)
    with pytest.raises(ValueError, match="four dimensions"):
        B._cache_desc("q", t[0], t.device)
    with pytest.raises(ValueError, match="bfloat16"):
        B._cache_desc("q", t.float(), t.device)
    with pytest.raises(ValueError, match="shape"):
        B._cache_desc("v", t, t.device, torch.Size([1, 2, 4, 64]))
    with pytest.raises(ValueError, match="lens must be a CUDA tensor"):
        B._array_ptr("lens", torch.zeros(2, dtype=torch.int32), dev, torch.int32, (2,))
