"""Thin ctypes binding of libmfa.so (argument marshalling only).

Every computation runs in the library's CUDA kernels; this module only turns
torch tensors and mask descriptions into the C structs of ``include/mfa.h``
and calls the entry points of the same names. It raises if the library is
missing or a call fails: there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
from typing import Optional

import numpy as np
import torch

from . import workloads as W

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmfa.so")

MFA_OK, MFA_ERR_INVALID_ARG, MFA_ERR_UNSUPPORTED, MFA_ERR_SHAPE_MISMATCH, MFA_ERR_CUDA, MFA_ERR_DEVICE = range(6)
MFA_BF16, MFA_F32 = 0, 1
DEVERR_BOUNDS, DEVERR_SEL, DEVERR_TIMEOUT, DEVERR_MAP = 1, 2, 4, 8

EXPORTS = ("mfa_abi_version", "mfa_status_string", "mfa_tile_map_bytes", "mfa_tile_map_init",
           "mfa_build_tile_map", "mfa_fwd", "mfa_fwd_noalloc", "mfa_get_device_status",
           "mfa_mask_from_sparse_mode", "mfa_bwd_workspace_bytes", "mfa_bwd", "mfa_decode_workspace_bytes",
           "mfa_decode", "mfa_fwd_bias", "mfa_test_arm_fwd_timeout", "mfa_tree_decode_workspace_bytes",
           "mfa_tree_decode", "mfa_key_weights", "mfa_evict_select", "mfa_cache_compact")
BIAS_NONE, BIAS_ALIBI, BIAS_ALIBI_SQRT, BIAS_ALIBI_LEFT = 0, 1, 2, 3
NOALLOC_SCRATCH_BYTES = 16 << 20
TREE_MAX_NODES = 256


class MfaTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("N", ctypes.c_int64), ("D", ctypes.c_int64),
                ("stride", ctypes.c_int64 * 4)]


class MfaTileMap(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hm", ctypes.c_int32), ("Nq", ctypes.c_int32), ("Nk", ctypes.c_int32),
                ("block_q", ctypes.c_int32), ("block_k", ctypes.c_int32), ("nqt", ctypes.c_int32),
                ("nkt", ctypes.c_int32), ("kind", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("kminmax", ctypes.c_void_p), ("tile_class", ctypes.c_void_p), ("tile_list", ctypes.c_void_p),
                ("tile_count", ctypes.c_void_p), ("order", ctypes.c_void_p), ("err", ctypes.c_void_p)]


class MfaMaskDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("B", ctypes.c_int32), ("Hm", ctypes.c_int32), ("Nq", ctypes.c_int32),
                ("Nk", ctypes.c_int32), ("sel_k", ctypes.c_int32), ("sel_block", ctypes.c_int32),
                ("reserved", ctypes.c_int32),
                ("lts", ctypes.c_void_p), ("lte", ctypes.c_void_p), ("uts", ctypes.c_void_p), ("ute", ctypes.c_void_p),
                ("pre_tokens", ctypes.c_int64), ("next_tokens", ctypes.c_int64),
                ("sel", ctypes.c_void_p), ("map", ctypes.POINTER(MfaTileMap))]


class MfaSparseMode(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("pre_tokens", ctypes.c_int64), ("next_tokens", ctypes.c_int64),
                ("prefix", ctypes.c_void_p), ("seq_q", ctypes.c_void_p), ("seq_kv", ctypes.c_void_p),
                ("n_seq", ctypes.c_int32), ("reserved2", ctypes.c_int32)]


class MfaBias(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("slopes", ctypes.c_void_p)]


class MfaError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} returned {status} ({msg})")
        self.status = status


_lib: Optional[ctypes.CDLL] = None


def load(path: str = _LIB_PATH) -> ctypes.CDLL:
    """Load libmfa.so (built in-tree by mask_aware_block_mfa_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: run `python -m mask_aware_block_mfa_b200.build`")
    lib = ctypes.CDLL(path)
    lib.mfa_abi_version.restype = ctypes.c_int32
    lib.mfa_status_string.restype = ctypes.c_char_p
    lib.mfa_status_string.argtypes = [ctypes.c_int]
    lib.mfa_tile_map_bytes.restype = ctypes.c_size_t
    lib.mfa_tile_map_bytes.argtypes = [ctypes.c_int32] * 6
    lib.mfa_tile_map_init.restype = ctypes.c_int
    lib.mfa_tile_map_init.argtypes = [ctypes.POINTER(MfaTileMap), ctypes.c_void_p, ctypes.c_size_t] + [ctypes.c_int32] * 6
    lib.mfa_build_tile_map.restype = ctypes.c_int
    lib.mfa_build_tile_map.argtypes = [ctypes.POINTER(MfaMaskDesc), ctypes.POINTER(MfaTileMap), ctypes.c_void_p]
    lib.mfa_fwd.restype = ctypes.c_int
    lib.mfa_fwd.argtypes = [ctypes.POINTER(MfaTensor)] * 3 + [ctypes.POINTER(MfaMaskDesc), ctypes.POINTER(MfaTensor),
                                                              ctypes.c_void_p, ctypes.c_void_p]
    lib.mfa_fwd_noalloc.restype = ctypes.c_int
    lib.mfa_fwd_noalloc.argtypes = [ctypes.POINTER(MfaTensor)] * 3 + [ctypes.POINTER(MfaMaskDesc), ctypes.c_int32,
                                                                      ctypes.c_int32, ctypes.POINTER(MfaTensor),
                                                                      ctypes.c_void_p, ctypes.c_void_p,
                                                                      ctypes.c_void_p]
    lib.mfa_get_device_status.restype = ctypes.c_int
    lib.mfa_get_device_status.argtypes = [ctypes.POINTER(MfaTileMap), ctypes.c_void_p,
                                          ctypes.POINTER(ctypes.c_uint32)]
    lib.mfa_mask_from_sparse_mode.restype = ctypes.c_int
    lib.mfa_mask_from_sparse_mode.argtypes = [ctypes.POINTER(MfaSparseMode)] + [ctypes.c_int32] * 3 + \
        [ctypes.c_void_p] * 4 + [ctypes.POINTER(MfaMaskDesc), ctypes.c_void_p]
    lib.mfa_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.mfa_bwd_workspace_bytes.argtypes = [ctypes.c_int32] * 5
    lib.mfa_bwd.restype = ctypes.c_int
    lib.mfa_bwd.argtypes = [ctypes.POINTER(MfaTensor)] * 5 + [ctypes.c_void_p, ctypes.POINTER(MfaMaskDesc)] + \
        [ctypes.POINTER(MfaTensor)] * 3 + [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.mfa_fwd_bias.restype = ctypes.c_int
    lib.mfa_fwd_bias.argtypes = [ctypes.POINTER(MfaTensor)] * 3 + [ctypes.POINTER(MfaMaskDesc),
                                                                   ctypes.POINTER(MfaBias),
                                                                   ctypes.POINTER(MfaTensor), ctypes.c_void_p,
                                                                   ctypes.c_void_p]
    lib.mfa_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.mfa_decode_workspace_bytes.argtypes = [ctypes.c_int32] * 7
    lib.mfa_decode.restype = ctypes.c_int
    lib.mfa_decode.argtypes = [ctypes.POINTER(MfaTensor)] * 3 + [ctypes.c_void_p, ctypes.c_int32,
                                                                 ctypes.POINTER(MfaTensor), ctypes.c_void_p,
                                                                 ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                                                                 ctypes.c_void_p, ctypes.c_void_p]
    T, P, I = ctypes.POINTER(MfaTensor), ctypes.c_void_p, ctypes.c_int32
    lib.mfa_tree_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.mfa_tree_decode_workspace_bytes.argtypes = [I] * 5
    lib.mfa_tree_decode.restype = ctypes.c_int
    lib.mfa_tree_decode.argtypes = [T, T, T, P, P, T, P, P, ctypes.c_size_t, P, P]
    lib.mfa_key_weights.restype = ctypes.c_int
    lib.mfa_key_weights.argtypes = [T, T, P, P, P, P, P, ctypes.c_float, P, P, P]
    lib.mfa_evict_select.restype = ctypes.c_int
    lib.mfa_evict_select.argtypes = [P, P, I, I, I, I, I, P, P, P, P]
    lib.mfa_cache_compact.restype = ctypes.c_int
    lib.mfa_cache_compact.argtypes = [T, T, P, P, P, I, I, P, P, T, T, P, P, P]
    lib.mfa_test_arm_fwd_timeout.restype = ctypes.c_int
    lib.mfa_test_arm_fwd_timeout.argtypes = [ctypes.c_uint32]
    if lib.mfa_abi_version() != 1:
        raise RuntimeError("libmfa.so ABI version mismatch")
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().mfa_status_string(code).decode()


def _check(fn: str, code: int) -> None:
    if code != MFA_OK:
        raise MfaError(fn, code, status_string(code))


def _on_device(name: str, t, device=None, dtype=None, shape=None, contiguous=False) -> None:
    """Host-side checks of a tensor handed to the library as a raw device
    pointer: a CUDA tensor, on `device` when given, with the dtype, shape and
    layout the call reads or writes (the C ABI cannot check these for plain
    pointers, and a host pointer would fault the kernel)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_lse(lse, q) -> None:
    _on_device("lse", lse, q.device, torch.float32, tuple(q.shape[:3]), contiguous=True)


def _dev(q):
    """The device of the call (q's), after checking that q is a CUDA tensor."""
    _on_device("q", q)
    return q.device


def _same_device(q, *holders) -> None:
    """The device arrays of masks and tile maps must live on q's device."""
    for h in holders:
        ts = [getattr(h, "buf", None), getattr(h, "bounds", None)] + list(getattr(h, "_keep", []))
        for t in ts:
            if isinstance(t, torch.Tensor) and t.device != q.device:
                raise ValueError(f"a mask or tile-map array is on {t.device}, q on {q.device}")


def tensor_desc(t: torch.Tensor, device=None) -> MfaTensor:
    _on_device("tensor", t, device)
    if t.dim() != 4:
        raise ValueError("expected a [B, H, N, D] tensor")
    dt = {torch.bfloat16: MFA_BF16, torch.float32: MFA_F32}.get(t.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    d = MfaTensor()
    d.data = t.data_ptr()
    d.dtype = dt
    d.B, d.H, d.N, d.D = (int(x) for x in t.shape)
    for i in range(4):
        d.stride[i] = int(t.stride(i))
    return d


def _stream_ptr(stream, device=None) -> int:
    """The raw handle of `stream`, by default the current stream of `device`.
    A stream of another device is rejected: the library launches on the
    current device, which every wrapper below sets to the tensors' device."""
    if device is not None:
        device = torch.device(device)
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif device is not None and device.type == "cuda" and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the call runs on {device}")
    return int(stream.cuda_stream)


def _on(device):
    """Make `device` current for the duration of one library call (the C ABI
    launches on the current device and looks up per-device state there)."""
    return torch.cuda.device(torch.device(device))


class DeviceMask:
    """A mask description whose arrays live on the device, plus its C struct."""

    def __init__(self, mask: W.MaskDesc, device="cuda"):
        self.mask = mask
        self.kind, self.B, self.Hm, self.Nq, self.Nk = mask.kind, mask.B, mask.Hm, mask.Nq, mask.Nk
        self._keep = []
        d = MfaMaskDesc()
        d.kind, d.B, d.Hm, d.Nq, d.Nk = mask.kind, mask.B, mask.Hm, mask.Nq, mask.Nk
        d.sel_k, d.sel_block = mask.sel_k, mask.sel_block
        for f in ("lts", "lte", "uts", "ute", "sel"):
            a = getattr(mask, f)
            if a is None:
                setattr(d, f, None)
                continue
            t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)
            self._keep.append(t)
            setattr(d, f, t.data_ptr())
        d.pre_tokens, d.next_tokens = int(mask.pre_tokens), int(mask.next_tokens)
        d.map = None
        self.desc = d


class SparseModeMask:
    """An Ascend sparse mode turned into a device mask description by
    mfa_mask_from_sparse_mode (band modes on the host, prefix and varlen modes
    by a kernel into column-wise bounds owned here). Usable wherever a
    DeviceMask is (build_tile_map, fwd, Attention)."""

    def __init__(self, mode: int, B: int, Nq: int, Nk: int, pre_tokens: int = 0, next_tokens: int = 0,
                 prefix=None, seq_q=None, seq_kv=None, device="cuda", stream=None):
        self.B, self.Hm, self.Nq, self.Nk = B, 1, Nq, Nk
        self._keep = []
        sm = MfaSparseMode()
        sm.mode, sm.pre_tokens, sm.next_tokens = mode, int(pre_tokens), int(next_tokens)

        def dev64(a):
            if a is None:
                return None
            t = torch.as_tensor(np.asarray(a, dtype=np.int64)).to(device)
            self._keep.append(t)
            return t.data_ptr()

        sm.prefix, sm.seq_q, sm.seq_kv = dev64(prefix), dev64(seq_q), dev64(seq_kv)
        sm.n_seq = 0 if seq_q is None else len(seq_q)
        self.sm = sm
        self.bounds = torch.empty(4, max(B, 1), 1, max(Nk, 1), dtype=torch.int32, device=device)
        self.desc = MfaMaskDesc()
        self.convert(stream)
        self.kind = self.desc.kind

    def convert(self, stream=None) -> None:
        """(Re)write the description, and for modes 5-8 the bounds, from the
        mode's inputs already on the device (no allocation, graph-capturable)."""
        ptrs = [self.bounds[i].data_ptr() for i in range(4)]  # lts, lte, uts, ute
        dev = self.bounds.device
        with _on(dev):
            _check("mfa_mask_from_sparse_mode",
                   load().mfa_mask_from_sparse_mode(ctypes.byref(self.sm), self.B, self.Nq, self.Nk, *ptrs,
                                                    ctypes.byref(self.desc), _stream_ptr(stream, dev)))


class TileMap:
    """A tile map in one caller-owned device buffer (see mfa_tile_map in mfa.h)."""

    def __init__(self, B, Hm, Nq, Nk, block_q, block_k, device="cuda"):
        lib = load()
        nbytes = lib.mfa_tile_map_bytes(B, Hm, Nq, Nk, block_q, block_k)
        if nbytes == 0:
            raise MfaError("mfa_tile_map_bytes", MFA_ERR_INVALID_ARG, "bad shape or block sizes")
        self.buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        base = self.buf.data_ptr()
        aligned = (base + 255) & ~255
        self.m = MfaTileMap()
        _check("mfa_tile_map_init", lib.mfa_tile_map_init(ctypes.byref(self.m), aligned, nbytes,
                                                          B, Hm, Nq, Nk, block_q, block_k))
        self.offset = aligned - base
        self.nbytes = nbytes

    def arrays(self):
        """Views of the map arrays as torch tensors on the device."""
        m = self.m
        BH, nqt, nkt = m.B * m.Hm, m.nqt, m.nkt

        def view(ptr, dtype, count):
            off = ptr - self.buf.data_ptr()
            el = torch.tensor([], dtype=dtype).element_size()
            return self.buf[off:off + count * el].view(dtype)

        return {
            "kminmax": view(m.kminmax, torch.int32, BH * nkt * 8).view(m.B, m.Hm, nkt, 8),
            "tile_class": view(m.tile_class, torch.uint8, BH * nqt * nkt).view(m.B, m.Hm, nqt, nkt),
            "tile_list": view(m.tile_list, torch.int32, BH * nqt * nkt).view(m.B, m.Hm, nqt, nkt),
            "tile_count": view(m.tile_count, torch.int32, BH * nqt).view(m.B, m.Hm, nqt),
            "order": view(m.order, torch.int32, BH * nqt),
            "err": view(m.err, torch.int32, 1),
        }


def build_tile_map(dmask: DeviceMask, tmap: TileMap, stream=None) -> None:
    dev = tmap.buf.device
    _same_device(tmap.buf, dmask)
    with _on(dev):
        _check("mfa_build_tile_map", load().mfa_build_tile_map(ctypes.byref(dmask.desc), ctypes.byref(tmap.m),
                                                               _stream_ptr(stream, dev)))


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dmask: DeviceMask, tmap: TileMap,
        out: torch.Tensor, lse: torch.Tensor, stream=None) -> None:
    """out, lse <- attention(q, k, v) under dmask, through the tile map (both on the device)."""
    qd, kd, vd, od = (tensor_desc(t, _dev(q)) for t in (q, k, v, out))
    _check_lse(lse, q)
    _same_device(q, tmap, dmask)
    dmask.desc.map = ctypes.pointer(tmap.m)
    with _on(q.device):
        _check("mfa_fwd", load().mfa_fwd(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd),
                                         ctypes.byref(dmask.desc), ctypes.byref(od), lse.data_ptr(),
                                         _stream_ptr(stream, q.device)))


def fwd_bias(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dmask, tmap: TileMap, kind: int,
             slopes: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, stream=None) -> None:
    """Forward pass with an additive ALiBi bias (kind BIAS_*, slopes: float32 device tensor [Hq])."""
    qd, kd, vd, od = (tensor_desc(t, _dev(q)) for t in (q, k, v, out))
    _check_lse(lse, q)
    _on_device("slopes", slopes, q.device, torch.float32, (int(q.shape[1]),), contiguous=True)
    _same_device(q, tmap, dmask)
    dmask.desc.map = ctypes.pointer(tmap.m)
    bias = MfaBias(kind, 0, slopes.data_ptr())
    with _on(q.device):
        _check("mfa_fwd_bias", load().mfa_fwd_bias(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd),
                                                   ctypes.byref(dmask.desc), ctypes.byref(bias), ctypes.byref(od),
                                                   lse.data_ptr(), _stream_ptr(stream, q.device)))


def fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dmask: DeviceMask, block_q: int, block_k: int,
                out: torch.Tensor, lse: torch.Tensor, dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """Forward pass with the tile map in the library's own device array (no allocation by anyone)."""
    qd, kd, vd, od = (tensor_desc(t, _dev(q)) for t in (q, k, v, out))
    _check_lse(lse, q)
    if dev_err is not None:
        _on_device("dev_err", dev_err, q.device)
        if dev_err.numel() * dev_err.element_size() < 4:
            raise ValueError("dev_err must hold at least 4 bytes")
    _same_device(q, dmask)
    err_ptr = None if dev_err is None else dev_err.data_ptr()
    # The library picks its scratch array and launches on the current device.
    with _on(q.device):
        _check("mfa_fwd_noalloc", load().mfa_fwd_noalloc(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd),
                                                         ctypes.byref(dmask.desc), block_q, block_k,
                                                         ctypes.byref(od), lse.data_ptr(), err_ptr,
                                                         _stream_ptr(stream, q.device)))


def bwd_workspace_bytes(B: int, Hq: int, Nq: int, Nk: int, D: int) -> int:
    return int(load().mfa_bwd_workspace_bytes(B, Hq, Nq, Nk, D))


def bwd(q, k, v, out, dout, lse, dmask, tmap: TileMap, dq, dk, dv, workspace: torch.Tensor, stream=None) -> None:
    """dq, dk, dv <- gradients of attention(q, k, v) under dmask for the output
    gradient dout (out, lse from the forward pass; the map built with 128-key
    tiles); workspace is a uint8 device tensor of bwd_workspace_bytes()."""
    ds = [tensor_desc(t, _dev(q)) for t in (q, k, v, out, dout, dq, dk, dv)]
    _check_lse(lse, q)
    _on_device("workspace", workspace, q.device, torch.uint8, contiguous=True)
    _same_device(q, tmap, dmask)
    dmask.desc.map = ctypes.pointer(tmap.m)
    with _on(q.device):
        _check("mfa_bwd", load().mfa_bwd(*(ctypes.byref(d) for d in ds[:5]), lse.data_ptr(),
                                         ctypes.byref(dmask.desc), *(ctypes.byref(d) for d in ds[5:]),
                                         workspace.data_ptr(), workspace.numel(), _stream_ptr(stream, q.device)))


def decode_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, D: int, sel_k: int, n_split: int = 0) -> int:
    return int(load().mfa_decode_workspace_bytes(B, Hq, Hkv, Nq, D, sel_k, n_split))


class Decode:
    """Selected-key attention for a few query rows (mfa_decode): keeps the
    split-K workspace and the device error word between calls."""

    def __init__(self, n_split: int = 0):
        self.n_split = n_split
        self.ws = None
        self.err = None

    def __call__(self, q, k, v, sel, out=None, lse=None, stream=None):
        """sel: int32 device tensor [B, Hkv, Nq, sel_k] of 64-key block indices (-1 = none)."""
        qd, kd, vd = (tensor_desc(t, _dev(q)) for t in (q, k, v))
        B_, Hq, Nq, D = q.shape
        Hkv = int(k.shape[1])
        if sel.dim() != 4:
            raise ValueError("sel must be a [B, Hkv, Nq, sel_k] tensor")
        sel_k = int(sel.shape[-1])
        _on_device("sel", sel, q.device, torch.int32, (B_, Hkv, Nq, sel_k), contiguous=True)
        need = decode_workspace_bytes(B_, Hq, Hkv, Nq, D, sel_k, self.n_split)
        if need == 0:
            raise ValueError("invalid decode sizes")
        if self.ws is None or self.ws.numel() < need or self.ws.device != q.device:
            self.ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        if self.err is None or self.err.device != q.device:
            self.err = torch.zeros(1, dtype=torch.int32, device=q.device)
        out = torch.empty_like(q) if out is None else out
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device) if lse is None else lse
        od = tensor_desc(out, q.device)
        _check_lse(lse, q)
        with _on(q.device):
            _check("mfa_decode", load().mfa_decode(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd),
                                                   sel.data_ptr(), sel_k, ctypes.byref(od), lse.data_ptr(),
                                                   self.n_split, self.ws.data_ptr(), self.ws.numel(),
                                                   self.err.data_ptr(), _stream_ptr(stream, q.device)))
        return out, lse

    def status(self) -> int:
        """Synchronise and return the device error bits (0 = none)."""
        torch.cuda.synchronize()
        return 0 if self.err is None else int(self.err.item())


# The calls below take a few microseconds on the device, so their marshalling is
# kept short: descriptors are packed as bytes and handed over as addresses.
_DESC = struct.Struct("Pii8q")
_DESC_BF16 = MFA_BF16
_cache_lib = None


def _cache_fns():
    """The cache operators' entry points, with descriptors as plain addresses."""
    global _cache_lib
    if _cache_lib is None:
        lib = ctypes.CDLL(load()._name)
        P, I = ctypes.c_void_p, ctypes.c_int32
        for name, args in (("mfa_tree_decode", [P] * 8 + [ctypes.c_size_t, P, P]),
                           ("mfa_key_weights", [P] * 7 + [ctypes.c_float, P, P, P]),
                           ("mfa_evict_select", [P, P] + [I] * 5 + [P] * 4),
                           ("mfa_cache_compact", [P] * 5 + [I, I] + [P] * 7)):
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = ctypes.c_int, args
        _cache_lib = lib
    return _cache_lib


def _cache_desc(name: str, t, device, shape=None) -> bytes:
    """The C descriptor of a bf16 [B, H, N, D] tensor on `device`."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        _on_device(name, t, device)
    if t.dtype is not torch.bfloat16 or t.dim() != 4:
        raise ValueError(f"{name} must be a bfloat16 tensor of four dimensions, got {t.dtype} {tuple(t.shape)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return _DESC.pack(t.data_ptr(), _DESC_BF16, 0, *t.shape, *t.stride())


def _array_ptr(name: str, t, device, dtype, shape) -> int:
    """The address of a contiguous array handed over as a plain pointer."""
    if not isinstance(t, torch.Tensor) or t.device != device or t.dtype is not dtype or t.shape != shape or \
            not t.is_contiguous():
        _on_device(name, t, device, dtype, shape, contiguous=True)
    return t.data_ptr()


class _CacheOp:
    """What the cache operators keep between calls: the device error word, made
    here (outside any capture), so that the first call may already be captured."""

    def __init__(self, device="cuda"):
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"the cache operators run on a CUDA device, got {device}")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        home = torch.cuda.current_stream(device)
        home.synchronize()  # calls may come on any stream
        self._err = self.err.data_ptr()
        self._kept = [(self.err, home.cuda_stream)]  # tensors of the object, and the stream whose memory they are

    def status(self) -> int:
        """Synchronise and return the device error bits since the last clear() (0 = none)."""
        torch.cuda.synchronize(self.device)
        return int(self.err.item())

    def clear(self) -> None:
        """Forget the error bits (on the current stream)."""
        self.err.zero_()

    @staticmethod
    def _on_stream(stream):
        """Memory allocated for a call belongs to the call's stream."""
        return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)

    def _stream(self, stream) -> int:
        """The handle of `stream` (None: the device's current one); the object's tensors are in use there."""
        if stream is None:
            ptr = torch._C._cuda_getCurrentRawStream(self.device.index)
        else:
            ptr = _stream_ptr(stream, self.device)
        for t, home in self._kept:
            if ptr != home:
                t.record_stream(torch.cuda.current_stream(self.device) if stream is None else stream)
        return ptr

    @staticmethod
    def _lend(stream, *tensors):
        """The caller's tensors are in use on a stream given by name: their memory is not
        handed out again before that work is done."""
        for t in tensors:
            if t is not None:
                t.record_stream(stream)

    def _call(self, name: str, fn, *args):
        """Call an entry point with the object's device current."""
        index = self.device.index
        if torch._C._cuda_getDevice() == index:
            code = fn(*args)
        else:
            with torch.cuda.device(index):
                code = fn(*args)
        if code != MFA_OK:
            _check(name, code)


def tree_decode_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, D: int) -> int:
    return int(load().mfa_tree_decode_workspace_bytes(B, Hq, Hkv, T, D))


class TreeDecode(_CacheOp):
    """Attention of T drafted tokens per sequence, a tree or a chain, over a
    cache (mfa_tree_decode): keeps the workspace between calls. Calls of one
    object must not overlap on the GPU (one stream, or ordered streams)."""

    def __init__(self, device="cuda"):
        super().__init__(device)
        self.ws, self._ws, self._ws_bytes = None, None, 0
        self._need = {}

    def __call__(self, q, k, v, lens, parents=None, out=None, lse=None, stream=None):
        """q [B, Hq, T, D], k / v [B, Hkv, N, D]: bf16; lens int32 [B]: keys held before the
        drafted tokens, whose rows are lens[b] + t; parents int32 [B, T] (-1: the sequence's
        end, -2: no node) or None for a chain. Returns out and the natural-log lse."""
        dev = self.device
        qd, kd = _cache_desc("q", q, dev), _cache_desc("k", k, dev)
        vd = _cache_desc("v", v, dev, k.shape)
        B_, Hq, T, D = q.shape
        lens_p = _array_ptr("lens", lens, dev, torch.int32, (B_,))
        par_p = None if parents is None else _array_ptr("parents", parents, dev, torch.int32, (B_, T))
        key = (B_, Hq, k.shape[1], T, D)
        need = self._need.get(key)
        if need is None:
            with _on(dev):
                need = tree_decode_workspace_bytes(*key)
            if need == 0:
                raise ValueError("invalid tree decode sizes")
            self._need[key] = need
        if out is None or lse is None or self._ws_bytes < need:
            with self._on_stream(stream):
                if self._ws_bytes < need:
                    # A smaller one stays: a graph captured with it may be replayed.
                    self.ws = torch.empty(need, dtype=torch.uint8, device=dev)
                    self._ws, self._ws_bytes = self.ws.data_ptr(), need
                    self._kept.append((self.ws, torch.cuda.current_stream(dev).cuda_stream))
                if out is None:
                    out = torch.empty(q.shape, dtype=q.dtype, device=dev)
                if lse is None:
                    lse = torch.empty(B_, Hq, T, dtype=torch.float32, device=dev)
        od = _cache_desc("out", out, dev, q.shape)
        lse_p = _array_ptr("lse", lse, dev, torch.float32, (B_, Hq, T))
        if stream is not None:
            self._lend(stream, q, k, v, lens, parents, out, lse)
        self._call("mfa_tree_decode", _cache_fns().mfa_tree_decode, qd, kd, vd, lens_p, par_p, od, lse_p, self._ws,
                   self._ws_bytes, self._err, self._stream(stream))
        return out, lse


class KeyWeights(_CacheOp):
    """The attention weight every cached key got from a call's rows (mfa_key_weights)."""

    def __call__(self, q, k, lse, lens, parents=None, row_scale=None, weights_in=None, decay=1.0, weights_out=None,
                 stream=None):
        """weights_out[b, g, j] = decay * weights_in[b, g, j] + the rows' softmax weights of key j,
        summed over the group's heads and, times row_scale float32 [B, T], over the rows.
        Weights are float32 [B, Hkv, N]; weights_in None is zeros, and may be weights_out
        (None: new, zeros past the keys held). A drafted key goes on from what weights_in holds at
        its place: zeros, for a new key. q, k, lens, parents, lse: TreeDecode's."""
        dev = self.device
        qd, kd = _cache_desc("q", q, dev), _cache_desc("k", k, dev)
        B_, Hq, T, _ = q.shape
        shape = k.shape[:3]
        lens_p = _array_ptr("lens", lens, dev, torch.int32, (B_,))
        par_p = None if parents is None else _array_ptr("parents", parents, dev, torch.int32, (B_, T))
        lse_p = _array_ptr("lse", lse, dev, torch.float32, (B_, Hq, T))
        row_p = None if row_scale is None else _array_ptr("row_scale", row_scale, dev, torch.float32, (B_, T))
        in_p = None if weights_in is None else _array_ptr("weights_in", weights_in, dev, torch.float32, shape)
        if weights_out is None:
            with self._on_stream(stream):
                weights_out = torch.zeros(shape, dtype=torch.float32, device=dev)
        out_p = _array_ptr("weights_out", weights_out, dev, torch.float32, shape)
        if stream is not None:
            self._lend(stream, q, k, lse, lens, parents, row_scale, weights_in, weights_out)
        self._call("mfa_key_weights", _cache_fns().mfa_key_weights, qd, kd, lse_p, lens_p, par_p, row_p, in_p, float(decay),
                   out_p, self._err, self._stream(stream))
        return weights_out


class CacheCompact(_CacheOp):
    """Moves cache rows together (mfa_cache_compact)."""

    def __call__(self, k, v, idx, count, weights=None, start=None, zero_end=None, k_out=None, v_out=None,
                 weights_out=None, stream=None):
        """Row start[b] + t of k, v and weights takes row start[b] + idx[b, g, t], t < count[b]: in
        place, or in k_out, v_out (and weights_out). idx int32 [B, Hkv or 1, n]; count, start and
        zero_end int32 [B]. With start = lens and the accepted nodes, ascending, a branch of a
        tree is committed; the caller then adds count to lens."""
        kd, vd, w_p, zero_p, kod, vod, wo_p, B_, H, _ = self._tensors(k, v, weights, zero_end, k_out, v_out, weights_out)
        dev = self.device
        if not isinstance(idx, torch.Tensor) or idx.dim() != 3 or idx.shape[1] not in (1, H):
            raise ValueError("idx must be an int32 [B, Hkv or 1, n] tensor")
        idx_p = _array_ptr("idx", idx, dev, torch.int32, (B_, idx.shape[1], idx.shape[2]))
        count_p = _array_ptr("count", count, dev, torch.int32, (B_,))
        start_p = None if start is None else _array_ptr("start", start, dev, torch.int32, (B_,))
        if stream is not None:
            self._lend(stream, k, v, weights, zero_end, k_out, v_out, weights_out, idx, count, start)
        self._call("mfa_cache_compact", _cache_fns().mfa_cache_compact, kd, vd, w_p, start_p, idx_p, idx.shape[1],
                   idx.shape[2], count_p, zero_p, kod, vod, wo_p, self._err, self._stream(stream))

    def _tensors(self, k, v, weights, zero_end, k_out, v_out, weights_out):
        """Descriptors and addresses of what is moved, checked, and k's sizes B, H, N."""
        dev = self.device
        if (k_out is None) != (v_out is None):
            raise ValueError("k_out and v_out are given together")
        if k_out is not None and (weights is None) != (weights_out is None):
            raise ValueError("weights and weights_out are given together")
        kd = _cache_desc("k", k, dev)
        vd = _cache_desc("v", v, dev, k.shape)
        B_, H, N, _ = k.shape
        if k_out is None:
            if weights_out is not None:
                raise ValueError("weights_out without k_out and v_out")
            kod, vod, weights_out, N_out = kd, vd, weights, N
        else:
            kod = _cache_desc("k_out", k_out, dev)
            vod = _cache_desc("v_out", v_out, dev, k_out.shape)
            N_out = k_out.shape[2]
        w_p = wo_p = None
        if weights is not None:
            w_p = _array_ptr("weights", weights, dev, torch.float32, (B_, H, N))
            wo_p = w_p if weights_out is weights else _array_ptr("weights_out", weights_out, dev, torch.float32, (B_, H, N_out))
        zero_p = None if zero_end is None else _array_ptr("zero_end", zero_end, dev, torch.int32, (B_,))
        return kd, vd, w_p, zero_p, kod, vod, wo_p, B_, H, N


class Evictor(_CacheOp):
    """Evicts a cache's keys by their accumulated attention weight: of every
    (batch, head) the last `recent` keys stay and, up to `budget` in all, those
    of the largest weight (mfa_evict_select, then mfa_cache_compact)."""

    def __init__(self, budget: int, recent: int, device="cuda"):
        if budget < 1 or not 0 <= recent <= budget:
            raise ValueError(f"budget must be at least 1 and recent in [0, budget], got {budget} and {recent}")
        super().__init__(device)
        self.budget, self.recent = int(budget), int(recent)
        self.compact = CacheCompact(device)
        self.compact.err, self.compact._err, self.compact._kept = self.err, self._err, self._kept

    def _lists(self, lens, H, stream, keep=None, new_lens=None):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._lists(lens, H, None, keep, new_lens)
        if keep is None:
            keep = lens.new_empty((lens.shape[0], H, self.budget))
        if new_lens is None:
            new_lens = torch.empty_like(lens)
        return keep, new_lens

    def select(self, weights, lens, keep=None, new_lens=None, stream=None):
        """keep int32 [B, Hkv, budget] (ascending rows, then -1) and new_lens int32 [B]."""
        dev = self.device
        if not isinstance(weights, torch.Tensor) or weights.dim() != 3:
            raise ValueError("weights must be a float32 [B, Hkv, N] tensor")
        B_, H, N = weights.shape
        w_p = _array_ptr("weights", weights, dev, torch.float32, (B_, H, N))
        lens_p = _array_ptr("lens", lens, dev, torch.int32, (B_,))
        if keep is None or new_lens is None:
            keep, new_lens = self._lists(lens, H, stream, keep, new_lens)
        keep_p = _array_ptr("keep", keep, dev, torch.int32, (B_, H, self.budget))
        new_p = _array_ptr("new_lens", new_lens, dev, torch.int32, (B_,))
        if stream is not None:
            self._lend(stream, weights, lens, keep, new_lens)
        self._call("mfa_evict_select", _cache_fns().mfa_evict_select, w_p, lens_p, B_, H, N, self.budget, self.recent,
                   keep_p, new_p, self._err, self._stream(stream))
        return keep, new_lens

    def __call__(self, k, v, weights, lens, k_out=None, v_out=None, weights_out=None, zero_end=None, stream=None):
        """Select, then move the kept rows of k, v and weights together, in place or into
        k_out, v_out and weights_out. Returns keep and new_lens; lens is left to the caller. In place,
        zero_end=lens clears the sums that stay behind: where weights go on adding up (KeyWeights with
        weights_in), the next keys in those places would begin with them."""
        if weights is None:
            raise ValueError("weights must be a float32 [B, Hkv, N] tensor")
        kd, vd, w_p, zero_p, kod, vod, wo_p, B_, H, N = self.compact._tensors(k, v, weights, zero_end, k_out, v_out, weights_out)
        lens_p = _array_ptr("lens", lens, self.device, torch.int32, (B_,))
        keep, new_lens = self._lists(lens, H, stream)
        if stream is not None:
            self._lend(stream, k, v, weights, lens, k_out, v_out, weights_out, zero_end)
        keep_p, new_p, s, fns = keep.data_ptr(), new_lens.data_ptr(), self._stream(stream), _cache_fns()
        self._call("mfa_evict_select", fns.mfa_evict_select, w_p, lens_p, B_, H, N, self.budget, self.recent, keep_p,
                   new_p, self._err, s)
        self._call("mfa_cache_compact", fns.mfa_cache_compact, kd, vd, w_p, None, keep_p, H, self.budget, new_p, zero_p,
                   kod, vod, wo_p, self._err, s)
        return keep, new_lens


def arm_fwd_timeout_test(wait_us: int) -> None:
    """Test hook: the next bf16 forward launch withholds one K tile and uses a
    wait limit of wait_us microseconds, so one bounded wait runs out (see
    mfa_test_arm_fwd_timeout in mfa.h)."""
    _check("mfa_test_arm_fwd_timeout", load().mfa_test_arm_fwd_timeout(int(wait_us)))


def device_status(tmap: TileMap, stream=None) -> int:
    """Synchronise and return the map's device error bits (0 = none)."""
    bits = ctypes.c_uint32(0)
    dev = tmap.buf.device
    with _on(dev):
        code = load().mfa_get_device_status(ctypes.byref(tmap.m), _stream_ptr(stream, dev), ctypes.byref(bits))
    if code not in (MFA_OK, MFA_ERR_DEVICE):
        _check("mfa_get_device_status", code)
    return int(bits.value)


class Attention:
    """Convenience wrapper: upload a mask, build its map once, run forward passes."""

    def __init__(self, mask, block_q: int = 64, block_k: int = 128, device="cuda"):
        # a workloads.MaskDesc (uploaded here) or a mask already on the device
        self.dmask = DeviceMask(mask, device) if isinstance(mask, W.MaskDesc) else mask
        self.tmap = TileMap(mask.B, mask.Hm, mask.Nq, mask.Nk, block_q, block_k, device)
        self.device = device

    def build(self, stream=None):
        build_tile_map(self.dmask, self.tmap, stream)

    def __call__(self, q, k, v, out=None, lse=None, stream=None, bias=None):
        """bias: None or (kind, slopes) with kind one of BIAS_* and slopes a float32 device tensor [Hq]."""
        if out is None:
            out = torch.empty_like(q)
        if lse is None:
            lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        if bias is None:
            fwd(q, k, v, self.dmask, self.tmap, out, lse, stream)
        else:
            fwd_bias(q, k, v, self.dmask, self.tmap, bias[0], bias[1], out, lse, stream)
        return out, lse

    def backward(self, q, k, v, out, lse, dout, dq=None, dk=None, dv=None, stream=None):
        """Gradients for the output gradient dout (the map must use 128-key tiles)."""
        B_, Hq, Nq, D = q.shape
        need = bwd_workspace_bytes(B_, Hq, Nq, int(k.shape[2]), D)
        if need == 0:
            raise ValueError("invalid shapes for the backward pass")
        ws = getattr(self, "_bwd_ws", None)
        if ws is None or ws.numel() < need or ws.device != q.device:
            ws = self._bwd_ws = torch.empty(need, dtype=torch.uint8, device=q.device)
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        bwd(q, k, v, out, dout, lse, self.dmask, self.tmap, dq, dk, dv, ws, stream)
        return dq, dk, dv
