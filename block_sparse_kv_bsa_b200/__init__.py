"""Python binding of libbsa.so: block-sparse KV attention on a B200 (sm_100a).

Thin ctypes marshalling over the C ABI declared in ``include/bsa.h``: torch
tensors supply device pointers, the current CUDA stream supplies the stream,
and every computation runs in the library's CUDA kernels.  There is no CPU
or PyTorch fallback: importing this package fails when ``libbsa.so`` is
missing, and every call raises :class:`BsaError` when the library reports a
non-OK status.

The functions carry the C names:

* :func:`bsa_gilbert_perm` - host Gilbert order of a T x H x W chunk
* :func:`bsa_kv_append` - scatter a chunk's K/V into the block cache
* :func:`bsa_tokens_to_blocks` / :func:`bsa_blocks_to_tokens` - reorder Q / O
* :func:`bsa_tokens_to_blocks_mean` - reorder Q and pool its blocks in one pass
* :func:`bsa_route` - pooled-score top-K route per query block
* :func:`bsa_route_qmean` - the same route from precomputed query means
* :func:`bsa_attn` - indexed block-sparse attention (O and LSE)
* :func:`bsa_attn_tokens` - the same with O and LSE in raster token order
* :class:`Rope`, :func:`bsa_rope` - rotary positions on tokens, and their gradient
* :func:`bsa_tokens_to_blocks_rope` / :func:`bsa_kv_append_rope` - the same on
  the way into block order
* :class:`KVCache8`, :func:`bsa_kv8_append` - a cache in e4m3 with one scale per
  block and head
* :func:`bsa_kv8_attn` / :func:`bsa_kv8_attn_decode` - attention over it, by query
  blocks or by a few query tokens
* :func:`bsa_check_device_error` - read and clear the device error word

Method: "Velox: Spatial Memory Makes World Models Efficient" (Key
Contributions 3; Methodology Steps 4-6).
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional, Tuple

import numpy as np
import torch

BLK = 128
_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsa.so")

STATUS_NAMES = {
    0: "BSA_OK", 1: "BSA_ERR_INVALID_ARG", 2: "BSA_ERR_SHAPE", 3: "BSA_ERR_CAPACITY",
    4: "BSA_ERR_UNSUPPORTED", 5: "BSA_ERR_CUDA", 6: "BSA_ERR_DEVICE_FAULT", 7: "BSA_ERR_TIMEOUT",
}
DEV_CODES = {0: "BSA_DEV_OK", 1: "BSA_DEV_BAD_INDEX", 2: "BSA_DEV_BAD_COUNT",
             3: "BSA_DEV_BAD_VALID", 4: "BSA_DEV_BAD_PERM", 5: "BSA_DEV_WAIT_TIMEOUT",
             6: "BSA_DEV_BAD_SCALE"}

# Every symbol include/bsa.h declares (checked by the tests).
EXPORTS = ("bsa_abi_version", "bsa_status_string", "bsa_gilbert_perm", "bsa_kv_append",
           "bsa_kv_pool_means",
           "bsa_tokens_to_blocks", "bsa_tokens_to_blocks_mean", "bsa_blocks_to_tokens",
           "bsa_route_workspace_size", "bsa_route", "bsa_route_qmean", "bsa_route_velox",
           "bsa_route_velox_qmean",
           "bsa_route_noalloc", "bsa_attn", "bsa_attn_tokens",
           "bsa_geometry_prior",
           "bsa_rope_frequencies", "bsa_rope_phases", "bsa_rope", "bsa_tokens_to_blocks_rope",
           "bsa_kv_append_rope", "bsa_kv8_append", "bsa_kv8_attn",
           "bsa_kv8_attn_decode_workspace_size", "bsa_kv8_attn_decode",
           "bsa_check_device_error",
           "bsa_selftest_bounded_wait")


class BsaError(RuntimeError):
    """A libbsa call returned a non-OK status."""

    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        name = STATUS_NAMES.get(status, f"status {status}")
        super().__init__(f"{fn}: {name}{(' - ' + detail) if detail else ''}")


if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libbsa.so not found at {LIB_PATH}; build it with "
        "`python -m block_sparse_kv_bsa_b200._build` (there is no fallback path)")

_lib = ctypes.CDLL(LIB_PATH)


class CCache(ctypes.Structure):
    """ctypes mirror of ``bsa_kv_cache``."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("block_valid", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("Hh", ctypes.c_int32), ("D", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("n_blocks", ctypes.c_int32),
                ("kmean", ctypes.c_void_p)]


class CVeloxRoute(ctypes.Structure):
    """ctypes mirror of ``bsa_velox_route``."""
    _fields_ = [("coverage", ctypes.c_void_p), ("eta_cov", ctypes.c_float),
                ("tau", ctypes.c_float), ("k_cov", ctypes.c_int32), ("k_unc", ctypes.c_int32),
                ("mass", ctypes.c_float), ("prev_first", ctypes.c_int32),
                ("n_prev", ctypes.c_int32), ("window_half", ctypes.c_int32),
                ("ref_first", ctypes.c_int32), ("n_ref", ctypes.c_int32)]


class CRope(ctypes.Structure):
    """ctypes mirror of ``bsa_rope_desc``."""
    _fields_ = [("phase", ctypes.c_void_p), ("n_pairs", ctypes.c_int32 * 3),
                ("n_axes", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("amplitude", ctypes.c_float),
                ("pos", ctypes.c_void_p), ("origin", ctypes.c_int32 * 3)]


class CCache8(ctypes.Structure):
    """ctypes mirror of ``bsa_kv_cache8``."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("block_valid", ctypes.c_void_p),
                ("B", ctypes.c_int32), ("Hh", ctypes.c_int32), ("D", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("n_blocks", ctypes.c_int32),
                ("kmean", ctypes.c_void_p)]


_i, _p, _f, _sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
_sig = {
    "bsa_abi_version": (ctypes.c_int, []),
    "bsa_status_string": (ctypes.c_char_p, [_i]),
    "bsa_gilbert_perm": (_i, [_i, _i, _i, _p]),
    "bsa_kv_append": (_i, [ctypes.POINTER(CCache), _p, _p, _i, _i, _i, _p, _p, _p]),
    "bsa_kv_pool_means": (_i, [ctypes.POINTER(CCache), _i, _i, _p, _p]),
    "bsa_tokens_to_blocks": (_i, [_p, _p, _i, _i, _i, _i, _i, _i, _p, _p, _p]),
    "bsa_tokens_to_blocks_mean": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _i, _p, _p, _p]),
    "bsa_blocks_to_tokens": (_i, [_p, _p, _i, _i, _i, _i, _i, _i, _p, _p, _p]),
    "bsa_route_workspace_size": (_i, [_i, _i, _i, _i, _i, ctypes.POINTER(_sz)]),
    "bsa_route": (_i, [_p, ctypes.POINTER(CCache), _p, _i, _i, _i, _p, _f, _f, _f, _i,
                       _p, _p, _i, _p, _sz, _p, _p]),
    "bsa_route_qmean": (_i, [_p, ctypes.POINTER(CCache), _i, _i, _i, _p, _f, _f, _f, _i,
                             _p, _p, _i, _p, _sz, _p, _p]),
    "bsa_geometry_prior": (_i, [_p, _i, _f, _f, _f, _f, _p, _p, _i, _p, _p, _i, _i, _i, _p, _p,
                                _p, _i, _p, _p, _p, _p]),
    "bsa_route_velox": (_i, [_p, ctypes.POINTER(CCache), _p, _i, _i, _i, _p, _f, _f, _f,
                             ctypes.POINTER(CVeloxRoute), _p, _p, _i, _p, _sz, _p, _p]),
    "bsa_route_velox_qmean": (_i, [_p, ctypes.POINTER(CCache), _i, _i, _i, _p, _f, _f, _f,
                                   ctypes.POINTER(CVeloxRoute), _p, _p, _i, _p, _sz, _p, _p]),
    "bsa_route_noalloc": (_i, [_p, ctypes.POINTER(CCache), _p, _i, _i, _i, _p, _f, _f, _f, _i,
                               _p, _p, _i, _p, _p]),
    "bsa_attn": (_i, [_p, ctypes.POINTER(CCache), _p, _p, _p, _i, _i, _f, _p, _p, _p, _p]),
    "bsa_attn_tokens": (_i, [_p, ctypes.POINTER(CCache), _p, _p, _p, _i, _f, _i, _i, _i, _p, _p,
                             _p, _p, _p]),
    "bsa_rope_frequencies": (_i, [_i, ctypes.c_double, _i, ctypes.c_double, ctypes.c_double,
                                  ctypes.c_double, ctypes.c_double, _p, _p]),
    "bsa_rope_phases": (_i, [_p, _i, _p]),
    "bsa_rope": (_i, [_p, _p, _i, _i, _i, _i, _i, _i, ctypes.POINTER(CRope), _p]),
    "bsa_tokens_to_blocks_rope": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _i, _p,
                                       ctypes.POINTER(CRope), _p, _p]),
    "bsa_kv_append_rope": (_i, [ctypes.POINTER(CCache), _p, _p, _i, _i, _i, _p,
                                ctypes.POINTER(CRope), _p, _p]),
    "bsa_kv8_append": (_i, [ctypes.POINTER(CCache8), _p, _p, _i, _i, _i, _p,
                            ctypes.POINTER(CRope), _p, _p]),
    "bsa_kv8_attn": (_i, [_p, ctypes.POINTER(CCache8), _i, _p, _p, _p, _i, _i, _f, _p, _p, _p,
                          _p]),
    "bsa_kv8_attn_decode_workspace_size": (_i, [_i, _i, _i, _i, _i, _i, ctypes.POINTER(_sz)]),
    "bsa_kv8_attn_decode": (_i, [_p, ctypes.POINTER(CCache8), _i, _i, _p, _p, _i, _f, _p, _p, _p,
                                 _sz, _p, _p]),
    "bsa_check_device_error": (_i, [_p, _p, ctypes.POINTER(ctypes.c_int32)]),
    "bsa_selftest_bounded_wait": (_i, [_p, ctypes.c_longlong, _p]),
}
for _name, (_res, _args) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def lib() -> ctypes.CDLL:
    """The loaded library handle."""
    return _lib


def _check(fn: str, status: int):
    if status != 0:
        raise BsaError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(device) -> torch.device:
    """A device with an explicit index (``cuda`` -> ``cuda:<current>``)."""
    if isinstance(device, torch.device) and device.index is not None:
        return device
    d = torch.device(device)
    if d.type == "cuda" and d.index is None:
        d = torch.device("cuda", torch.cuda.current_device())
    return d


# The current stream's handle without building a Stream object (2.4 us less on
# a call), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> ctypes.c_void_p:
    if _raw_stream is not None and isinstance(device, torch.device) and device.index is not None:
        return ctypes.c_void_p(_raw_stream(device.index))
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t: torch.Tensor, name: str, dtype, device=None, shape=None):
    # The common case in few steps; what is wrong is found out below.
    if (type(t) is torch.Tensor and t.dtype is dtype and t.is_cuda and t.is_contiguous()
            and (device is None or t.device == device) and (shape is None or t.shape == shape)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != _dev(device):
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


_err_words = {}
_lock = threading.Lock()


def error_word(device) -> torch.Tensor:
    """The per-device int32 word kernels report BSA_DEV_* codes into."""
    device = _dev(device)
    with _lock:
        w = _err_words.get(device)
        if w is None:
            w = torch.zeros(1, dtype=torch.int32, device=device)
            _err_words[device] = w
    return w


def abi_version() -> int:
    return int(_lib.bsa_abi_version())


def status_string(status: int) -> str:
    return _lib.bsa_status_string(int(status)).decode()


def n_blocks_for(T: int, H: int, W: int) -> int:
    return -(-T * H * W // BLK)


# ---------------------------------------------------------------------------
# Gilbert order
# ---------------------------------------------------------------------------

_perm_cache = {}


def bsa_gilbert_perm(T: int, H: int, W: int) -> np.ndarray:
    """perm[i] = curve position of raster token i (host int32 [T*H*W])."""
    n = T * H * W
    out = np.empty(max(n, 1), dtype=np.int32)
    _check("bsa_gilbert_perm", _lib.bsa_gilbert_perm(int(T), int(H), int(W),
                                                      out.ctypes.data_as(ctypes.c_void_p)))
    return out[:n]


def gilbert_perm_device(T: int, H: int, W: int, device) -> torch.Tensor:
    """The Gilbert table of a chunk shape on ``device``, computed once and cached."""
    key = (int(T), int(H), int(W), _dev(device))
    with _lock:
        t = _perm_cache.get(key)
    if t is None:
        t = torch.from_numpy(bsa_gilbert_perm(T, H, W)).to(device)
        with _lock:
            _perm_cache[key] = t
    return t


# ---------------------------------------------------------------------------
# KV cache
# ---------------------------------------------------------------------------

class KVCache:
    """A caller-owned block KV cache: K, V bf16 [B, Hh, max_blocks, 128, D] and
    the valid-row count of every block."""

    def __init__(self, B: int, Hh: int, D: int, max_blocks: int, device="cuda",
                 pooled_keys: bool = False):
        self.B, self.Hh, self.D, self.max_blocks = int(B), int(Hh), int(D), int(max_blocks)
        self.device = _dev(device)
        shape = (self.B, self.Hh, self.max_blocks, BLK, self.D)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
        self.v = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
        self.block_valid = torch.zeros(self.max_blocks, dtype=torch.int32, device=self.device)
        # Optional pooled-key cache: block means of K, written at append time
        # and read by bsa_route instead of the history keys.
        self.kmean = (torch.zeros((self.B, self.Hh, self.max_blocks, self.D), dtype=torch.float32,
                                  device=self.device) if pooled_keys else None)
        self.n_blocks = 0

    def c_struct(self) -> CCache:
        return CCache(self.k.data_ptr(), self.v.data_ptr(), self.block_valid.data_ptr(),
                      self.B, self.Hh, self.D, self.max_blocks, self.n_blocks,
                      None if self.kmean is None else self.kmean.data_ptr())


def bsa_kv_append(cache: KVCache, k_tok: torch.Tensor, v_tok: torch.Tensor,
                  T: int, H: int, W: int, d_err: Optional[torch.Tensor] = None,
                  table: bool = True) -> int:
    """Append one chunk (bf16 [B, T*H*W, Hh, D] K and V); returns its first block.
    table=False passes no permutation table: the kernels locate the Gilbert
    slots themselves (the same order)."""
    shape = (cache.B, T * H * W, cache.Hh, cache.D)
    _need(k_tok, "k_tok", torch.bfloat16, cache.device, shape)
    _need(v_tok, "v_tok", torch.bfloat16, cache.device, shape)
    perm = gilbert_perm_device(T, H, W, cache.device) if table else None
    err = error_word(cache.device) if d_err is None else d_err
    cs = cache.c_struct()
    first = cache.n_blocks
    _check("bsa_kv_append", _lib.bsa_kv_append(ctypes.byref(cs), _ptr(k_tok), _ptr(v_tok),
                                                int(T), int(H), int(W), _ptr(perm), _ptr(err),
                                                _stream(cache.device)))
    cache.n_blocks = int(cs.n_blocks)
    return first


def bsa_kv_pool_means(cache: KVCache, first: int = 0, count: Optional[int] = None):
    """(Re)compute the pooled-key cache for blocks [first, first + count)."""
    if cache.kmean is None:
        raise ValueError("the cache was created without pooled_keys")
    if count is None:
        count = cache.n_blocks - first
    cs = cache.c_struct()
    _check("bsa_kv_pool_means", _lib.bsa_kv_pool_means(
        ctypes.byref(cs), int(first), int(count), _ptr(error_word(cache.device)),
        _stream(cache.device)))


def bsa_tokens_to_blocks(x_tok: torch.Tensor, T: int, H: int, W: int,
                         out: Optional[torch.Tensor] = None, table: bool = True) -> torch.Tensor:
    """[B, T*H*W, Hh, D] raster tokens -> [B, Hh, nb*128, D] Gilbert blocks (zero pads)."""
    if x_tok.dim() != 4:
        raise ValueError("x_tok must be [B, T*H*W, Hh, D]")
    B, N, Hh, D = x_tok.shape
    _need(x_tok, "x_tok", torch.bfloat16)
    nb = n_blocks_for(T, H, W)
    if out is None:
        out = torch.empty((B, Hh, nb * BLK, D), dtype=torch.bfloat16, device=x_tok.device)
    _need(out, "out", torch.bfloat16, x_tok.device, (B, Hh, nb * BLK, D))
    perm = gilbert_perm_device(T, H, W, x_tok.device) if table else None
    _check("bsa_tokens_to_blocks", _lib.bsa_tokens_to_blocks(
        _ptr(x_tok), _ptr(out), B, Hh, D, int(T), int(H), int(W), _ptr(perm),
        _ptr(error_word(x_tok.device)), _stream(x_tok.device)))
    return out


def bsa_tokens_to_blocks_mean(x_tok: torch.Tensor, T: int, H: int, W: int,
                              out: Optional[torch.Tensor] = None,
                              mean: Optional[torch.Tensor] = None, table: bool = True
                              ) -> Tuple[torch.Tensor, torch.Tensor]:
    """bsa_tokens_to_blocks plus the fp32 mean of every block's valid rows:
    returns (blocks [B, Hh, nb*128, D], means [B, Hh, nb, D])."""
    if x_tok.dim() != 4:
        raise ValueError("x_tok must be [B, T*H*W, Hh, D]")
    B, N, Hh, D = x_tok.shape
    _need(x_tok, "x_tok", torch.bfloat16)
    nb = n_blocks_for(T, H, W)
    if out is None:
        out = torch.empty((B, Hh, nb * BLK, D), dtype=torch.bfloat16, device=x_tok.device)
    if mean is None:
        mean = torch.empty((B, Hh, nb, D), dtype=torch.float32, device=x_tok.device)
    _need(out, "out", torch.bfloat16, x_tok.device, (B, Hh, nb * BLK, D))
    _need(mean, "mean", torch.float32, x_tok.device, (B, Hh, nb, D))
    perm = gilbert_perm_device(T, H, W, x_tok.device) if table else None
    _check("bsa_tokens_to_blocks_mean", _lib.bsa_tokens_to_blocks_mean(
        _ptr(x_tok), _ptr(out), _ptr(mean), B, Hh, D, int(T), int(H), int(W), _ptr(perm),
        _ptr(error_word(x_tok.device)), _stream(x_tok.device)))
    return out, mean


def bsa_blocks_to_tokens(x_blk: torch.Tensor, T: int, H: int, W: int,
                         out: Optional[torch.Tensor] = None, table: bool = True) -> torch.Tensor:
    """[B, Hh, nb*128, D] Gilbert blocks -> [B, T*H*W, Hh, D] raster tokens."""
    if x_blk.dim() != 4:
        raise ValueError("x_blk must be [B, Hh, nb*128, D]")
    B, Hh, R, D = x_blk.shape
    _need(x_blk, "x_blk", torch.bfloat16)
    if R != n_blocks_for(T, H, W) * BLK:
        raise ValueError("x_blk rows do not match the chunk shape")
    if out is None:
        out = torch.empty((B, T * H * W, Hh, D), dtype=torch.bfloat16, device=x_blk.device)
    _need(out, "out", torch.bfloat16, x_blk.device, (B, T * H * W, Hh, D))
    perm = gilbert_perm_device(T, H, W, x_blk.device) if table else None
    _check("bsa_blocks_to_tokens", _lib.bsa_blocks_to_tokens(
        _ptr(x_blk), _ptr(out), B, Hh, D, int(T), int(H), int(W), _ptr(perm),
        _ptr(error_word(x_blk.device)), _stream(x_blk.device)))
    return out


# ---------------------------------------------------------------------------
# Routing and attention
# ---------------------------------------------------------------------------

def bsa_route_workspace_size(B: int, Hh: int, D: int, n_q_blocks: int, n_hist: int) -> int:
    n = ctypes.c_size_t(0)
    _check("bsa_route_workspace_size", _lib.bsa_route_workspace_size(
        int(B), int(Hh), int(D), int(n_q_blocks), int(n_hist), ctypes.byref(n)))
    return int(n.value)


def route_max_sel(top_k: int, n_hist: int, n_own: int) -> int:
    return min(int(top_k), int(n_hist)) + int(n_own)


def bsa_route(q_blk: torch.Tensor, cache: KVCache, n_hist: int, own_first: int, n_own: int,
              top_k: int, g: Optional[torch.Tensor] = None, lam: float = 2.0,
              g_ref: float = 0.2, sm_scale: Optional[float] = None,
              q_valid: Optional[torch.Tensor] = None, max_sel: Optional[int] = None,
              idx: Optional[torch.Tensor] = None, cnt: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Route every (b, h, query block); returns (idx [B,Hh,n_own,max_sel], cnt [B,Hh,n_own])."""
    dev = cache.device
    _need(q_blk, "q_blk", torch.bfloat16, dev, (cache.B, cache.Hh, n_own * BLK, cache.D))
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(cache.D)
    if max_sel is None:
        max_sel = route_max_sel(top_k, n_hist, n_own)
    if idx is None:
        idx = torch.empty((cache.B, cache.Hh, n_own, max_sel), dtype=torch.int32, device=dev)
    if cnt is None:
        cnt = torch.empty((cache.B, cache.Hh, n_own), dtype=torch.int32, device=dev)
    _need(idx, "idx", torch.int32, dev, (cache.B, cache.Hh, n_own, max_sel))
    _need(cnt, "cnt", torch.int32, dev, (cache.B, cache.Hh, n_own))
    if g is not None:
        _need(g, "g", torch.float32, dev, (cache.B, n_own, n_hist))
    if q_valid is not None:
        _need(q_valid, "q_valid", torch.int32, dev, (n_own,))
    ws_bytes = bsa_route_workspace_size(cache.B, cache.Hh, cache.D, n_own, n_hist)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    cs = cache.c_struct()
    _check("bsa_route", _lib.bsa_route(
        _ptr(q_blk), ctypes.byref(cs), _ptr(q_valid), int(n_hist), int(own_first), int(n_own),
        _ptr(g), float(lam), float(g_ref), float(sm_scale), int(top_k), _ptr(idx), _ptr(cnt),
        int(max_sel), _ptr(workspace), workspace.numel(), _ptr(error_word(dev)), _stream(dev)))
    return idx, cnt


def bsa_route_qmean(q_mean: torch.Tensor, cache: KVCache, n_hist: int, own_first: int,
                    n_own: int, top_k: int, g: Optional[torch.Tensor] = None, lam: float = 2.0,
                    g_ref: float = 0.2, sm_scale: Optional[float] = None,
                    max_sel: Optional[int] = None, idx: Optional[torch.Tensor] = None,
                    cnt: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None
                    ) -> Tuple[torch.Tensor, torch.Tensor]:
    """bsa_route from the query-block means [B, Hh, n_own, D] (fp32), e.g.
    those of bsa_tokens_to_blocks_mean; returns (idx, cnt)."""
    dev = cache.device
    _need(q_mean, "q_mean", torch.float32, dev, (cache.B, cache.Hh, n_own, cache.D))
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(cache.D)
    if max_sel is None:
        max_sel = route_max_sel(top_k, n_hist, n_own)
    if idx is None:
        idx = torch.empty((cache.B, cache.Hh, n_own, max_sel), dtype=torch.int32, device=dev)
    if cnt is None:
        cnt = torch.empty((cache.B, cache.Hh, n_own), dtype=torch.int32, device=dev)
    _need(idx, "idx", torch.int32, dev, (cache.B, cache.Hh, n_own, max_sel))
    _need(cnt, "cnt", torch.int32, dev, (cache.B, cache.Hh, n_own))
    if g is not None:
        _need(g, "g", torch.float32, dev, (cache.B, n_own, n_hist))
    ws_bytes = bsa_route_workspace_size(cache.B, cache.Hh, cache.D, n_own, n_hist)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    cs = cache.c_struct()
    _check("bsa_route_qmean", _lib.bsa_route_qmean(
        _ptr(q_mean), ctypes.byref(cs), int(n_hist), int(own_first), int(n_own), _ptr(g),
        float(lam), float(g_ref), float(sm_scale), int(top_k), _ptr(idx), _ptr(cnt),
        int(max_sel), _ptr(workspace), workspace.numel(), _ptr(error_word(dev)), _stream(dev)))
    return idx, cnt


def velox_max_sel(n_hist: int, n_own: int, k_cov: int = 80, k_unc: int = 150, n_prev: int = 0,
                  window_half: int = 13, n_ref: int = 0) -> int:
    """Smallest max_sel bsa_route_velox accepts."""
    budget = max(k_cov, n_prev, k_unc)
    return min(n_hist, budget + 2 * window_half + 1 + n_ref) + n_own


def bsa_route_velox(q_blk: Optional[torch.Tensor], cache: KVCache, n_hist: int, own_first: int,
                    n_own: int, g: Optional[torch.Tensor] = None,
                    coverage: Optional[torch.Tensor] = None, lam: float = 2.0,
                    g_ref: float = 0.2, sm_scale: Optional[float] = None, tau: float = 0.1,
                    eta_cov: float = 0.9, k_cov: int = 80, k_unc: int = 150, mass: float = 0.9,
                    prev_first: int = 0, n_prev: int = 0, window_half: int = 13,
                    ref_first: int = 0, n_ref: int = 0, q_valid: Optional[torch.Tensor] = None,
                    max_sel: Optional[int] = None, idx: Optional[torch.Tensor] = None,
                    cnt: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    q_mean: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The page's full route; returns (idx [B,Hh,n_own,max_sel] padded with -1, cnt).
    With ``q_mean`` ([B, Hh, n_own, D] fp32, e.g. from
    bsa_tokens_to_blocks_mean) the query means are taken from it
    (bsa_route_velox_qmean) and ``q_blk`` may be None."""
    dev = cache.device
    if q_mean is not None:
        _need(q_mean, "q_mean", torch.float32, dev, (cache.B, cache.Hh, n_own, cache.D))
    else:
        _need(q_blk, "q_blk", torch.bfloat16, dev, (cache.B, cache.Hh, n_own * BLK, cache.D))
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(cache.D)
    if max_sel is None:
        max_sel = velox_max_sel(n_hist, n_own, k_cov, k_unc, n_prev, window_half, n_ref)
    if idx is None:
        idx = torch.empty((cache.B, cache.Hh, n_own, max_sel), dtype=torch.int32, device=dev)
    if cnt is None:
        cnt = torch.empty((cache.B, cache.Hh, n_own), dtype=torch.int32, device=dev)
    _need(idx, "idx", torch.int32, dev, (cache.B, cache.Hh, n_own, max_sel))
    _need(cnt, "cnt", torch.int32, dev, (cache.B, cache.Hh, n_own))
    if g is not None:
        _need(g, "g", torch.float32, dev, (cache.B, n_own, n_hist))
    if coverage is not None:
        _need(coverage, "coverage", torch.float32, dev, (cache.B, n_own))
    if q_valid is not None:
        _need(q_valid, "q_valid", torch.int32, dev, (n_own,))
    ws_bytes = bsa_route_workspace_size(cache.B, cache.Hh, cache.D, n_own, n_hist)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    opts = CVeloxRoute(None if coverage is None else coverage.data_ptr(), float(eta_cov),
                       float(tau), int(k_cov), int(k_unc), float(mass), int(prev_first),
                       int(n_prev), int(window_half), int(ref_first), int(n_ref))
    cs = cache.c_struct()
    if q_mean is not None:
        _check("bsa_route_velox_qmean", _lib.bsa_route_velox_qmean(
            _ptr(q_mean), ctypes.byref(cs), int(n_hist), int(own_first), int(n_own), _ptr(g),
            float(lam), float(g_ref), float(sm_scale), ctypes.byref(opts), _ptr(idx), _ptr(cnt),
            int(max_sel), _ptr(workspace), workspace.numel(), _ptr(error_word(dev)),
            _stream(dev)))
        return idx, cnt
    _check("bsa_route_velox", _lib.bsa_route_velox(
        _ptr(q_blk), ctypes.byref(cs), _ptr(q_valid), int(n_hist), int(own_first), int(n_own),
        _ptr(g), float(lam), float(g_ref), float(sm_scale), ctypes.byref(opts), _ptr(idx),
        _ptr(cnt), int(max_sel), _ptr(workspace), workspace.numel(), _ptr(error_word(dev)),
        _stream(dev)))
    return idx, cnt


def bsa_geometry_prior(cams: torch.Tensor, intr, h_cam: torch.Tensor, h_rect: torch.Tensor,
                       q_cam: Optional[torch.Tensor] = None, q_rect: Optional[torch.Tensor] = None,
                       tok_cam: Optional[torch.Tensor] = None,
                       tok_uvd: Optional[torch.Tensor] = None,
                       q_valid: Optional[torch.Tensor] = None, grid_n: int = 8,
                       g: Optional[torch.Tensor] = None, coverage: Optional[torch.Tensor] = None,
                       want_g: bool = True, want_coverage: bool = True):
    """Overlap prior g [B, n_q, n_hist] and coverage [B, n_q] from slabs.

    cams float32 [B, n_cams, 12]; intr = (fx, fy, cx, cy); h_cam int32
    [B, n_hist, S], h_rect float32 [B, n_hist, S, 6]; q_cam/q_rect likewise
    for the query blocks (needed for g); tok_cam int32 [B, n_q, 128] and
    tok_uvd float32 [B, n_q, 128, 3] (needed for coverage).  Returns (g,
    coverage), either None when not requested."""
    dev = _dev(cams.device)
    B, n_cams = cams.shape[0], cams.shape[1]
    _need(cams, "cams", torch.float32, dev, (B, n_cams, 12))
    n_hist, S = h_cam.shape[1], h_cam.shape[2]
    _need(h_cam, "h_cam", torch.int32, dev, (B, n_hist, S))
    _need(h_rect, "h_rect", torch.float32, dev, (B, n_hist, S, 6))
    n_q = (q_cam if q_cam is not None else tok_cam).shape[1]
    if want_g:
        _need(q_cam, "q_cam", torch.int32, dev, (B, n_q, S))
        _need(q_rect, "q_rect", torch.float32, dev, (B, n_q, S, 6))
        if g is None:
            g = torch.empty((B, n_q, n_hist), dtype=torch.float32, device=dev)
        _need(g, "g", torch.float32, dev, (B, n_q, n_hist))
    else:
        g = None
    if want_coverage:
        _need(tok_cam, "tok_cam", torch.int32, dev, (B, n_q, BLK))
        _need(tok_uvd, "tok_uvd", torch.float32, dev, (B, n_q, BLK, 3))
        if coverage is None:
            coverage = torch.empty((B, n_q), dtype=torch.float32, device=dev)
        _need(coverage, "coverage", torch.float32, dev, (B, n_q))
    else:
        coverage = None
    if q_valid is not None:
        _need(q_valid, "q_valid", torch.int32, dev, (n_q,))
    fx, fy, cx, cy = (float(v) for v in intr)
    _check("bsa_geometry_prior", _lib.bsa_geometry_prior(
        _ptr(cams), int(n_cams), fx, fy, cx, cy, _ptr(q_cam), _ptr(q_rect), int(n_q),
        _ptr(h_cam), _ptr(h_rect), int(n_hist), int(S), int(grid_n), _ptr(tok_cam), _ptr(tok_uvd),
        _ptr(q_valid), int(B), _ptr(g), _ptr(coverage), _ptr(error_word(dev)), _stream(dev)))
    return g, coverage


def bsa_attn(q_blk: torch.Tensor, cache: KVCache, idx: torch.Tensor, cnt: torch.Tensor,
             q_valid: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None,
             o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None
             ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Indexed block-sparse attention; returns (O bf16 [B,Hh,nQB*128,D], LSE fp32 [B,Hh,nQB*128])."""
    dev = cache.device
    if q_blk.dim() != 4:
        raise ValueError("q_blk must be [B, Hh, nQB*128, D]")
    B, Hh, R, D = q_blk.shape
    if (B, Hh, D) != (cache.B, cache.Hh, cache.D) or R % BLK:
        raise ValueError("q_blk does not match the cache")
    nqb = R // BLK
    _need(q_blk, "q_blk", torch.bfloat16, dev)
    if idx.dim() != 4 or tuple(idx.shape[:3]) != (B, Hh, nqb):
        raise ValueError("idx must be [B, Hh, nQB, max_sel]")
    max_sel = idx.shape[3]
    _need(idx, "idx", torch.int32, dev)
    _need(cnt, "cnt", torch.int32, dev, (B, Hh, nqb))
    if q_valid is not None:
        _need(q_valid, "q_valid", torch.int32, dev, (nqb,))
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    if o is None:
        o = torch.empty_like(q_blk)
    if lse is None:
        lse = torch.empty((B, Hh, R), dtype=torch.float32, device=dev)
    _need(o, "o", torch.bfloat16, dev, tuple(q_blk.shape))
    _need(lse, "lse", torch.float32, dev, (B, Hh, R))
    cs = cache.c_struct()
    _check("bsa_attn", _lib.bsa_attn(
        _ptr(q_blk), ctypes.byref(cs), _ptr(q_valid), _ptr(idx), _ptr(cnt), int(nqb),
        int(max_sel), float(sm_scale), _ptr(o), _ptr(lse), _ptr(error_word(dev)), _stream(dev)))
    return o, lse


def bsa_attn_tokens(q_blk: torch.Tensor, cache: KVCache, idx: torch.Tensor, cnt: torch.Tensor,
                    T: int, H: int, W: int, q_valid: Optional[torch.Tensor] = None,
                    sm_scale: Optional[float] = None, o: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None,
                    table: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """bsa_attn writing O and LSE in raster token order; returns
    (O bf16 [B, T*H*W, Hh, D], LSE fp32 [B, T*H*W, Hh])."""
    dev = cache.device
    if q_blk.dim() != 4:
        raise ValueError("q_blk must be [B, Hh, nQB*128, D]")
    B, Hh, R, D = q_blk.shape
    nqb = n_blocks_for(T, H, W)
    if (B, Hh, D) != (cache.B, cache.Hh, cache.D) or R != nqb * BLK:
        raise ValueError("q_blk does not match the cache and the chunk shape")
    _need(q_blk, "q_blk", torch.bfloat16, dev)
    if idx.dim() != 4 or tuple(idx.shape[:3]) != (B, Hh, nqb):
        raise ValueError("idx must be [B, Hh, nQB, max_sel]")
    max_sel = idx.shape[3]
    _need(idx, "idx", torch.int32, dev)
    _need(cnt, "cnt", torch.int32, dev, (B, Hh, nqb))
    if q_valid is not None:
        _need(q_valid, "q_valid", torch.int32, dev, (nqb,))
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    N = T * H * W
    if o is None:
        o = torch.empty((B, N, Hh, D), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, N, Hh), dtype=torch.float32, device=dev)
    _need(o, "o", torch.bfloat16, dev, (B, N, Hh, D))
    _need(lse, "lse", torch.float32, dev, (B, N, Hh))
    perm = gilbert_perm_device(T, H, W, dev) if table else None
    cs = cache.c_struct()
    _check("bsa_attn_tokens", _lib.bsa_attn_tokens(
        _ptr(q_blk), ctypes.byref(cs), _ptr(q_valid), _ptr(idx), _ptr(cnt), int(max_sel),
        float(sm_scale), int(T), int(H), int(W), _ptr(perm), _ptr(o), _ptr(lse),
        _ptr(error_word(dev)), _stream(dev)))
    return o, lse


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------

ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}


def _whole(x) -> int:
    """A position or a count as an int; a fraction is refused, not cut off."""
    i = int(x)
    if i != x:
        raise TypeError(f"{x!r} is not a whole number")
    return i


def _chunk(T, H, W) -> Tuple[int, int, int]:
    if type(T) is type(H) is type(W) is int:
        return T, H, W
    return _whole(T), _whole(H), _whole(W)


def bsa_rope_frequencies(n_pairs: int, base: float = 10000.0, scaling: str = "none",
                         factor: float = 1.0, original_length: float = 1.0,
                         beta_fast: float = 32.0, beta_slow: float = 1.0
                         ) -> Tuple[np.ndarray, float]:
    """(frequencies in radians per position (host float64 [n_pairs]), amplitude)
    of one axis; ``scaling`` is "none", "linear", "base" or "by_parts"."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    n_pairs = _whole(n_pairs)
    out = np.empty(max(n_pairs, 1), dtype=np.float64)
    amp = ctypes.c_double(1.0)
    _check("bsa_rope_frequencies", _lib.bsa_rope_frequencies(
        n_pairs, float(base), ROPE_SCALINGS[scaling], float(factor), float(original_length),
        float(beta_fast), float(beta_slow), out.ctypes.data_as(ctypes.c_void_p),
        ctypes.byref(amp)))
    return out[:n_pairs], float(amp.value)


def bsa_rope_phases(freqs) -> np.ndarray:
    """Frequencies (radians per position) as 64-bit fractions of a turn (host int64)."""
    f = np.ascontiguousarray(freqs, dtype=np.float64).reshape(-1)
    out = np.empty(max(f.size, 1), dtype=np.int64)
    _check("bsa_rope_phases", _lib.bsa_rope_phases(f.ctypes.data_as(ctypes.c_void_p), f.size,
                                                    out.ctypes.data_as(ctypes.c_void_p)))
    return out[:f.size]


class Rope:
    """Rotary positions: the phase table on a device, the pairs of each axis, the
    layout and the amplitude.

    ``pairs`` is (P,) for one position per token or (Pt, Ph, Pw) for the
    (t, h, w) positions of a chunk's grid; every axis with its own frequencies
    base^(-i / pairs of the axis), scaled as in :func:`bsa_rope_frequencies`."""

    def __init__(self, pairs, layout: str = "interleaved", base: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, original_length: float = 1.0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
        pairs = tuple(_whole(p) for p in pairs)
        made = [bsa_rope_frequencies(p, base, scaling, factor, original_length, beta_fast,
                                     beta_slow) for p in pairs if p > 0]
        if not made:
            raise ValueError("pairs must turn at least one pair")
        self._set(np.concatenate([f for f, _ in made]), pairs, layout, made[0][1], device)

    @classmethod
    def from_frequencies(cls, freqs, pairs, layout: str = "interleaved", amplitude: float = 1.0,
                         device="cuda") -> "Rope":
        """From frequencies in radians per position, section by section."""
        self = cls.__new__(cls)
        self._set(freqs, pairs, layout, amplitude, device)
        return self

    def _set(self, freqs, pairs, layout, amplitude, device):
        pairs = tuple(_whole(p) for p in pairs)
        if len(pairs) not in (1, 3) or min(pairs) < 0:
            raise ValueError("pairs must be (P,) or (Pt, Ph, Pw)")
        if layout not in ROPE_LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
        phase = bsa_rope_phases(freqs)
        if phase.size != sum(pairs):
            raise ValueError(f"{phase.size} frequencies for {sum(pairs)} pairs")
        self.pairs, self.layout, self.amplitude = pairs, layout, float(amplitude)
        self.device = _dev(device)
        self.phase = torch.from_numpy(phase).to(self.device)
        p = pairs + (0,) * (3 - len(pairs))
        self._struct = CRope(None, (ctypes.c_int32 * 3)(*p), len(pairs), ROPE_LAYOUTS[layout], 0,
                             self.amplitude, None, (ctypes.c_int32 * 3)(0, 0, 0))

    @property
    def n_axes(self) -> int:
        return len(self.pairs)

    def c_struct(self, B: int, N: int, pos: Optional[torch.Tensor], origin,
                 inverse: bool = False) -> CRope:
        if pos is not None:
            _need(pos, "pos", torch.int32, self.device, (self.n_axes, B, N))
        c = CRope.from_buffer_copy(self._struct)
        c.phase = self.phase.data_ptr()
        if pos is not None:
            c.pos = pos.data_ptr()
        c.inverse = int(bool(inverse))
        origin = tuple(origin)
        at = tuple(map(int, origin))
        if at != origin:
            raise TypeError("origin must be three whole positions")
        o0, o1, o2 = at
        for x in (o0, o1, o2):
            if not -(1 << 31) <= x < (1 << 31):
                raise ValueError("origin must be three int32 positions")
        c.origin[0], c.origin[1], c.origin[2] = o0, o1, o2
        return c


def _on(device, fn: str, *args):
    """Call the library with ``device`` current."""
    call = getattr(_lib, fn)
    if device.index == torch.cuda.current_device():
        _check(fn, call(*args))
    else:
        with torch.cuda.device(device):
            _check(fn, call(*args))


def _rope_struct(rope: Optional[Rope], dev, B, N, pos, origin, inverse=False):
    if rope is None:
        return None
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    if rope.device != dev:
        raise ValueError(f"rope is on {rope.device}, expected {dev}")
    return ctypes.byref(rope.c_struct(B, N, pos, origin, inverse))


def _perm_or_gilbert(perm: Optional[torch.Tensor], T: int, H: int, W: int, dev):
    """The caller's slot table, or the Gilbert table, or (for chunks too large
    for a table) None: the kernels then walk the curve."""
    if perm is not None:
        _need(perm, "perm", torch.int32, dev, (T * H * W,))
        return perm
    return gilbert_perm_device(T, H, W, dev) if T * H * W <= GATHER_MAX_TOKENS else None


GATHER_MAX_TOKENS = 1 << 14


def _tokens_shape(x: torch.Tensor, name: str, T: int, H: int, W: int):
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        raise ValueError(f"{name} must be [B, T*H*W, Hh, D]")
    if x.shape[1] != T * H * W:
        raise ValueError(f"{name} has {x.shape[1]} tokens, expected {T * H * W}")
    _need(x, name, torch.bfloat16)
    return x.shape


def bsa_rope(x_tok: torch.Tensor, T: int, H: int, W: int, rope: Rope,
             pos: Optional[torch.Tensor] = None, origin=(0, 0, 0), inverse: bool = False,
             out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotary positions of raster tokens (bf16 [B, T*H*W, Hh, D]); a sequence of
    n tokens is T = n, H = W = 1.  ``pos`` (int32 [axes, B, T*H*W]) gives every
    token's positions, otherwise the grid does; ``origin`` is added to both.
    ``inverse`` turns back: the gradient of the call.  ``out`` may be x_tok."""
    T, H, W = _chunk(T, H, W)
    B, N, Hh, D = _tokens_shape(x_tok, "x_tok", T, H, W)
    dev = x_tok.device
    if out is None:
        out = torch.empty_like(x_tok)
    else:
        _need(out, "out", torch.bfloat16, dev, x_tok.shape)
    if rope is None:
        raise TypeError("rope must be a Rope")
    _on(dev, "bsa_rope", _ptr(x_tok), _ptr(out), B, Hh, D, T, H, W,
        _rope_struct(rope, dev, B, N, pos, origin, inverse), _stream(dev))
    return out


def bsa_tokens_to_blocks_rope(x_tok: torch.Tensor, T: int, H: int, W: int, rope: Rope,
                              pos: Optional[torch.Tensor] = None, origin=(0, 0, 0),
                              out: Optional[torch.Tensor] = None,
                              mean: Optional[torch.Tensor] = None, want_mean: bool = False,
                              perm: Optional[torch.Tensor] = None):
    """bsa_tokens_to_blocks of the turned tokens in one pass; returns the blocks,
    or (blocks, means) with ``want_mean`` or a ``mean`` buffer (the means by a second
    kernel).  ``perm`` (int32
    [T*H*W], token -> slot) replaces the Gilbert order."""
    T, H, W = _chunk(T, H, W)
    B, N, Hh, D = _tokens_shape(x_tok, "x_tok", T, H, W)
    dev = x_tok.device
    nb = n_blocks_for(T, H, W)
    if out is None:
        out = torch.empty((B, Hh, nb * BLK, D), dtype=torch.bfloat16, device=dev)
    else:
        _need(out, "out", torch.bfloat16, dev, (B, Hh, nb * BLK, D))
    if mean is not None:
        _need(mean, "mean", torch.float32, dev, (B, Hh, nb, D))
    elif want_mean:
        mean = torch.empty((B, Hh, nb, D), dtype=torch.float32, device=dev)
    if rope is None:
        raise TypeError("rope must be a Rope")
    table = _perm_or_gilbert(perm, T, H, W, dev)
    _on(dev, "bsa_tokens_to_blocks_rope", _ptr(x_tok), _ptr(out), _ptr(mean), B, Hh, D, T, H, W,
        _ptr(table), _rope_struct(rope, dev, B, N, pos, origin),
        _ptr(error_word(dev)), _stream(dev))
    return out if mean is None else (out, mean)


def bsa_kv_append_rope(cache: KVCache, k_tok: torch.Tensor, v_tok: torch.Tensor, T: int, H: int,
                       W: int, rope: Rope, pos: Optional[torch.Tensor] = None, origin=(0, 0, 0),
                       perm: Optional[torch.Tensor] = None) -> int:
    """bsa_kv_append with the keys turned on the way; returns the first block."""
    T, H, W = _chunk(T, H, W)
    dev = cache.device
    shape = (cache.B, T * H * W, cache.Hh, cache.D)
    _need(k_tok, "k_tok", torch.bfloat16, dev, shape)
    _need(v_tok, "v_tok", torch.bfloat16, dev, shape)
    if rope is None:
        raise TypeError("rope must be a Rope")
    table = _perm_or_gilbert(perm, T, H, W, dev)
    cs = cache.c_struct()
    first = cache.n_blocks
    _on(dev, "bsa_kv_append_rope", ctypes.byref(cs), _ptr(k_tok), _ptr(v_tok), T, H, W,
        _ptr(table), _rope_struct(rope, dev, cache.B, T * H * W, pos, origin),
        _ptr(error_word(dev)), _stream(dev))
    cache.n_blocks = int(cs.n_blocks)
    return first


# ---------------------------------------------------------------------------
# 8-bit KV cache
# ---------------------------------------------------------------------------

class KVCache8:
    """A caller-owned block KV cache in 8 bits: K, V e4m3 [B, Hh, max_blocks, 128,
    D], one fp32 scale per (batch, head, block) for each, the valid-row counts,
    and optionally the pooled keys.  The route calls take it as they take a
    :class:`KVCache` with pooled keys (they read only those)."""

    def __init__(self, B: int, Hh: int, D: int, max_blocks: int, device="cuda",
                 pooled_keys: bool = False):
        dev = _dev(device)
        shape = (int(B), int(Hh), int(max_blocks), BLK, int(D))
        self._set(torch.zeros(shape, dtype=torch.float8_e4m3fn, device=dev),
                  torch.ones(shape[:3], dtype=torch.float32, device=dev),
                  torch.zeros(shape, dtype=torch.float8_e4m3fn, device=dev),
                  torch.ones(shape[:3], dtype=torch.float32, device=dev),
                  torch.zeros(shape[2], dtype=torch.int32, device=dev), 0,
                  torch.zeros(shape[:3] + shape[4:], dtype=torch.float32, device=dev)
                  if pooled_keys else None)

    @classmethod
    def from_tensors(cls, k: torch.Tensor, k_scale: torch.Tensor, v: torch.Tensor,
                     v_scale: torch.Tensor, block_valid: torch.Tensor, n_blocks: int,
                     kmean: Optional[torch.Tensor] = None) -> "KVCache8":
        """A cache over the caller's own tensors, ``n_blocks`` blocks of it in use."""
        self = cls.__new__(cls)
        self._set(k, k_scale, v, v_scale, block_valid, n_blocks, kmean)
        return self

    def _set(self, k, k_scale, v, v_scale, block_valid, n_blocks, kmean):
        if not isinstance(k, torch.Tensor) or k.dim() != 5 or k.shape[3] != BLK:
            raise ValueError("k must be [B, Hh, max_blocks, 128, D]")
        B, Hh, nb, _, D = k.shape
        _need(k, "k", torch.float8_e4m3fn)
        _need(v, "v", torch.float8_e4m3fn, k.device, k.shape)
        _need(k_scale, "k_scale", torch.float32, k.device, (B, Hh, nb))
        _need(v_scale, "v_scale", torch.float32, k.device, (B, Hh, nb))
        _need(block_valid, "block_valid", torch.int32, k.device, (nb,))
        if kmean is not None:
            _need(kmean, "kmean", torch.float32, k.device, (B, Hh, nb, D))
        if not 0 <= int(n_blocks) <= nb:
            raise ValueError(f"n_blocks must lie in [0, {nb}]")
        self.k, self.k_scale, self.v, self.v_scale = k, k_scale, v, v_scale
        self.block_valid, self.kmean = block_valid, kmean
        self.B, self.Hh, self.D, self.max_blocks = B, Hh, D, nb
        self.n_blocks, self.device = int(n_blocks), k.device

    def c_struct(self) -> CCache:
        """The route calls' view: pooled keys, no bf16 K or V."""
        return CCache(None, None, self.block_valid.data_ptr(), self.B, self.Hh, self.D,
                      self.max_blocks, self.n_blocks,
                      None if self.kmean is None else self.kmean.data_ptr())

    def c_struct8(self) -> CCache8:
        return CCache8(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(),
                       self.v_scale.data_ptr(), self.block_valid.data_ptr(), self.B, self.Hh,
                       self.D, self.max_blocks, self.n_blocks,
                       None if self.kmean is None else self.kmean.data_ptr())


def _need_cache8(cache):
    if not isinstance(cache, KVCache8):
        raise TypeError("cache must be a KVCache8")


def bsa_kv8_append(cache: KVCache8, k_tok: torch.Tensor, v_tok: torch.Tensor, T: int, H: int,
                   W: int, rope: Optional[Rope] = None, pos: Optional[torch.Tensor] = None,
                   origin=(0, 0, 0), perm: Optional[torch.Tensor] = None) -> int:
    """Append one chunk (bf16 [B, T*H*W, Hh, D] K and V) to an 8-bit cache, the keys
    turned on the way when ``rope`` is given; returns its first block."""
    _need_cache8(cache)
    T, H, W = _chunk(T, H, W)
    dev = cache.device
    shape = (cache.B, T * H * W, cache.Hh, cache.D)
    _need(k_tok, "k_tok", torch.bfloat16, dev, shape)
    _need(v_tok, "v_tok", torch.bfloat16, dev, shape)
    table = _perm_or_gilbert(perm, T, H, W, dev)
    cs = cache.c_struct8()
    first = cache.n_blocks
    _on(dev, "bsa_kv8_append", ctypes.byref(cs), _ptr(k_tok), _ptr(v_tok), T, H, W,
        _ptr(table), _rope_struct(rope, dev, cache.B, T * H * W, pos, origin),
        _ptr(error_word(dev)), _stream(dev))
    cache.n_blocks = int(cs.n_blocks)
    return first


def bsa_kv8_attn(q_blk: torch.Tensor, cache: KVCache8, idx: torch.Tensor, cnt: torch.Tensor,
                 q_valid: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None,
                 o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, torch.Tensor]:
    """bsa_attn over an 8-bit cache: q_blk bf16 [B, Hq, nQB*128, D] with Hq a multiple
    of the cache's Hh, one route per cache head (idx [B, Hh, nQB, max_sel], cnt [B,
    Hh, nQB]); returns (O like q_blk, LSE fp32 [B, Hq, nQB*128]).  For grouped heads,
    bsa_route_qmean takes the query means averaged over each group."""
    _need_cache8(cache)
    dev = cache.device
    if q_blk.dim() != 4:
        raise ValueError("q_blk must be [B, Hq, nQB*128, D]")
    B, Hq, R, D = q_blk.shape
    if (B, D) != (cache.B, cache.D) or Hq % cache.Hh or Hq == 0 or R % BLK:
        raise ValueError("q_blk does not match the cache")
    nqb = R // BLK
    _need(q_blk, "q_blk", torch.bfloat16, dev)
    if idx.dim() != 4 or tuple(idx.shape[:3]) != (B, cache.Hh, nqb):
        raise ValueError("idx must be [B, Hh, nQB, max_sel]")
    _need(idx, "idx", torch.int32, dev)
    _need(cnt, "cnt", torch.int32, dev, (B, cache.Hh, nqb))
    if q_valid is not None:
        _need(q_valid, "q_valid", torch.int32, dev, (nqb,))
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    if o is None:
        o = torch.empty_like(q_blk)
    if lse is None:
        lse = torch.empty((B, Hq, R), dtype=torch.float32, device=dev)
    _need(o, "o", torch.bfloat16, dev, q_blk.shape)
    _need(lse, "lse", torch.float32, dev, (B, Hq, R))
    cs = cache.c_struct8()
    _on(dev, "bsa_kv8_attn", _ptr(q_blk), ctypes.byref(cs), Hq, _ptr(q_valid), _ptr(idx),
        _ptr(cnt), nqb, idx.shape[3], float(sm_scale), _ptr(o), _ptr(lse), _ptr(error_word(dev)),
        _stream(dev))
    return o, lse


def bsa_kv8_attn_decode_workspace_size(B: int, Hq: int, Hh: int, D: int, n_tok: int,
                                       n_sel: int) -> int:
    """Bytes of workspace for routes of at most n_sel blocks (or n_sel blocks in use)."""
    n = ctypes.c_size_t(0)
    _check("bsa_kv8_attn_decode_workspace_size", _lib.bsa_kv8_attn_decode_workspace_size(
        int(B), int(Hq), int(Hh), int(D), int(n_tok), int(n_sel), ctypes.byref(n)))
    return int(n.value)


def bsa_kv8_attn_decode(q_tok: torch.Tensor, cache: KVCache8, idx: Optional[torch.Tensor] = None,
                        cnt: Optional[torch.Tensor] = None, sm_scale: Optional[float] = None,
                        o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of a few query tokens (bf16 [B, n_tok, Hq, D], n_tok * Hq / Hh at most
    128) over an 8-bit cache: over the blocks of one route per cache head (idx [B,
    Hh, max_sel], cnt [B, Hh]), or over every block in use when both are None.
    Returns (O like q_tok, LSE fp32 [B, n_tok, Hq])."""
    _need_cache8(cache)
    dev = cache.device
    if q_tok.dim() != 4:
        raise ValueError("q_tok must be [B, n_tok, Hq, D]")
    B, n_tok, Hq, D = q_tok.shape
    if (B, D) != (cache.B, cache.D) or Hq % cache.Hh or Hq == 0 or n_tok == 0:
        raise ValueError("q_tok does not match the cache")
    _need(q_tok, "q_tok", torch.bfloat16, dev)
    if (idx is None) != (cnt is None):
        raise ValueError("idx and cnt come together")
    max_sel = 0
    if idx is not None:
        if idx.dim() != 3 or tuple(idx.shape[:2]) != (B, cache.Hh):
            raise ValueError("idx must be [B, Hh, max_sel]")
        _need(idx, "idx", torch.int32, dev)
        _need(cnt, "cnt", torch.int32, dev, (B, cache.Hh))
        max_sel = idx.shape[2]
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    if o is None:
        o = torch.empty_like(q_tok)
    if lse is None:
        lse = torch.empty((B, n_tok, Hq), dtype=torch.float32, device=dev)
    _need(o, "o", torch.bfloat16, dev, q_tok.shape)
    _need(lse, "lse", torch.float32, dev, (B, n_tok, Hq))
    if workspace is None:
        size = bsa_kv8_attn_decode_workspace_size(B, Hq, cache.Hh, D, n_tok,
                                                  cache.n_blocks if idx is None else max_sel)
        workspace = torch.empty(max(size, 256), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    cs = cache.c_struct8()
    _on(dev, "bsa_kv8_attn_decode", _ptr(q_tok), ctypes.byref(cs), Hq, n_tok, _ptr(idx), _ptr(cnt),
        max_sel, float(sm_scale), _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(),
        _ptr(error_word(dev)), _stream(dev))
    return o, lse


def bsa_check_device_error(device="cuda", d_err: Optional[torch.Tensor] = None) -> Tuple[int, int]:
    """Synchronise, read and clear the device error word: (status, raw BSA_DEV_* code)."""
    dev = _dev(device)
    err = error_word(dev) if d_err is None else d_err
    code = ctypes.c_int32(0)
    st = _lib.bsa_check_device_error(_ptr(err), _stream(dev), ctypes.byref(code))
    return int(st), int(code.value)


def bsa_selftest_bounded_wait(device="cuda", limit_cycles: int = 2_000_000) -> Tuple[int, int]:
    """Run the bounded-wait self-test; returns bsa_check_device_error's
    (status, code), which should be (BSA_ERR_TIMEOUT, BSA_DEV_WAIT_TIMEOUT)."""
    dev = _dev(device)
    _check("bsa_selftest_bounded_wait", _lib.bsa_selftest_bounded_wait(
        _ptr(error_word(dev)), int(limit_cycles), _stream(dev)))
    return bsa_check_device_error(dev)


def raise_on_device_error(device="cuda"):
    """Raise :class:`BsaError` if a kernel reported a device-side problem."""
    st, code = bsa_check_device_error(device)
    if st != 0:
        raise BsaError("device", st, DEV_CODES.get(code, str(code)))
