"""CSA2 hot path on B200: a thin ctypes binding over libcsa2.so.

Every function here only marshals arguments (torch tensors -> device
pointers, sizes, the current CUDA stream) and calls the C ABI declared in
``include/csa2.h``; all computation runs in the library's sm_100a kernels.
There is no CPU fallback: if the library is missing or a tensor is not on
a CUDA device, the call raises.

Functions mirror the C entry points: ``pack_fp4``, ``unpack_fp4``,
``index_topk``, ``sparse_attn_decode``, ``sparse_attn_prefill``,
``layer_group_run``, plus ``validate_modes``, ``group_cache_bytes`` and
``get_device_status``; and, for the 8-bit paged key/value cache (``KV8Cache``),
``block_tables``, ``kv8_append``, ``kv8_unpack``, ``kv8_select`` and
``kv8_attn``.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Dict, List, Optional, Sequence, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcsa2.so")

CSA2_OK, CSA2_ERR_INVALID_ARG, CSA2_ERR_UNSUPPORTED, CSA2_ERR_CUDA = 0, 1, 2, 3
CSA2_ERR_WORKSPACE, CSA2_ERR_DEVICE_STATUS = 4, 5
FULL, REINDEX, REUSE, REINDEX_POOL = 0, 1, 2, 3

EXPORTED = (
    "csa2_status_string", "csa2_version", "csa2_pack_fp4", "csa2_unpack_fp4",
    "csa2_index_topk_workspace_size", "csa2_index_topk", "csa2_sparse_attn_workspace_size",
    "csa2_sparse_attn_decode", "csa2_sparse_attn_prefill", "csa2_validate_modes",
    "csa2_group_cache_bytes", "csa2_layer_group_workspace_size", "csa2_layer_group_run",
    "csa2_get_device_status", "csa2_trace_enable", "csa2_trace_count", "csa2_trace_get",
    "csa2_layer_run", "csa2_index_topk_noalloc", "csa2_index_pool_workspace_size",
    "csa2_index_pool", "csa2_pool_topk_workspace_size", "csa2_pool_topk", "csa2_append_entry",
    "csa2_pack_index_keys_fp4", "csa2_index_topk_fp4k_workspace_size", "csa2_index_topk_fp4k",
    "csa2_wait_timeout_selftest", "csa2_set_decode_kernel", "csa2_get_decode_kernel",
    "csa2_stage_copies", "csa2_block_tables", "csa2_kv8_append", "csa2_kv8_unpack",
    "csa2_kv8_select_workspace_size", "csa2_kv8_select", "csa2_kv8_attn_workspace_size",
    "csa2_kv8_attn",
)
DECODE_SCAN_CLUSTER, DECODE_FUSED = 0, 1


class CSA2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib().csa2_status_string(status).decode()}")


class LayerMode(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int32), ("kv_src", ctypes.c_int32), ("idx_src", ctypes.c_int32)]


class Dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("D", ctypes.c_int32), ("N", ctypes.c_int64), ("H_I", ctypes.c_int32),
                ("d_I", ctypes.c_int32), ("topk", ctypes.c_int32), ("W", ctypes.c_int32),
                ("n_prior", ctypes.c_int64), ("ratio", ctypes.c_int32),
                ("sm_scale", ctypes.c_float), ("pool_block", ctypes.c_int32),
                ("pool_blocks", ctypes.c_int32)]


class Copy2D(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("row_bytes", ctypes.c_int64), ("src_stride", ctypes.c_int64),
                ("dst_stride", ctypes.c_int64)]


class KV8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_sum", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("Hk", ctypes.c_int32), ("block", ctypes.c_int32),
                ("D", ctypes.c_int32)]


MAX_STAGE_COPIES = 16


class LayerIO(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "q", "q_idx", "w", "win_k", "win_v", "codes", "scales", "k_idx", "idx", "out", "lse",
        "k_exps", "app_src", "app_key", "app_pos", "pool")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libcsa2.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m compressed_sparse_attention_topk_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_size_t)
    sig = {
        "csa2_status_string": ([i32], ctypes.c_char_p),
        "csa2_version": ([], i32),
        "csa2_pack_fp4": ([P, i64, i32, P, P, P], i32),
        "csa2_unpack_fp4": ([P, P, i64, i32, P, P], i32),
        "csa2_append_entry": ([P, P, P, i32, i32, i32, i64, P, P, P, P], i32),
        "csa2_pack_index_keys_fp4": ([P, i64, i32, P, P, P], i32),
        "csa2_index_topk_fp4k_workspace_size": ([i32, i32, i32, i64, i32], sz),
        "csa2_index_topk_fp4k": ([P, P, P, P, i32, i32, i32, i64, i32, P, P, sz, P], i32),
        "csa2_index_topk_workspace_size": ([i32, i32, i32, i32, i64, i32], sz),
        "csa2_index_topk": ([P, P, P, i32, i32, i32, i32, i64, i64, i32, i32, P, P, P, sz, P], i32),
        "csa2_sparse_attn_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
        "csa2_sparse_attn_decode": ([P, P, P, P, P, P, i32, i32, i32, i64, i32, i32, f32, P, P, P,
                                     sz, P], i32),
        "csa2_sparse_attn_prefill": ([P, P, P, P, P, P, i32, i32, i32, i32, i64, i32, i32, f32, P,
                                      P, P, sz, P], i32),
        "csa2_validate_modes": ([P, i32], i32),
        "csa2_group_cache_bytes": ([P, i32, i64, i64, i64, P], i32),
        "csa2_layer_group_workspace_size": ([P], sz),
        "csa2_layer_group_run": ([P, P, i32, P, P, sz, P], i32),
        "csa2_layer_run": ([P, P, i32, i32, P, P, sz, P], i32),
        "csa2_index_topk_noalloc": ([P, P, P, i32, i32, i32, i32, i64, i64, i32, i32, P, P, P],
                                    i32),
        "csa2_index_pool_workspace_size": ([i32, i32, i32, i64, i32, i32], sz),
        "csa2_index_pool": ([P, P, P, i32, i32, i32, i64, i32, i32, P, P, sz, P], i32),
        "csa2_pool_topk_workspace_size": ([i32, i32, i32], sz),
        "csa2_pool_topk": ([P, P, P, i32, i32, i32, i64, P, i32, i32, P, P, sz, P], i32),
        "csa2_stage_copies": ([P, i32, P], i32),
        "csa2_block_tables": ([P, P, i32, i32, P, i32, P, i32, P, P, P, P, i64, P, P], i32),
        "csa2_kv8_append": ([P, P, i64, P, i64, P, i64, P], i32),
        "csa2_kv8_unpack": ([P, P, i64, P, P, P], i32),
        "csa2_kv8_select_workspace_size": ([i64, i32, i32], sz),
        "csa2_kv8_select": ([P, i64, P, P, i32, P, P, i32, i64, i32, i32, i32, i32, P, P, sz, P],
                            i32),
        "csa2_kv8_attn_workspace_size": ([i64, i32, i32, i32, i32, i32], sz),
        "csa2_kv8_attn": ([P, i64, P, P, i32, P, P, i32, i64, i32, P, i32, f32, P, P, P, sz, P],
                          i32),
        "csa2_get_device_status": ([P, P], i32),
        "csa2_wait_timeout_selftest": ([i64, P], i32),
        "csa2_set_decode_kernel": ([i32], i32),
        "csa2_get_decode_kernel": ([], i32),
        "csa2_trace_enable": ([i32], i32),
        "csa2_trace_count": ([], i32),
        "csa2_trace_get": ([i32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(f32)], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(rc: int, what: str):
    if rc != CSA2_OK:
        raise CSA2Error(rc, what)


# --- torch marshalling --------------------------------------------------------

def _torch():
    import torch
    return torch


def _dev(t, name, dtype=None):
    torch = _torch()
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device=None) -> int:
    return _torch().cuda.current_stream(device).cuda_stream


_ws_cache: Dict[int, object] = {}


def workspace(nbytes: int, device=None):
    """A cached uint8 device buffer of at least nbytes (grown on demand)."""
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    key = dev.index if dev.index is not None else torch.cuda.current_device()
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < max(nbytes, 1):
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        _ws_cache[key] = buf
    return buf


# --- staging copies -----------------------------------------------------------

def _rows_of(t, name):
    """(rows, row bytes, row stride in bytes) of a tensor whose last dim is
    contiguous and whose leading dims collapse to rows of one stride."""
    es = t.element_size()
    if t.dim() == 0:
        return 1, es, es
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dim must be contiguous")
    if t.dim() == 1:
        return 1, t.shape[0] * es, t.shape[0] * es
    for i in range(t.dim() - 2):
        if t.shape[i] > 1 and t.stride(i) != t.stride(i + 1) * t.shape[i + 1]:
            raise ValueError(f"{name}: the leading dims must collapse to rows of one stride")
    rows = 1
    for n in t.shape[:-1]:
        rows *= n
    return rows, t.shape[-1] * es, t.stride(-2) * es


def stage_copies(pairs):
    """One launch copying each (src, dst) tensor pair (same shape and dtype;
    each a CUDA tensor of the current device or a pinned CPU tensor; last
    dim contiguous, leading dims collapsing to rows of one stride; 16-byte
    aligned rows), at most MAX_STAGE_COPIES pairs, on the current stream."""
    torch = _torch()
    pairs = list(pairs)
    if len(pairs) > MAX_STAGE_COPIES:
        raise ValueError(f"at most {MAX_STAGE_COPIES} copies per launch")
    arr = (Copy2D * max(len(pairs), 1))()
    for i, (src, dst) in enumerate(pairs):
        for name, t in (("src", src), ("dst", dst)):
            if not isinstance(t, torch.Tensor) or not (t.is_cuda or t.is_pinned()):
                raise TypeError(f"pairs[{i}].{name} must be a CUDA or pinned CPU tensor")
        if src.shape != dst.shape or src.dtype != dst.dtype:
            raise ValueError(f"pairs[{i}]: src and dst differ in shape or dtype")
        rows, rb, ss = _rows_of(src, f"pairs[{i}].src")
        _, _, ds = _rows_of(dst, f"pairs[{i}].dst")
        arr[i] = Copy2D(src.data_ptr(), dst.data_ptr(), rows, rb, ss, ds)
    _check(lib().csa2_stage_copies(arr, len(pairs), _stream()), "csa2_stage_copies")


# --- FP4 ----------------------------------------------------------------------

def pack_fp4(src, codes=None, scales=None) -> Tuple[object, object]:
    """fp32 [..., D] -> (uint8 [..., D/2] codes, fp32 [..., D/16] scales)."""
    torch = _torch()
    src = _dev(src, "src", torch.float32)
    D = src.shape[-1]
    rows = src.numel() // D if D else 0
    if codes is None:
        codes = torch.empty(src.shape[:-1] + (D // 2,), dtype=torch.uint8, device=src.device)
    if scales is None:
        scales = torch.empty(src.shape[:-1] + (D // 16,), dtype=torch.float32, device=src.device)
    _check(lib().csa2_pack_fp4(_ptr(src), rows, D, _ptr(codes), _ptr(scales), _stream()),
           "csa2_pack_fp4")
    return codes, scales


def append_entry(src, key, pos, codes, scales, k_idx):
    """One decode step's entry append, in place: for each sequence b with
    pos[b] >= 0, src[b] (fp32 [B, D]) packed to FP4 into row pos[b] of
    codes [B, N, D/2] / scales [B, N, D/16] and key[b] (int8 [B, d_I]) into
    row pos[b] of k_idx [B, N, d_I]; pos is int64 [B] on the device."""
    torch = _torch()
    src = _dev(src, "src", torch.float32)
    key = _dev(key, "key", torch.int8)
    pos = _dev(pos, "pos", torch.int64)
    codes = _dev(codes, "codes", torch.uint8)
    scales = _dev(scales, "scales", torch.float32)
    k_idx = _dev(k_idx, "k_idx", torch.int8)
    B, D = src.shape
    d_I = key.shape[1]
    N = codes.shape[1]
    _check(lib().csa2_append_entry(_ptr(src), _ptr(key), _ptr(pos), B, D, d_I, N, _ptr(codes),
                                   _ptr(scales), _ptr(k_idx), _stream()), "csa2_append_entry")


def unpack_fp4(codes, scales, D: int, out=None):
    torch = _torch()
    codes = _dev(codes, "codes", torch.uint8)
    scales = _dev(scales, "scales", torch.float32)
    rows = codes.numel() // (D // 2)
    if out is None:
        out = torch.empty(codes.shape[:-1] + (D,), dtype=torch.float32, device=codes.device)
    _check(lib().csa2_unpack_fp4(_ptr(codes), _ptr(scales), rows, D, _ptr(out), _stream()),
           "csa2_unpack_fp4")
    return out


# --- indexer + top-k ----------------------------------------------------------

def index_topk_workspace_size(B, T, H_I, d_I, N, topk) -> int:
    return int(lib().csa2_index_topk_workspace_size(B, T, H_I, d_I, N, topk))


def index_topk(q_idx, w, k_idx, topk: int, n_prior: int = -1, ratio: int = 4, idx_out=None,
               want_scores: bool = False, ws=None):
    """q_idx int8 [B,T,H_I,d_I], w fp32 [B,T,H_I], k_idx int8 [B,N,d_I] ->
    idx int32 [B,T,topk] (and fp32 scores [B,T,N] when want_scores)."""
    torch = _torch()
    q_idx = _dev(q_idx, "q_idx", torch.int8)
    w = _dev(w, "w", torch.float32)
    k_idx = _dev(k_idx, "k_idx", torch.int8)
    B, T, H_I, d_I = q_idx.shape
    N = k_idx.shape[1]
    if idx_out is None:
        idx_out = torch.empty((B, T, topk), dtype=torch.int32, device=q_idx.device)
    scores = (torch.empty((B, T, N), dtype=torch.float32, device=q_idx.device)
              if want_scores else None)
    need = index_topk_workspace_size(B, T, H_I, d_I, N, topk)
    if ws is None:
        ws = workspace(need)
    _check(lib().csa2_index_topk(_ptr(q_idx), _ptr(w), _ptr(k_idx), B, T, H_I, d_I, N, n_prior,
                                 ratio, topk, _ptr(idx_out), _ptr(scores), _ptr(ws), ws.numel(),
                                 _stream()), "csa2_index_topk")
    return (idx_out, scores) if want_scores else idx_out


# --- FP4 index keys -----------------------------------------------------------

def pack_index_keys_fp4(src, codes=None, exps=None):
    """fp32 [..., d_I] -> (uint8 [..., d_I/2] E2M1 codes, uint8 [..., d_I/32]
    biased block exponents): FP4 index keys with one power-of-two scale per
    32 elements."""
    torch = _torch()
    src = _dev(src, "src", torch.float32)
    d_I = src.shape[-1]
    rows = src.numel() // d_I if d_I else 0
    if codes is None:
        codes = torch.empty(src.shape[:-1] + (d_I // 2,), dtype=torch.uint8, device=src.device)
    if exps is None:
        exps = torch.empty(src.shape[:-1] + (d_I // 32,), dtype=torch.uint8, device=src.device)
    _check(lib().csa2_pack_index_keys_fp4(_ptr(src), rows, d_I, _ptr(codes), _ptr(exps),
                                          _stream()), "csa2_pack_index_keys_fp4")
    return codes, exps


def index_topk_fp4k(q_idx, w, codes, exps, topk: int, idx_out=None, ws=None):
    """Decode rows over FP4 index keys: q_idx int8 [B,H_I,d_I] (or
    [B,1,H_I,d_I]), w fp32 [B,H_I], codes uint8 [B,N,d_I/2], exps uint8
    [B,N,d_I/32] -> idx int32 [B, topk]."""
    torch = _torch()
    q_idx = _dev(q_idx, "q_idx", torch.int8)
    w = _dev(w, "w", torch.float32)
    codes = _dev(codes, "codes", torch.uint8)
    exps = _dev(exps, "exps", torch.uint8)
    B = q_idx.shape[0]
    H_I, d_I = q_idx.shape[-2:]
    N = codes.shape[1]
    if idx_out is None:
        idx_out = torch.empty((B, topk), dtype=torch.int32, device=q_idx.device)
    if ws is None:
        ws = workspace(int(lib().csa2_index_topk_fp4k_workspace_size(B, H_I, d_I, N, topk)))
    _check(lib().csa2_index_topk_fp4k(_ptr(q_idx), _ptr(w), _ptr(codes), _ptr(exps), B, H_I, d_I,
                                      N, topk, _ptr(idx_out), _ptr(ws), ws.numel(), _stream()),
           "csa2_index_topk_fp4k")
    return idx_out


# --- hierarchical indexer -----------------------------------------------------

def index_pool_workspace_size(B, H_I, d_I, N, block, n_blocks) -> int:
    return int(lib().csa2_index_pool_workspace_size(B, H_I, d_I, N, block, n_blocks))


def index_pool(q_idx, w, k_idx, block: int = 8, n_blocks: int = 2048, ws=None):
    """Candidate pool of each sequence's Full-layer query: q_idx int8
    [B,H_I,d_I], w fp32 [B,H_I], k_idx int8 [B,N,d_I] -> int32
    [B, n_blocks*block] positions ascending, then -1."""
    torch = _torch()
    q_idx = _dev(q_idx, "q_idx", torch.int8)
    w = _dev(w, "w", torch.float32)
    k_idx = _dev(k_idx, "k_idx", torch.int8)
    B, H_I, d_I = q_idx.shape
    N = k_idx.shape[1]
    pool = torch.empty((B, n_blocks * block), dtype=torch.int32, device=q_idx.device)
    if ws is None:
        ws = workspace(index_pool_workspace_size(B, H_I, d_I, N, block, n_blocks))
    _check(lib().csa2_index_pool(_ptr(q_idx), _ptr(w), _ptr(k_idx), B, H_I, d_I, N, block,
                                 n_blocks, _ptr(pool), _ptr(ws), ws.numel(), _stream()),
           "csa2_index_pool")
    return pool


def pool_topk_workspace_size(B, P, topk) -> int:
    return int(lib().csa2_pool_topk_workspace_size(B, P, topk))


def pool_topk(q_idx, w, k_idx, pool, topk: int, ws=None):
    """Top-k of each sequence's query within its pool (int32 [B, P],
    positions ascending then -1) -> int32 [B, topk] positions ascending,
    then -1."""
    torch = _torch()
    q_idx = _dev(q_idx, "q_idx", torch.int8)
    w = _dev(w, "w", torch.float32)
    k_idx = _dev(k_idx, "k_idx", torch.int8)
    pool = _dev(pool, "pool", torch.int32)
    B, H_I, d_I = q_idx.shape
    N = k_idx.shape[1]
    P = pool.shape[1]
    out = torch.empty((B, topk), dtype=torch.int32, device=q_idx.device)
    if ws is None:
        ws = workspace(pool_topk_workspace_size(B, P, topk))
    _check(lib().csa2_pool_topk(_ptr(q_idx), _ptr(w), _ptr(k_idx), B, H_I, d_I, N, _ptr(pool), P,
                                topk, _ptr(out), _ptr(ws), ws.numel(), _stream()),
           "csa2_pool_topk")
    return out


# --- attention ----------------------------------------------------------------

def sparse_attn_workspace_size(B, T, H, D, topk, W) -> int:
    return int(lib().csa2_sparse_attn_workspace_size(B, T, H, D, topk, W))


def _attn_common(q, codes, scales, idx, win_k, win_v):
    torch = _torch()
    q = _dev(q, "q", torch.bfloat16)
    codes = _dev(codes, "codes", torch.uint8)
    scales = _dev(scales, "scales", torch.float32)
    idx = _dev(idx, "idx", torch.int32)
    win_k = _dev(win_k, "win_k", torch.bfloat16)
    win_v = _dev(win_v, "win_v", torch.bfloat16)
    return q, codes, scales, idx, win_k, win_v


def sparse_attn_decode(q, codes, scales, idx, win_k, win_v, sm_scale: Optional[float] = None,
                       out=None, lse=None, ws=None):
    """q bf16 [B,H,D]; codes u8 [B,N,D/2]; scales fp32 [B,N,D/16]; idx int32
    [B,topk]; win_k/win_v bf16 [B,W,D] (or None) -> (out fp32 [B,H,D], lse fp32 [B,H])."""
    torch = _torch()
    q, codes, scales, idx, win_k, win_v = _attn_common(q, codes, scales, idx, win_k, win_v)
    B, H, D = q.shape
    N = codes.shape[1]
    topk = idx.shape[-1]
    W = 0 if win_k is None else win_k.shape[1]
    sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    need = sparse_attn_workspace_size(B, 1, H, D, topk, W)
    if ws is None:
        ws = workspace(need)
    _check(lib().csa2_sparse_attn_decode(_ptr(q), _ptr(codes), _ptr(scales), _ptr(idx),
                                         _ptr(win_k), _ptr(win_v), B, H, D, N, topk, W,
                                         sm_scale, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                         _stream()), "csa2_sparse_attn_decode")
    return out, lse


def sparse_attn_prefill(q, codes, scales, idx, win_k, win_v, sm_scale: Optional[float] = None,
                        out=None, lse=None, ws=None):
    """q bf16 [B,T,H,D]; idx int32 [B,T,topk]; win_k/win_v bf16 [B,W-1+T,D]
    -> (out fp32 [B,T,H,D], lse fp32 [B,T,H])."""
    torch = _torch()
    q, codes, scales, idx, win_k, win_v = _attn_common(q, codes, scales, idx, win_k, win_v)
    B, T, H, D = q.shape
    N = codes.shape[1]
    topk = idx.shape[-1]
    W = 0 if win_k is None else win_k.shape[1] - T + 1
    sm_scale = 1.0 / math.sqrt(D) if sm_scale is None else sm_scale
    if out is None:
        out = torch.empty((B, T, H, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    need = sparse_attn_workspace_size(B, T, H, D, topk, W)
    if ws is None:
        ws = workspace(need)
    _check(lib().csa2_sparse_attn_prefill(_ptr(q), _ptr(codes), _ptr(scales), _ptr(idx),
                                          _ptr(win_k), _ptr(win_v), B, T, H, D, N, topk, W,
                                          sm_scale, _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
                                          _stream()), "csa2_sparse_attn_prefill")
    return out, lse


# --- 8-bit paged key/value cache ------------------------------------------------
#
# These calls serve decode steps of a few microseconds, so their marshalling
# is kept short: types and layouts are checked, the fixed parts of a cache
# once (KV8Cache), and the current stream is read without building a Stream.

_types = None


def _kv8_types():
    """(torch, int32, int64, bfloat16, float32, uint8), imported once."""
    global _types
    if _types is None:
        torch = _torch()
        _types = (torch, torch.int32, torch.int64, torch.bfloat16, torch.float32, torch.uint8)
    return _types


def _check_dense(t, name, dtype, dev):
    """A contiguous CUDA tensor of this dtype on device `dev` (the current one:
    the calls launch on its current stream)."""
    if not isinstance(t, _types[0].Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    return t


def _check_tokens(t, name, D, heads, dev):
    """A bf16 [n, heads, D] CUDA tensor whose tokens may be strided, the heads
    of a token dense; returns (n, heads, token stride in elements)."""
    if not isinstance(t, _types[0].Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != _types[3]:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [n, heads, {D}]")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if d != D or (heads is not None and h != heads):
        raise ValueError(f"{name} must be [n, {'heads' if heads is None else heads}, {D}]")
    if n > 0 and (s2 != 1 or (h > 1 and s1 != D)):
        raise ValueError(f"{name}: the heads of a token must be dense")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    return n, h, (s0 if n > 1 else h * D)  # (one token's stride leads nowhere)


def _check_step(cache, table, cu, lens, dev):
    """table [B, width], cu [B + 1] and lens [B] of a step, and the cache's
    device; returns (B, width)."""
    i32 = _types[1]
    _check_dense(table, "table", i32, dev)
    _check_dense(cu, "cu", i32, dev)
    _check_dense(lens, "lens", i32, dev)
    B, width = table.shape
    if cu.numel() != B + 1 or lens.numel() != B:
        raise ValueError("table is [B, width], cu [B+1], lens [B]")
    if cache.device != dev:
        raise ValueError(f"the cache is on cuda:{cache.device}, the current device is cuda:{dev}")
    return B, width


@functools.lru_cache(maxsize=256)
def _ws_bytes(dev, query, *sizes):
    """A workspace query's answer: it depends on the device and the sizes alone."""
    return max(int(getattr(lib(), query)(*sizes)), 256)


def _scratch(ws, like, dev, query, *sizes):
    """The caller's workspace, or a new one of this call: from the caching
    allocator, so calls on other streams and captured graphs never share it."""
    if ws is not None:
        return _check_dense(ws, "ws", _types[5], dev)
    return like.new_empty(_ws_bytes(dev, query, *sizes), dtype=_types[5])


def block_tables(lens, add, table, free_pages, block: int, cap: int, out=None):
    """Block tables and slot maps of a step: request b holds lens[b] tokens and
    adds add[b] (int32 [B]); the pages it needs are taken, request by request,
    from the front of free_pages (int32) and written into its row of table
    (int32 [B, width], updated).  Returns (lens + add int32 [B], cu int32
    [B+1], slots int64 [cap], pos int32 [cap], used int32 [1]): token offsets,
    each token's slot (page * block + row) and position (-1 past the last
    token), pages taken.  ``out``: those five tensors, to write into (they
    overlap nothing else)."""
    torch, i32, i64 = _kv8_types()[:3]
    dev = torch.cuda.current_device()
    _check_dense(lens, "lens", i32, dev)
    _check_dense(add, "add", i32, dev)
    _check_dense(table, "table", i32, dev)
    _check_dense(free_pages, "free_pages", i32, dev)
    B, width = table.shape
    n_free = free_pages.numel()
    if lens.numel() != B or add.numel() != B:
        raise ValueError("lens and add are [B], table [B, width]")
    if out is None:
        lens_out, cu, pos, used = lens.new_empty(2 * B + 2 + cap).split((B, B + 1, cap, 1))
        slots = lens.new_empty(cap, dtype=i64)
        out = (lens_out, cu, slots, pos, used)
    else:
        for t, name, n, dt in zip(out, ("lens", "cu", "slots", "pos", "used"),
                                  (B, B + 1, cap, cap, 1), (i32, i32, i64, i32, i32)):
            if _check_dense(t, "out." + name, dt, dev).numel() != n:
                raise ValueError(f"out.{name} must have {n} elements")
        lens_out, cu, slots, pos, used = out
    rc = lib().csa2_block_tables(lens.data_ptr(), add.data_ptr(), B, block, table.data_ptr(),
                                 width, free_pages.data_ptr(), n_free, lens_out.data_ptr(),
                                 cu.data_ptr(), slots.data_ptr(), pos.data_ptr(), cap,
                                 used.data_ptr(), torch._C._cuda_getCurrentRawStream(dev))
    _check(rc, "csa2_block_tables")
    return out


class KV8Cache:
    """The tensors of an 8-bit paged cache, checked and marshalled once: int8
    k, v [pages, Hk, block, D], fp32 k_scale, v_scale [pages, Hk], int16 k_sum
    [pages, Hk, D] (contiguous CUDA tensors, kept alive by this handle, which
    takes no others later)."""

    def __init__(self, k, v, k_scale, v_scale, k_sum):
        torch = _kv8_types()[0]
        k, v = _dev(k, "k", torch.int8), _dev(v, "v", torch.int8)
        k_scale = _dev(k_scale, "k_scale", torch.float32)
        v_scale = _dev(v_scale, "v_scale", torch.float32)
        k_sum = _dev(k_sum, "k_sum", torch.int16)
        if k.dim() != 4:
            raise ValueError("k must be [pages, Hk, block, D]")
        P, Hk, block, D = k.shape
        if (v.shape != k.shape or k_scale.shape != (P, Hk) or v_scale.shape != (P, Hk)
                or k_sum.shape != (P, Hk, D)):
            raise ValueError("v must be like k, k_scale and v_scale [pages, Hk], k_sum "
                             "[pages, Hk, D]")
        device = k.get_device()
        if any(x.get_device() != device for x in (v, k_scale, v_scale, k_sum)):
            raise ValueError("the tensors of a cache must be on one device")
        c = KV8(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(k_sum), P, Hk, block, D)
        self.__dict__.update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, k_sum=k_sum, pages=P,
                             Hk=Hk, block=block, D=D, device=device, _c=c, _ref=ctypes.byref(c))

    def __setattr__(self, name, value):
        # the calls go by the pointers marshalled above: another tensor in an
        # attribute would leave them at memory that nothing keeps
        raise AttributeError(f"{name}: the tensors of a KV8Cache stay, make a new one")

    @classmethod
    def empty(cls, pages: int, Hk: int, block: int, D: int, device="cuda") -> "KV8Cache":
        """A new cache, all zeros."""
        torch = _torch()

        def zeros(dtype, *shape):
            return torch.zeros(shape, dtype=dtype, device=device)

        return cls(zeros(torch.int8, pages, Hk, block, D), zeros(torch.int8, pages, Hk, block, D),
                   zeros(torch.float32, pages, Hk), zeros(torch.float32, pages, Hk),
                   zeros(torch.int16, pages, Hk, D))


def kv8_append(cache: KV8Cache, k_new, v_new, slots):
    """Write tokens' keys and values (bf16 [n, Hk, D], tokens may be strided)
    at their slots (int64 [n], page * block + row; negative: nothing), in
    place.  The tokens of a page are consecutive, at ascending rows."""
    torch, _, i64 = _kv8_types()[:3]
    dev = torch.cuda.current_device()
    nk, _, ks = _check_tokens(k_new, "k_new", cache.D, cache.Hk, dev)
    nv, _, vs = _check_tokens(v_new, "v_new", cache.D, cache.Hk, dev)
    n = _check_dense(slots, "slots", i64, dev).numel()
    if nk != n or nv != n:
        raise ValueError("k_new, v_new and slots must have one row per token")
    if cache.device != dev:
        raise ValueError(f"the cache is on cuda:{cache.device}, the current device is cuda:{dev}")
    _check(lib().csa2_kv8_append(cache._ref, k_new.data_ptr(), ks, v_new.data_ptr(), vs,
                                 slots.data_ptr(), n, torch._C._cuda_getCurrentRawStream(dev)),
           "csa2_kv8_append")


def kv8_unpack(cache: KV8Cache, slots, k_out=None, v_out=None):
    """The rows at slots (int64 [n]) as fp32 [n, Hk, D] keys and values (zeros
    for a negative slot)."""
    torch, _, i64, _, f32, _ = _kv8_types()
    dev = torch.cuda.current_device()
    n = _check_dense(slots, "slots", i64, dev).numel()
    shape = (n, cache.Hk, cache.D)
    if cache.device != dev:
        raise ValueError(f"the cache is on cuda:{cache.device}, the current device is cuda:{dev}")
    if k_out is None:
        k_out = cache.k_scale.new_empty(shape)
    elif _check_dense(k_out, "k_out", f32, dev).shape != shape:
        raise ValueError("k_out must be [n, Hk, D]")
    if v_out is None:
        v_out = cache.v_scale.new_empty(shape)
    elif _check_dense(v_out, "v_out", f32, dev).shape != shape:
        raise ValueError("v_out must be [n, Hk, D]")
    _check(lib().csa2_kv8_unpack(cache._ref, slots.data_ptr(), n, k_out.data_ptr(),
                                 v_out.data_ptr(), torch._C._cuda_getCurrentRawStream(dev)),
           "csa2_kv8_unpack")
    return k_out, v_out


def kv8_select_workspace_size(n, Hk, width) -> int:
    return int(lib().csa2_kv8_select_workspace_size(n, Hk, width))


def kv8_select(q, cache: KV8Cache, table, cu, lens, n_sel: int, n_first: int = 1,
               n_last: int = 1, out=None, ws=None):
    """The n_sel blocks that each token (q bf16 [n, H, D]) and kv head attends
    to: its first n_first, its last n_last and the best-scored others, int32
    [n, Hk, n_sel] ascending, then -1.  table int32 [B, width], cu int32
    [B+1] token offsets, lens int32 [B] tokens in the cache."""
    torch, i32 = _kv8_types()[:2]
    dev = torch.cuda.current_device()
    n, H, stride = _check_tokens(q, "q", cache.D, None, dev)
    B, width = _check_step(cache, table, cu, lens, dev)
    if out is None:
        out = cu.new_empty((n, cache.Hk, n_sel))
    elif _check_dense(out, "out", i32, dev).shape != (n, cache.Hk, n_sel):
        raise ValueError("out must be [n, Hk, n_sel]")
    ws = _scratch(ws, cu, dev, "csa2_kv8_select_workspace_size", n, cache.Hk, width)
    _check(lib().csa2_kv8_select(q.data_ptr(), stride, cache._ref, table.data_ptr(), width,
                                 cu.data_ptr(), lens.data_ptr(), B, n, H, n_sel, n_first, n_last,
                                 out.data_ptr(), ws.data_ptr(), ws.numel(),
                                 torch._C._cuda_getCurrentRawStream(dev)), "csa2_kv8_select")
    return out


def kv8_attn_workspace_size(n, B, H, Hk, D, n_sel=0) -> int:
    return int(lib().csa2_kv8_attn_workspace_size(n, B, H, Hk, D, n_sel))


def kv8_attn(q, cache: KV8Cache, table, cu, lens, sel=None, sm_scale: Optional[float] = None,
             out=None, lse=None, ws=None):
    """Causal attention of a step's tokens over the cache (their own keys and
    values already appended): q bf16 [n, H, D], table int32 [B, width], cu
    int32 [B+1], lens int32 [B]; sel int32 [n, Hk, n_sel >= 1]: only the
    listed blocks -> (out bf16 [n, H, D], lse fp32 [n, H])."""
    torch, i32, _, bf16, f32, _ = _kv8_types()
    dev = torch.cuda.current_device()
    D = cache.D
    n, H, stride = _check_tokens(q, "q", D, None, dev)
    B, width = _check_step(cache, table, cu, lens, dev)
    sel_ptr, n_sel = None, 0
    if sel is not None:
        if _check_dense(sel, "sel", i32, dev).dim() != 3 or sel.shape[:2] != (n, cache.Hk):
            raise ValueError("sel must be [n, Hk, n_sel]")
        if sel.shape[2] == 0:  # (the C call takes a null pointer as every block)
            raise ValueError("sel must have room for a block: n_sel >= 1")
        sel_ptr, n_sel = sel.data_ptr(), sel.shape[2]
    if out is None:
        out = q.new_empty((n, H, D))
    elif _check_dense(out, "out", bf16, dev).shape != (n, H, D):
        raise ValueError("out must be [n, H, D]")
    if lse is None:
        lse = cache.k_scale.new_empty((n, H))
    elif _check_dense(lse, "lse", f32, dev).shape != (n, H):
        raise ValueError("lse must be [n, H]")
    ws = _scratch(ws, cu, dev, "csa2_kv8_attn_workspace_size", n, B, H, cache.Hk, D, n_sel)
    rc = lib().csa2_kv8_attn(q.data_ptr(), stride, cache._ref, table.data_ptr(), width,
                             cu.data_ptr(), lens.data_ptr(), B, n, H, sel_ptr, n_sel,
                             D ** -0.5 if sm_scale is None else sm_scale, out.data_ptr(),
                             lse.data_ptr(), ws.data_ptr(), ws.numel(),
                             torch._C._cuda_getCurrentRawStream(dev))
    _check(rc, "csa2_kv8_attn")
    return out, lse


# --- cross-layer groups ---------------------------------------------------------

def _modes_array(modes: Sequence[Tuple[int, int, int]]):
    arr = (LayerMode * len(modes))()
    for i, (m, kv, ix) in enumerate(modes):
        arr[i].mode, arr[i].kv_src, arr[i].idx_src = m, kv, ix
    return arr


def validate_modes(modes) -> bool:
    arr = _modes_array(modes)
    return lib().csa2_validate_modes(arr, len(modes)) == CSA2_OK


def group_cache_bytes(modes, entries: int, numbers_per_entry: int, bits_per_number: int) -> int:
    arr = _modes_array(modes)
    out = ctypes.c_uint64(0)
    _check(lib().csa2_group_cache_bytes(arr, len(modes), entries, numbers_per_entry,
                                        bits_per_number, ctypes.byref(out)),
           "csa2_group_cache_bytes")
    return int(out.value)


def make_dims(B, T, H, D, N, H_I, d_I, topk, W, n_prior=-1, ratio=4, sm_scale=None,
              pool_block=0, pool_blocks=0) -> Dims:
    return Dims(B, T, H, D, N, H_I, d_I, topk, W, n_prior, ratio,
                1.0 / math.sqrt(D) if sm_scale is None else sm_scale, pool_block, pool_blocks)


def layer_group_workspace_size(dims: Dims) -> int:
    return int(lib().csa2_layer_group_workspace_size(ctypes.byref(dims)))


def layer_group_run(modes, layers: List[dict], dims: Dims, ws=None):
    """Run a mode table.  ``layers[l]`` holds the layer's device tensors
    (q, q_idx, w, win_k, win_v, idx, out, lse and, for Full layers, codes,
    scales, k_idx)."""
    arr = _modes_array(modes)
    io = (LayerIO * len(layers))()
    for i, lay in enumerate(layers):
        for name, _ in LayerIO._fields_:
            t = lay.get(name)
            if t is not None:
                _dev(t, f"layers[{i}].{name}")
            setattr(io[i], name, _ptr(t))
    need = layer_group_workspace_size(dims)
    if ws is None:
        ws = workspace(need)
    _check(lib().csa2_layer_group_run(arr, io, len(layers), ctypes.byref(dims), _ptr(ws),
                                      ws.numel(), _stream()), "csa2_layer_group_run")


class LayerGroup:
    """A mode table with its layers' device tensors, marshalled once, so a
    layer (or the whole group) can be launched repeatedly with one C call
    (e.g. inside CUDA graph capture)."""

    def __init__(self, modes, layers: List[dict], dims: Dims, ws=None):
        self.modes = _modes_array(modes)
        self.L = len(layers)
        self.layers = layers
        self.io = (LayerIO * self.L)()
        for i, lay in enumerate(layers):
            for name, _ in LayerIO._fields_:
                t = lay.get(name)
                if t is not None:
                    _dev(t, f"layers[{i}].{name}")
                setattr(self.io[i], name, _ptr(t))
        self.dims = dims
        need = layer_group_workspace_size(dims)
        self.ws = workspace(need) if ws is None else ws

    def run_layer(self, layer: int):
        _check(lib().csa2_layer_run(self.modes, self.io, self.L, layer, ctypes.byref(self.dims),
                                    _ptr(self.ws), self.ws.numel(), _stream()), "csa2_layer_run")

    def run(self):
        _check(lib().csa2_layer_group_run(self.modes, self.io, self.L, ctypes.byref(self.dims),
                                          _ptr(self.ws), self.ws.numel(), _stream()),
               "csa2_layer_group_run")


def set_decode_kernel(kernel: int):
    """DECODE_SCAN_CLUSTER (default) or DECODE_FUSED: which kernels serve
    decode rows (process-wide)."""
    _check(lib().csa2_set_decode_kernel(kernel), "csa2_set_decode_kernel")


def get_decode_kernel() -> int:
    return int(lib().csa2_get_decode_kernel())


def get_device_status() -> int:
    code = ctypes.c_int32(0)
    rc = lib().csa2_get_device_status(_stream(), ctypes.byref(code))
    if rc not in (CSA2_OK, CSA2_ERR_DEVICE_STATUS):
        raise CSA2Error(rc, "csa2_get_device_status")
    return int(code.value)


# --- kernel timing trace -----------------------------------------------------------

def trace_enable(on: bool = True):
    _check(lib().csa2_trace_enable(1 if on else 0), "csa2_trace_enable")


def trace_records() -> List[Tuple[str, float]]:
    """(kernel name, device ms) of every launch recorded since trace_enable."""
    out = []
    name = ctypes.c_char_p()
    ms = ctypes.c_float()
    for i in range(lib().csa2_trace_count()):
        _check(lib().csa2_trace_get(i, ctypes.byref(name), ctypes.byref(ms)), "csa2_trace_get")
        out.append((name.value.decode(), float(ms.value)))
    return out
