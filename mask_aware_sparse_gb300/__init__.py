"""Python binding of libfm (include/fm.h): FlashMask column-wise masked attention on GB300.

Argument marshalling only. Every step of the computation runs in the CUDA
kernels of libfm.so; torch supplies device memory and the current stream.
Importing works without a GPU; the first call loads libfm.so and raises if it
is missing (build it with `mask_aware_sparse_gb300.build.build()`), so there
is no silent fallback.

Functions carry the names of the C entry points:
  fm_classify_tiles, fm_attn_fwd, fm_attn_fwd_fp8, fm_attn_bwd, fm_attn_fwd_heads and
  fm_attn_bwd_heads (per-head mask vectors), fm_attn_fwd_multi and fm_attn_bwd_multi
  (multi-interval masks), fm_attn_fwd_bwd_host (host buffers in
  and out, device workspace), fm_localize, fm_device_status,
  fm_selftest_wait_timeout, fm_profile_enable, fm_profile_read, fm_launch_count,
  fm_from_fms_fme, fm_merge_parts, fm_sum_parts, fm_chunk_loads,
  fm_balance_chunks, fm_needed_chunks (host code: the chunk balancer and the
  K / V exchange plan for context parallelism);
  fm_rope_freqs, fm_qk_norm_rope, fm_qk_norm_rope_bwd (per-head norm and rotation of
  queries and keys), fm_cache_write, fm_cache_read, fm_attn_paged (the paged key /
  value cache and the attention of new tokens over it), fm_cache_append (norm, rotation
  and the cache's write in one pass), fm_cache_copy, fm_attn_shared (the attention where
  groups of sequences share their first keys);
plus KVCache, PagedBatch, SharedPrefix and fm_cache_new (a cache, a batch and its groups,
checked once and kept by a serving program), QKNormRope (the norm and rotation of a
flashmask_attention call), fm_classify_tiles_heads (fm_classify_tiles over the B * H_q rows of
per-head vectors), fm_attn_multi_interval and fm_attn_per_head (the library
calls of a multi-interval / per-head forward and backward in sequence) and
flashmask_attention (autograd wrapper: the classification, forward and
backward calls in one differentiable op).
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading
from dataclasses import dataclass

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# FM_LIBRARY=debug selects the range-checked debug build (build.build(debug=True))
LIB_PATH = os.path.join(_HERE, "libfm_debug.so" if os.environ.get("FM_LIBRARY") == "debug" else "libfm.so")

FM_OK, FM_ERR_INVALID_ARG, FM_ERR_UNSUPPORTED, FM_ERR_WORKSPACE, FM_ERR_CUDA, FM_ERR_TIMEOUT, FM_ERR_DEVICE = range(7)
FM_DEVERR_TIMEOUT, FM_DEVERR_RANGE, FM_DEVERR_QUEUE, FM_DEVERR_DEBUG = 1, 2, 4, 8


class fm_problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("N", ctypes.c_int32),
                ("d", ctypes.c_int32), ("scale", ctypes.c_float), ("causal", ctypes.c_int32), ("N_kv", ctypes.c_int32)]


class fm_tiling(ctypes.Structure):
    _fields_ = [("block_m", ctypes.c_int32), ("block_n", ctypes.c_int32)]


class fm_balance_report(ctypes.Structure):
    _fields_ = [("lower_bound", ctypes.c_int64), ("lower_bound_kappa", ctypes.c_int64),
                ("makespan_lpt", ctypes.c_int64), ("makespan_pair", ctypes.c_int64),
                ("makespan", ctypes.c_int64), ("certified", ctypes.c_int32), ("pair_moves", ctypes.c_int32),
                ("triple_moves", ctypes.c_int32), ("budget_exhausted", ctypes.c_int32)]


class fm_view(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("sb", ctypes.c_int64), ("sh", ctypes.c_int64), ("sn", ctypes.c_int64)]


class fm_rows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("st", ctypes.c_int64), ("sh", ctypes.c_int64)]


class fm_qk_problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("w_f32", ctypes.c_int32), ("eps", ctypes.c_float), ("rot_scale", ctypes.c_float),
                ("pos", ctypes.c_void_p), ("pos_sb", ctypes.c_int64), ("inv_freq", ctypes.c_void_p),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p)]


class fm_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p), ("n_pages", ctypes.c_int32), ("H_kv", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("d", ctypes.c_int32)]


class fm_paged_batch(ctypes.Structure):
    _fields_ = [("q_off", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("R", ctypes.c_int32), ("width", ctypes.c_int32)]


class fm_shared_prefix(ctypes.Structure):
    _fields_ = [("seq_off", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p), ("S", ctypes.c_int32),
                ("max_prefix", ctypes.c_int32)]


class FMError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


_lib = None

_P = ctypes.c_void_p
_VIEW, _ROWS = ctypes.POINTER(fm_view), ctypes.POINTER(fm_rows)
_CACHE, _BATCH, _SHARED = (ctypes.POINTER(t) for t in (fm_kv_cache, fm_paged_batch, fm_shared_prefix))
_SIGS = {
    "fm_rope_freqs": (ctypes.c_int, [ctypes.c_int32, ctypes.c_double, ctypes.c_int32, ctypes.c_double, ctypes.c_int64,
                                     ctypes.c_double, ctypes.c_double, _P, ctypes.POINTER(ctypes.c_float)]),
    "fm_qk_norm_rope": (ctypes.c_int, [ctypes.POINTER(fm_qk_problem)] + [_VIEW] * 6 + [_P]),
    "fm_qk_norm_rope_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(fm_qk_problem)]),
    "fm_qk_norm_rope_bwd": (ctypes.c_int, [ctypes.POINTER(fm_qk_problem)] + [_VIEW] * 8 + [_P] * 3
                            + [ctypes.c_size_t, _P]),
    "fm_cache_write": (ctypes.c_int, [_CACHE, _BATCH, ctypes.c_int32, _ROWS, _ROWS, _P]),
    "fm_cache_read": (ctypes.c_int, [_CACHE, _P, _P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P, _P]),
    "fm_attn_paged_workspace_bytes": (ctypes.c_size_t, [_CACHE, _BATCH, ctypes.c_int32, ctypes.c_int32]),
    "fm_attn_paged": (ctypes.c_int, [_CACHE, _BATCH, ctypes.c_int32, ctypes.c_int32, _ROWS, ctypes.c_float,
                                     ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _ROWS, _P, _P, ctypes.c_size_t,
                                     _P]),
    "fm_cache_append": (ctypes.c_int, [_CACHE, _BATCH, ctypes.POINTER(fm_qk_problem)] + [_ROWS] * 4 + [_P]),
    "fm_cache_copy": (ctypes.c_int, [_CACHE, _P, _P, ctypes.c_int32, _P]),
    "fm_attn_shared_workspace_bytes": (ctypes.c_size_t, [_CACHE, _BATCH, _SHARED, ctypes.c_int32, ctypes.c_int32]),
    "fm_attn_shared": (ctypes.c_int, [_CACHE, _BATCH, _SHARED, ctypes.c_int32, ctypes.c_int32, _ROWS, ctypes.c_float,
                                      ctypes.c_int32, _ROWS, _P, _P, ctypes.c_size_t, _P]),
    "fm_abi_version": (ctypes.c_int32, []),
    "fm_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "fm_attn_tiling": (ctypes.c_int, [ctypes.POINTER(fm_tiling)]),
    "fm_tile_counts": (ctypes.c_int, [ctypes.POINTER(fm_problem), ctypes.POINTER(fm_tiling),
                                      ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]),
    "fm_classify_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(fm_problem), ctypes.POINTER(fm_tiling)]),
    "fm_classify_tiles": (ctypes.c_int, [ctypes.POINTER(fm_problem), ctypes.POINTER(fm_tiling)] + [_P] * 9
                          + [_P, ctypes.c_size_t, _P]),
    "fm_attn_fwd_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(fm_problem)]),
    "fm_attn_fwd": (ctypes.c_int, [ctypes.POINTER(fm_problem)] + [_P] * 11 + [_P, ctypes.c_size_t, _P]),
    "fm_attn_fwd_noalloc": (ctypes.c_int, [ctypes.POINTER(fm_problem)] + [_P] * 11 + [_P]),
    "fm_attn_fwd_fp8": (ctypes.c_int, [ctypes.POINTER(fm_problem)] + [_P] * 3 + [ctypes.c_float] * 3 + [_P] * 8
                        + [_P, ctypes.c_size_t, _P]),
    "fm_attn_bwd_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(fm_problem)]),
    "fm_attn_fwd_heads_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(fm_problem)]),
    "fm_attn_fwd_heads": (ctypes.c_int, [ctypes.POINTER(fm_problem)] + [_P] * 11 + [_P, ctypes.c_size_t, _P]),
    "fm_attn_bwd_heads": (ctypes.c_int, [ctypes.POINTER(fm_problem)] + [_P] * 15 + [_P, ctypes.c_size_t, _P]),
    "fm_classify_multi_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(fm_problem), ctypes.POINTER(fm_tiling),
                                                            ctypes.c_int32]),
    "fm_classify_tiles_multi": (ctypes.c_int, [ctypes.POINTER(fm_problem), ctypes.POINTER(fm_tiling),
                                               ctypes.c_int32] + [_P] * 7 + [_P, ctypes.c_size_t, _P]),
    "fm_attn_fwd_multi": (ctypes.c_int, [ctypes.POINTER(fm_problem), ctypes.c_int32] + [_P] * 9 +
                          [_P, ctypes.c_size_t, _P]),
    "fm_attn_bwd_multi": (ctypes.c_int, [ctypes.POINTER(fm_problem), ctypes.c_int32] + [_P] * 13 +
                          [_P, ctypes.c_size_t, _P]),
    "fm_attn_host_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(fm_problem)]),
    "fm_attn_fwd_bwd_host": (ctypes.c_int, [ctypes.POINTER(fm_problem)] + [_P] * 13 + [_P, ctypes.c_size_t, _P]),
    "fm_attn_bwd": (ctypes.c_int, [ctypes.POINTER(fm_problem)] + [_P] * 15 + [_P, ctypes.c_size_t, _P]),
    "fm_localize": (ctypes.c_int, [_P, ctypes.c_int64, _P, ctypes.c_int32, ctypes.c_int32, _P, _P]),
    "fm_from_fms_fme": (ctypes.c_int, [_P, _P, ctypes.c_int64, ctypes.c_int32, _P, _P, _P, _P, _P]),
    "fm_merge_parts": (ctypes.c_int, [ctypes.c_int32, _P, _P, ctypes.c_int64, ctypes.c_int32, _P, _P, _P]),
    "fm_sum_parts": (ctypes.c_int, [ctypes.c_int32, _P, ctypes.c_int64, _P, _P]),
    "fm_device_status": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "fm_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_int64, _P]),
    "fm_profile_enable": (ctypes.c_int, [ctypes.c_int32]),
    "fm_profile_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int32),
                                       ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int32)]),
    "fm_launch_count": (ctypes.c_int64, []),
    "fm_chunk_loads": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                      ctypes.c_int64, ctypes.c_int64, _P]),
    "fm_balance_chunks": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_int64, _P, ctypes.POINTER(fm_balance_report)]),
    "fm_needed_chunks": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, ctypes.c_int32,
                                        ctypes.c_int32, ctypes.c_int32, _P]),
}
EXPORTS = tuple(_SIGS)


def lib():
    """The loaded libfm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with mask_aware_sparse_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(s: int) -> str:
    try:
        return lib().fm_status_string(int(s)).decode()
    except Exception:  # library not loadable: still give a message
        return "status"


def _check(st: int, what: str):
    if st != FM_OK:
        raise FMError(st, what)


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _problem(B, H_q, H_kv, N, d, scale, causal, N_kv=0) -> fm_problem:
    return fm_problem(int(B), int(H_q), int(H_kv), int(N), int(d), float(scale), 1 if causal else 0, int(N_kv))


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _like(t, name, shape, dtype):
    """t is a contiguous torch tensor of this shape and dtype (device checked separately)."""
    _need(isinstance(t, torch.Tensor), f"{name} must be a torch tensor")
    _need(tuple(t.shape) == tuple(shape), f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    _need(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
    _need(t.is_contiguous(), f"{name} must be contiguous")


def _same_cuda(**ts):
    """Every given tensor lives on one CUDA device (the library computes on the GPU only)."""
    dev = None
    for name, t in ts.items():
        if t is None:
            continue
        _need(t.is_cuda, f"{name} must be a CUDA tensor: the library computes on the GPU only")
        dev = t.device if dev is None else dev
        _need(t.device == dev, f"{name} is on {t.device}, the other tensors on {dev}")


def _vec_ok(*vs, shape=None):
    """Mask vectors: contiguous int32 CUDA tensors of one (B, N_kv) shape."""
    shape = tuple(vs[0].shape) if shape is None else tuple(shape)
    _need(len(shape) == 2, "mask vectors must be (B, N_kv)")
    for i, v in enumerate(vs):
        _like(v, f"mask vector {i}", shape, torch.int32)
    _same_cuda(**{f"mask vector {i}": v for i, v in enumerate(vs)})


def _bf16_ok(*ts):
    for t in ts:
        _need(isinstance(t, torch.Tensor) and t.dim() == 4,
              "Q/K/V/O/dO must be contiguous bf16 CUDA tensors of shape (B, H, N, d)")
        _like(t, "Q/K/V/O/dO", t.shape, torch.bfloat16)
    _same_cuda(**{f"tensor {i}": t for i, t in enumerate(ts)})


def _attn_args(q, k, v, vec, queues, *, backward, o=None, lse=None, do=None, dq=None, dk=None, dv=None, ws=None,
               heads=False, intervals=0):
    """Shapes, dtypes and devices of an attention call, checked before the library
    sees any pointer (the C ABI receives bare pointers and cannot check them).
    Shape checks come first, so a mismatch is reported as such. heads: per-head
    mask vectors (B, H_q, N_kv) and queues over B * H_q rows; intervals = M > 0:
    multi-interval FMS / FME (M, B, N_kv) (vec holds the two) and the union
    classification's queues over B rows."""
    _need(isinstance(q, torch.Tensor) and q.dim() == 4, "q must be a (B, H_q, N, d) tensor")
    B, Hq, N, d = q.shape
    _need(isinstance(k, torch.Tensor) and k.dim() == 4 and k.shape[0] == B and k.shape[3] == d,
          f"k has shape {tuple(k.shape)}, expected (B={B}, H_kv, N_kv, d={d})")
    Hkv, Nk = k.shape[1], k.shape[2]
    _need(Hkv > 0 and Hq % Hkv == 0, f"H_q={Hq} must be a multiple of H_kv={Hkv}")
    _like(q, "q", (B, Hq, N, d), torch.bfloat16)
    _like(k, "k", (B, Hkv, Nk, d), torch.bfloat16)
    _like(v, "v", (B, Hkv, Nk, d), torch.bfloat16)
    vshape = (B, Hq, Nk) if heads else (intervals, B, Nk) if intervals else (B, Nk)
    for i, x in enumerate(vec):
        _like(x, f"mask vector {i}", vshape, torch.int32)
    for name, t in (("o", o), ("do", do), ("dq", dq)):
        if t is not None:
            _like(t, name, (B, Hq, N, d), torch.bfloat16)
    if lse is not None:
        _like(lse, "lse", (B, Hq, N), torch.float32)
    for name, t in (("dk", dk), ("dv", dv)):
        if t is not None:
            _like(t, name, (B, Hkv, Nk, d), torch.bfloat16)
    if ws is not None:
        _need(isinstance(ws, torch.Tensor) and ws.is_contiguous(), "ws must be a contiguous tensor")
    _need(isinstance(queues, TileQueues), "queues must come from fm_classify_tiles")
    bm, bn = attn_tiling()
    _need((queues.block_m, queues.block_n) == (bm, bn),
          f"queues were built with {queues.block_m} x {queues.block_n} tiles; the kernels need {bm} x {bn}")
    nq, nk = -(-N // bm), -(-Nk // bn)
    R = B * Hq if heads else B  # queue rows per Q (K) block
    off, qu, nrows = (queues.k_off, queues.k_queue, R * nk) if backward else (queues.q_off, queues.q_queue, R * nq)
    _like(off, "queue offsets", (nrows + 1,), torch.int32)
    _need(isinstance(qu, torch.Tensor) and qu.dtype == torch.int32 and qu.is_contiguous()
          and qu.numel() >= max(1, R * nq * nk),
          f"queue entries must be int32 with capacity {R} * nQ * nK")
    _same_cuda(q=q, k=k, v=v, o=o, lse=lse, do=do, dq=dq, dk=dk, dv=dv, ws=ws, queue_offsets=off, queue=qu,
               **{f"mask vector {i}": x for i, x in enumerate(vec)})


def attn_tiling():
    t = fm_tiling()
    _check(lib().fm_attn_tiling(ctypes.byref(t)), "fm_attn_tiling")
    return t.block_m, t.block_n


@dataclass
class TileQueues:
    """Outputs of fm_classify_tiles (device tensors) and the tiling they were built with."""
    tile_class: torch.Tensor  # (B, nQ, nK) uint8: 0 skip, 1 partial, 2 unmasked
    q_off: torch.Tensor       # (B*nQ + 1,) int32
    q_queue: torch.Tensor     # (capacity,) int32, (kb << 1) | partial, kb descending per row
    k_off: torch.Tensor       # (B*nK + 1,) int32
    k_queue: torch.Tensor     # (capacity,) int32, (qb << 1) | partial, qb ascending per column
    block_m: int
    block_n: int


def fm_classify_tiles(lts, lte, uts, ute, *, causal: bool, block_m: int = 128, block_n: int = 128, n_rows=None,
                      stream=None):
    """Classify every (Q-block, KV-block) tile and build both compacted queues.

    The vectors are (B, N_kv); n_rows is the number of query rows N (default
    N_kv: the square problem)."""
    _vec_ok(lts, lte, uts, ute)
    B, Nk = lts.shape
    N = Nk if n_rows is None else int(n_rows)
    prob = _problem(B, 1, 1, N, 128, 1.0, causal, Nk)
    til = fm_tiling(block_m, block_n)
    nq, nk = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().fm_tile_counts(ctypes.byref(prob), ctypes.byref(til), ctypes.byref(nq), ctypes.byref(nk)),
           "fm_tile_counts")
    nq, nk = nq.value, nk.value
    dev = lts.device
    cap = max(1, B * nq * nk)
    cls = torch.empty((B, nq, nk), dtype=torch.uint8, device=dev)
    q_off = torch.empty(B * nq + 1, dtype=torch.int32, device=dev)
    k_off = torch.empty(B * nk + 1, dtype=torch.int32, device=dev)
    q_queue = torch.empty(cap, dtype=torch.int32, device=dev)
    k_queue = torch.empty(cap, dtype=torch.int32, device=dev)
    wsb = lib().fm_classify_workspace_bytes(ctypes.byref(prob), ctypes.byref(til))
    ws = torch.empty(max(1, wsb), dtype=torch.uint8, device=dev)
    _check(lib().fm_classify_tiles(ctypes.byref(prob), ctypes.byref(til), _ptr(lts), _ptr(lte), _ptr(uts), _ptr(ute),
                                   _ptr(cls), _ptr(q_off), _ptr(q_queue), _ptr(k_off), _ptr(k_queue), _ptr(ws),
                                   ctypes.c_size_t(wsb), _stream(stream)), "fm_classify_tiles")
    return TileQueues(cls, q_off, q_queue, k_off, k_queue, block_m, block_n)


def fm_attn_fwd(q, k, v, lts, lte, uts, ute, queues: TileQueues, *, scale: float, causal: bool, o=None, lse=None,
                ws=None, stream=None):
    """Forward: returns (O bf16 (B,H_q,N,d), LSE fp32 (B,H_q,N)); K, V may hold N_kv != N rows."""
    _attn_args(q, k, v, (lts, lte, uts, ute), queues, backward=False, o=o, lse=lse, ws=ws)
    B, Hq, N, d = q.shape
    prob = _problem(B, Hq, k.shape[1], N, d, scale, causal, k.shape[2])
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if lse is None else lse
    wsb = lib().fm_attn_fwd_workspace_bytes(ctypes.byref(prob))
    if ws is None or ws.numel() < wsb:
        ws = torch.empty(max(1, wsb), dtype=torch.uint8, device=q.device)
    _check(lib().fm_attn_fwd(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(lts), _ptr(lte), _ptr(uts),
                             _ptr(ute), _ptr(queues.q_off), _ptr(queues.q_queue), _ptr(o), _ptr(lse), _ptr(ws),
                             ctypes.c_size_t(wsb), _stream(stream)), "fm_attn_fwd")
    return o, lse


def fm_attn_fwd_fp8(q, k, v, lts, lte, uts, ute, queues: TileQueues, *, q_scale: float, k_scale: float,
                    v_scale: float, scale: float, causal: bool, o=None, lse=None, ws=None, stream=None):
    """FP8 forward: q, k, v are float8_e4m3fn (B, H, N, 128) tensors standing for
    stored x q_scale (k_scale, v_scale). Returns (O bf16, LSE fp32)."""
    e4 = torch.float8_e4m3fn
    _need(isinstance(q, torch.Tensor) and q.dim() == 4, "q must be a (B, H_q, N, d) tensor")
    B, Hq, N, d = q.shape
    _need(isinstance(k, torch.Tensor) and k.dim() == 4 and k.shape[0] == B and k.shape[3] == d,
          f"k has shape {tuple(k.shape)}, expected (B={B}, H_kv, N_kv, d={d})")
    Hkv, Nk = k.shape[1], k.shape[2]
    _need(Hkv > 0 and Hq % Hkv == 0, f"H_q={Hq} must be a multiple of H_kv={Hkv}")
    _like(q, "q", (B, Hq, N, d), e4)
    _like(k, "k", (B, Hkv, Nk, d), e4)
    _like(v, "v", (B, Hkv, Nk, d), e4)
    for i, x in enumerate((lts, lte, uts, ute)):
        _like(x, f"mask vector {i}", (B, Nk), torch.int32)
    if o is not None:
        _like(o, "o", (B, Hq, N, d), torch.bfloat16)
    if lse is not None:
        _like(lse, "lse", (B, Hq, N), torch.float32)
    _need(isinstance(queues, TileQueues) and (queues.block_m, queues.block_n) == attn_tiling(),
          "queues must come from fm_classify_tiles with the attention tiling")
    nq = -(-N // queues.block_m)
    _like(queues.q_off, "queue offsets", (B * nq + 1,), torch.int32)
    _same_cuda(q=q, k=k, v=v, o=o, lse=lse, ws=ws, queue_offsets=queues.q_off, queue=queues.q_queue,
               **{f"mask vector {i}": x for i, x in enumerate((lts, lte, uts, ute))})
    prob = _problem(B, Hq, Hkv, N, d, scale, causal, Nk)
    o = torch.empty((B, Hq, N, d), dtype=torch.bfloat16, device=q.device) if o is None else o
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if lse is None else lse
    wsb = lib().fm_attn_fwd_workspace_bytes(ctypes.byref(prob))
    if ws is None or ws.numel() < wsb:
        ws = torch.empty(max(1, wsb), dtype=torch.uint8, device=q.device)
    _check(lib().fm_attn_fwd_fp8(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), float(q_scale), float(k_scale),
                                 float(v_scale), _ptr(lts), _ptr(lte), _ptr(uts), _ptr(ute), _ptr(queues.q_off),
                                 _ptr(queues.q_queue), _ptr(o), _ptr(lse), _ptr(ws), ctypes.c_size_t(wsb),
                                 _stream(stream)), "fm_attn_fwd_fp8")
    return o, lse


def fm_attn_bwd(q, k, v, o, lse, do, lts, lte, uts, ute, queues: TileQueues, *, scale: float, causal: bool,
                dq=None, dk=None, dv=None, ws=None, stream=None):
    """Backward: returns (dQ, dK, dV) bf16."""
    _attn_args(q, k, v, (lts, lte, uts, ute), queues, backward=True, o=o, lse=lse, do=do, dq=dq, dk=dk, dv=dv,
               ws=ws)
    B, Hq, N, d = q.shape
    prob = _problem(B, Hq, k.shape[1], N, d, scale, causal, k.shape[2])
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    wsb = lib().fm_attn_bwd_workspace_bytes(ctypes.byref(prob))
    if ws is None or ws.numel() < wsb:
        ws = torch.empty(max(1, wsb), dtype=torch.uint8, device=q.device)
    _check(lib().fm_attn_bwd(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(lts),
                             _ptr(lte), _ptr(uts), _ptr(ute), _ptr(queues.k_off), _ptr(queues.k_queue), _ptr(dq),
                             _ptr(dk), _ptr(dv), _ptr(ws), ctypes.c_size_t(wsb), _stream(stream)), "fm_attn_bwd")
    return dq, dk, dv


def fm_attn_fwd_bwd_host(q, k, v, do, lts, lte, uts, ute, *, scale: float, causal: bool, o=None, lse=None,
                         dq=None, dk=None, dv=None, ws=None, stream=None):
    """Forward + backward from HOST tensors (page-locked for asynchronous copies):
    the library copies the inputs to its device workspace `ws` (a CUDA uint8
    tensor of fm_attn_host_workspace_bytes bytes, allocated here if None),
    classifies, runs forward and backward, and copies O, LSE, dQ, dK, dV back
    into host tensors, all enqueued on `stream`. Returns (o, lse, dq, dk, dv)
    without waiting: synchronize the stream before reading them."""
    _need(isinstance(q, torch.Tensor) and q.dim() == 4, "q must be a (B, H_q, N, d) tensor")
    B, Hq, N, d = q.shape
    _need(isinstance(k, torch.Tensor) and k.dim() == 4 and k.shape[0] == B and k.shape[3] == d,
          f"k has shape {tuple(k.shape)}, expected (B={B}, H_kv, N_kv, d={d})")
    Hkv, Nk = k.shape[1], k.shape[2]
    bf = torch.bfloat16
    for name, t, shape, dt in (("q", q, (B, Hq, N, d), bf), ("k", k, (B, Hkv, Nk, d), bf), ("v", v, (B, Hkv, Nk, d), bf),
                               ("do", do, (B, Hq, N, d), bf)):
        _like(t, name, shape, dt)
    for i, x in enumerate((lts, lte, uts, ute)):
        _like(x, f"mask vector {i}", (B, Nk), torch.int32)
    host = dict(q=q, k=k, v=v, do=do, lts=lts, lte=lte, uts=uts, ute=ute)
    o = torch.empty((B, Hq, N, d), dtype=bf, pin_memory=True) if o is None else o
    lse = torch.empty((B, Hq, N), dtype=torch.float32, pin_memory=True) if lse is None else lse
    dq = torch.empty((B, Hq, N, d), dtype=bf, pin_memory=True) if dq is None else dq
    dk = torch.empty((B, Hkv, Nk, d), dtype=bf, pin_memory=True) if dk is None else dk
    dv = torch.empty((B, Hkv, Nk, d), dtype=bf, pin_memory=True) if dv is None else dv
    for name, t, shape, dt in (("o", o, (B, Hq, N, d), bf), ("lse", lse, (B, Hq, N), torch.float32),
                               ("dq", dq, (B, Hq, N, d), bf), ("dk", dk, (B, Hkv, Nk, d), bf),
                               ("dv", dv, (B, Hkv, Nk, d), bf)):
        _like(t, name, shape, dt)
        host[name] = t
    for name, t in host.items():
        _need(not t.is_cuda, f"{name} must be a host tensor for the host-buffer entry point")
    prob = _problem(B, Hq, Hkv, N, d, scale, causal, Nk)
    wsb = lib().fm_attn_host_workspace_bytes(ctypes.byref(prob))
    if ws is None:
        ws = torch.empty(max(1, wsb), dtype=torch.uint8, device="cuda")
    _need(isinstance(ws, torch.Tensor) and ws.is_cuda and ws.dtype == torch.uint8 and ws.numel() >= wsb,
          f"ws must be a CUDA uint8 tensor of at least {wsb} bytes")
    _check(lib().fm_attn_fwd_bwd_host(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(lts), _ptr(lte),
                                      _ptr(uts), _ptr(ute), _ptr(o), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                                      _ptr(ws), ctypes.c_size_t(wsb), _stream(stream)), "fm_attn_fwd_bwd_host")
    return o, lse, dq, dk, dv


def fm_localize(x, chunk_off, C: int, out=None, stream=None):
    """Rank-local boundaries of any int32 boundary values x for chunks at chunk_off (ascending)."""
    _like(x, "x", x.shape, torch.int32)
    _need(chunk_off.dim() == 1, "chunk_off must be one-dimensional")
    _like(chunk_off, "chunk_off", chunk_off.shape, torch.int32)
    if out is not None:
        _like(out, "out", x.shape, torch.int32)
    _same_cuda(x=x, chunk_off=chunk_off, out=out)
    out = torch.empty_like(x) if out is None else out
    _check(lib().fm_localize(_ptr(x), ctypes.c_int64(x.numel()), _ptr(chunk_off), int(chunk_off.numel()), int(C),
                             _ptr(out), _stream(stream)), "fm_localize")
    return out


def fm_from_fms_fme(fms, fme, n_rows=None, stream=None):
    """(lts, lte, uts, ute) for the FlashMask Guide's inclusive visible intervals
    [FMS_j, FME_j] (int32 CUDA tensors of one shape, e.g. (B, N_kv)); use the
    result with causal=False. n_rows: query rows N (default: the last dimension)."""
    _need(isinstance(fms, torch.Tensor) and isinstance(fme, torch.Tensor) and fms.shape == fme.shape,
          "fms and fme must be tensors of the same shape")
    _need(fms.dtype == torch.int32 and fme.dtype == torch.int32, "fms and fme must be int32")
    _same_cuda(fms=fms, fme=fme)
    fms, fme = fms.contiguous(), fme.contiguous()
    n = fms.shape[-1] if n_rows is None else int(n_rows)
    out = [torch.empty_like(fms) for _ in range(4)]
    _check(lib().fm_from_fms_fme(_ptr(fms), _ptr(fme), ctypes.c_int64(fms.numel()), n, *(_ptr(x) for x in out),
                                 _stream(stream)), "fm_from_fms_fme")
    return tuple(out)


def _ptr_array(ts):
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def fm_merge_parts(o_parts, lse_parts, o=None, lse=None, stream=None):
    """Log-sum-exp merge of M partial attentions (bf16 O_m, fp32 LSE_m of one shape each)."""
    _need(len(o_parts) == len(lse_parts) and len(o_parts) > 0, "one LSE per O part")
    oshape = tuple(o_parts[0].shape)
    _need(len(oshape) >= 1, "O parts must have a head dimension")
    for i, t in enumerate(o_parts):
        _like(t, f"O part {i}", oshape, torch.bfloat16)
    for i, t in enumerate(lse_parts):
        _like(t, f"LSE part {i}", oshape[:-1], torch.float32)
    if o is not None:
        _like(o, "o", oshape, torch.bfloat16)
    if lse is not None:
        _like(lse, "lse", oshape[:-1], torch.float32)
    _same_cuda(o=o, lse=lse, **{f"O part {i}": t for i, t in enumerate(o_parts)},
               **{f"LSE part {i}": t for i, t in enumerate(lse_parts)})
    o = torch.empty_like(o_parts[0]) if o is None else o
    lse = torch.empty_like(lse_parts[0]) if lse is None else lse
    d = oshape[-1]
    _check(lib().fm_merge_parts(len(o_parts), _ptr_array(o_parts), _ptr_array(lse_parts),
                                ctypes.c_int64(lse_parts[0].numel()), d, _ptr(o), _ptr(lse), _stream(stream)),
           "fm_merge_parts")
    return o, lse


def fm_sum_parts(parts, out=None, stream=None):
    """Elementwise sum of bf16 tensors of one shape (fp32 accumulation, one rounding)."""
    _need(len(parts) > 0, "at least one part")
    shape = tuple(parts[0].shape)
    for i, t in enumerate(parts):
        _like(t, f"part {i}", shape, torch.bfloat16)
    if out is not None:
        _like(out, "out", shape, torch.bfloat16)
    _same_cuda(out=out, **{f"part {i}": t for i, t in enumerate(parts)})
    out = torch.empty_like(parts[0]) if out is None else out
    _check(lib().fm_sum_parts(len(parts), _ptr_array(parts), ctypes.c_int64(parts[0].numel()), _ptr(out),
                              _stream(stream)), "fm_sum_parts")
    return out


def fm_classify_tiles_multi(fms, fme, *, causal: bool, n_rows=None, block_m: int = 128, block_n: int = 128,
                            stream=None):
    """Tile classes and queues of a multi-interval mask: fms, fme are
    (M, B, N_kv) int32 CUDA tensors (M <= 4), key j visible to rows
    [fms[m, b, j], fme[m, b, j]] for some m. Each column's visible rows are
    taken as their maximal runs (overlapping or touching intervals joined) and
    every tile gets the most visible of the runs' own classes; the queues have
    the layout of fm_classify_tiles for B batch entries."""
    _need(isinstance(fms, torch.Tensor) and fms.dim() == 3, "fms, fme must be (M, B, N_kv)")
    M, B, Nk = fms.shape
    for i, x in enumerate((fms, fme)):
        _like(x, ("fms", "fme")[i], (M, B, Nk), torch.int32)
    _same_cuda(fms=fms, fme=fme)
    N = Nk if n_rows is None else int(n_rows)
    prob = _problem(B, 1, 1, N, 128, 1.0, causal, Nk)
    til = fm_tiling(block_m, block_n)
    nq, nk = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().fm_tile_counts(ctypes.byref(prob), ctypes.byref(til), ctypes.byref(nq), ctypes.byref(nk)),
           "fm_tile_counts")
    nq, nk = nq.value, nk.value
    dev = fms.device
    cap = max(1, B * nq * nk)
    cls = torch.empty((B, nq, nk), dtype=torch.uint8, device=dev)
    q_off = torch.empty(B * nq + 1, dtype=torch.int32, device=dev)
    k_off = torch.empty(B * nk + 1, dtype=torch.int32, device=dev)
    q_queue = torch.empty(cap, dtype=torch.int32, device=dev)
    k_queue = torch.empty(cap, dtype=torch.int32, device=dev)
    wsb = lib().fm_classify_multi_workspace_bytes(ctypes.byref(prob), ctypes.byref(til), M)
    ws = torch.empty(max(1, wsb), dtype=torch.uint8, device=dev)
    _check(lib().fm_classify_tiles_multi(ctypes.byref(prob), ctypes.byref(til), M, _ptr(fms), _ptr(fme), _ptr(cls),
                                         _ptr(q_off), _ptr(q_queue), _ptr(k_off), _ptr(k_queue), _ptr(ws),
                                         ctypes.c_size_t(wsb), _stream(stream)), "fm_classify_tiles_multi")
    return TileQueues(cls, q_off, q_queue, k_off, k_queue, block_m, block_n)


def _multi_args(fms, fme):
    _need(isinstance(fms, torch.Tensor) and fms.dim() == 3, "multi-interval fms, fme must be (M, B, N_kv)")
    _need(isinstance(fme, torch.Tensor) and fme.shape == fms.shape, "fms and fme must have one shape")
    return fms.shape[0]


def fm_attn_fwd_multi(q, k, v, fms, fme, queues: TileQueues, *, scale: float, causal: bool, o=None, lse=None,
                      ws=None, stream=None):
    """Forward with a multi-interval mask (fms, fme (M, B, N_kv)) and the
    queues of fm_classify_tiles_multi. Returns (O bf16, LSE fp32)."""
    M = _multi_args(fms, fme)
    _attn_args(q, k, v, (fms, fme), queues, backward=False, o=o, lse=lse, ws=ws, intervals=M)
    B, Hq, N, d = q.shape
    prob = _problem(B, Hq, k.shape[1], N, d, scale, causal, k.shape[2])
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if lse is None else lse
    wsb = lib().fm_attn_fwd_workspace_bytes(ctypes.byref(prob))
    if ws is None or ws.numel() < wsb:
        ws = torch.empty(max(1, wsb), dtype=torch.uint8, device=q.device)
    _check(lib().fm_attn_fwd_multi(ctypes.byref(prob), M, _ptr(q), _ptr(k), _ptr(v), _ptr(fms), _ptr(fme),
                                   _ptr(queues.q_off), _ptr(queues.q_queue), _ptr(o), _ptr(lse), _ptr(ws),
                                   ctypes.c_size_t(wsb), _stream(stream)), "fm_attn_fwd_multi")
    return o, lse


def fm_attn_bwd_multi(q, k, v, o, lse, do, fms, fme, queues: TileQueues, *, scale: float, causal: bool, dq=None,
                      dk=None, dv=None, ws=None, stream=None):
    """Backward with a multi-interval mask (fms, fme (M, B, N_kv)): returns
    (dQ, dK, dV) bf16."""
    M = _multi_args(fms, fme)
    _attn_args(q, k, v, (fms, fme), queues, backward=True, o=o, lse=lse, do=do, dq=dq, dk=dk, dv=dv, ws=ws,
               intervals=M)
    B, Hq, N, d = q.shape
    prob = _problem(B, Hq, k.shape[1], N, d, scale, causal, k.shape[2])
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    wsb = lib().fm_attn_bwd_workspace_bytes(ctypes.byref(prob))
    if ws is None or ws.numel() < wsb:
        ws = torch.empty(max(1, wsb), dtype=torch.uint8, device=q.device)
    _check(lib().fm_attn_bwd_multi(ctypes.byref(prob), M, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                                   _ptr(fms), _ptr(fme), _ptr(queues.k_off), _ptr(queues.k_queue), _ptr(dq),
                                   _ptr(dk), _ptr(dv), _ptr(ws), ctypes.c_size_t(wsb), _stream(stream)),
           "fm_attn_bwd_multi")
    return dq, dk, dv


def fm_attn_multi_interval(q, k, v, fms, fme, *, scale: float, do=None, causal: bool = False, stream=None):
    """Attention under a multi-interval mask: fms, fme are (M, B, N_kv) int32
    CUDA tensors (M <= 4), key j visible to rows [fms[m, b, j], fme[m, b, j]]
    (inclusive) for some m (intervals may overlap), and to no row before j
    when causal. Library calls only: fm_classify_tiles_multi, then
    fm_attn_fwd_multi and, with do, fm_attn_bwd_multi (each block computed
    once, masked by the union of the intervals).
    Returns (o, lse) or (o, lse, dq, dk, dv)."""
    qs = fm_classify_tiles_multi(fms, fme, causal=causal, n_rows=q.shape[2], stream=stream)
    o, lse = fm_attn_fwd_multi(q, k, v, fms, fme, qs, scale=scale, causal=causal, stream=stream)
    if do is None:
        return o, lse
    dq, dk, dv = fm_attn_bwd_multi(q, k, v, o, lse, do, fms, fme, qs, scale=scale, causal=causal, stream=stream)
    return o, lse, dq, dk, dv


def fm_classify_tiles_heads(lts, lte, uts, ute, *, causal: bool, n_rows=None, stream=None):
    """Queues for per-head mask vectors (B, H_q, N_kv): fm_classify_tiles over
    the B * H_q rows, row b * H_q + h holding query head h of batch entry b."""
    _need(isinstance(lts, torch.Tensor) and lts.dim() == 3, "per-head mask vectors must be (B, H_q, N_kv)")
    B, Hq, Nk = lts.shape
    for i, x in enumerate((lts, lte, uts, ute)):
        _like(x, f"mask vector {i}", (B, Hq, Nk), torch.int32)
    return fm_classify_tiles(*(x.view(B * Hq, Nk) for x in (lts, lte, uts, ute)), causal=causal, n_rows=n_rows,
                             stream=stream)


def fm_attn_fwd_heads(q, k, v, lts, lte, uts, ute, queues: TileQueues, *, scale: float, causal: bool, o=None,
                      lse=None, ws=None, stream=None):
    """Forward with per-head mask vectors (B, H_q, N_kv) and the queues of
    fm_classify_tiles_heads: returns (O bf16, LSE fp32)."""
    _attn_args(q, k, v, (lts, lte, uts, ute), queues, backward=False, o=o, lse=lse, ws=ws, heads=True)
    B, Hq, N, d = q.shape
    prob = _problem(B, Hq, k.shape[1], N, d, scale, causal, k.shape[2])
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device) if lse is None else lse
    wsb = lib().fm_attn_fwd_heads_workspace_bytes(ctypes.byref(prob))
    if ws is None or ws.numel() < wsb:
        ws = torch.empty(max(1, wsb), dtype=torch.uint8, device=q.device)
    _check(lib().fm_attn_fwd_heads(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(lts), _ptr(lte), _ptr(uts),
                                   _ptr(ute), _ptr(queues.q_off), _ptr(queues.q_queue), _ptr(o), _ptr(lse),
                                   _ptr(ws), ctypes.c_size_t(wsb), _stream(stream)), "fm_attn_fwd_heads")
    return o, lse


def fm_attn_bwd_heads(q, k, v, o, lse, do, lts, lte, uts, ute, queues: TileQueues, *, scale: float, causal: bool,
                      dq=None, dk=None, dv=None, ws=None, stream=None):
    """Backward with per-head mask vectors: returns (dQ, dK, dV) bf16."""
    _attn_args(q, k, v, (lts, lte, uts, ute), queues, backward=True, o=o, lse=lse, do=do, dq=dq, dk=dk, dv=dv,
               ws=ws, heads=True)
    B, Hq, N, d = q.shape
    prob = _problem(B, Hq, k.shape[1], N, d, scale, causal, k.shape[2])
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    wsb = lib().fm_attn_bwd_workspace_bytes(ctypes.byref(prob))
    if ws is None or ws.numel() < wsb:
        ws = torch.empty(max(1, wsb), dtype=torch.uint8, device=q.device)
    _check(lib().fm_attn_bwd_heads(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                                   _ptr(lts), _ptr(lte), _ptr(uts), _ptr(ute), _ptr(queues.k_off),
                                   _ptr(queues.k_queue), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                                   ctypes.c_size_t(wsb), _stream(stream)), "fm_attn_bwd_heads")
    return dq, dk, dv


def fm_attn_per_head(q, k, v, lts, lte, uts, ute, *, causal: bool, scale: float, do=None, stream=None):
    """Attention with one set of mask vectors per query head: lts..ute are
    (B, H_q, N_kv) int32 CUDA tensors. One classification over the B * H_q
    vector rows, one forward and (with do) one backward, each a single launch
    over every head. Returns (o, lse) or (o, lse, dq, dk, dv)."""
    qs = fm_classify_tiles_heads(lts, lte, uts, ute, causal=causal, n_rows=q.shape[2] if q.dim() == 4 else None,
                                 stream=stream)
    o, lse = fm_attn_fwd_heads(q, k, v, lts, lte, uts, ute, qs, scale=scale, causal=causal, stream=stream)
    if do is None:
        return o, lse
    dq, dk, dv = fm_attn_bwd_heads(q, k, v, o, lse, do, lts, lte, uts, ute, qs, scale=scale, causal=causal,
                                   stream=stream)
    return o, lse, dq, dk, dv


def fm_device_status(stream=None):
    """(status, bits) of the device error word; synchronizes the stream and clears the word."""
    bits = ctypes.c_int32(0)
    st = lib().fm_device_status(_stream(stream), ctypes.byref(bits))
    return st, bits.value


def fm_selftest_wait_timeout(limit_us: int, stream=None):
    _check(lib().fm_selftest_wait_timeout(ctypes.c_int64(limit_us), _stream(stream)), "fm_selftest_wait_timeout")


def fm_profile_enable(on: bool):
    _check(lib().fm_profile_enable(1 if on else 0), "fm_profile_enable")


def fm_profile_read():
    """{'fwd_ms', 'fwd_launches', 'bwd_ms', 'bwd_launches'} since the last read (synchronizes)."""
    fm_, fl, bm_, bl = ctypes.c_double(), ctypes.c_int32(), ctypes.c_double(), ctypes.c_int32()
    _check(lib().fm_profile_read(ctypes.byref(fm_), ctypes.byref(fl), ctypes.byref(bm_), ctypes.byref(bl)),
           "fm_profile_read")
    return dict(fwd_ms=fm_.value, fwd_launches=fl.value, bwd_ms=bm_.value, bwd_launches=bl.value)


def fm_launch_count() -> int:
    return int(lib().fm_launch_count())


def _host_array(x, dtype):
    """A contiguous host numpy array of `dtype` holding x (numpy array or torch tensor, any device)."""
    if isinstance(x, torch.Tensor):
        x = x.detach().cpu().numpy()
    a = np.ascontiguousarray(x)
    if a.dtype != dtype:
        raise ValueError(f"expected {np.dtype(dtype).name} values, got {a.dtype}")
    return a


def fm_chunk_loads(tile_class, blocks_per_chunk: int, cost_partial: int, cost_unmasked: int) -> np.ndarray:
    """Per-chunk loads (int64) from the (B, nQ, nK) tile classes (copied to the host if on a GPU)."""
    cls = _host_array(tile_class, np.uint8)
    if cls.ndim != 3:
        raise ValueError("tile_class must be (B, nQ, nK)")
    B, nq, nk = cls.shape
    w = np.empty(-(-nq // int(blocks_per_chunk)) if blocks_per_chunk > 0 else 0, dtype=np.int64)
    _check(lib().fm_chunk_loads(ctypes.c_void_p(cls.ctypes.data), B, nq, nk, int(blocks_per_chunk),
                                int(cost_partial), int(cost_unmasked), ctypes.c_void_p(w.ctypes.data)),
           "fm_chunk_loads")
    return w


def fm_needed_chunks(tile_class, owner, P: int, blocks_per_chunk: int) -> np.ndarray:
    """(P, n_chunks) uint8: 1 where rank r's rows can see some key of chunk c."""
    cls = _host_array(tile_class, np.uint8)
    own = _host_array(np.asarray(owner, dtype=np.int32) if not isinstance(owner, torch.Tensor) else owner, np.int32)
    if cls.ndim != 3:
        raise ValueError("tile_class must be (B, nQ, nK)")
    B, nq, nk = cls.shape
    need = np.empty((int(P), own.size), dtype=np.uint8)
    _check(lib().fm_needed_chunks(ctypes.c_void_p(cls.ctypes.data), B, nq, nk, ctypes.c_void_p(own.ctypes.data),
                                  own.size, int(P), int(blocks_per_chunk), ctypes.c_void_p(need.ctypes.data)),
           "fm_needed_chunks")
    return need


def fm_balance_chunks(w, P: int, kappa: int, phases: int = 3, node_budget: int = 0):
    """HCC-IPO Stage 1 on chunk loads w: returns (owner int32 array, report dict)."""
    wa = _host_array(w, np.int64)
    owner = np.empty(wa.size, dtype=np.int32)
    rep = fm_balance_report()
    _check(lib().fm_balance_chunks(ctypes.c_void_p(wa.ctypes.data), int(wa.size), int(P), int(kappa), int(phases),
                                   int(node_budget), ctypes.c_void_p(owner.ctypes.data), ctypes.byref(rep)),
           "fm_balance_chunks")
    return owner, {name: int(getattr(rep, name)) for name, _ in fm_balance_report._fields_}


# ------------------------------------------------ norm, rotation, paged cache
# These calls are made many times a token, on tensors whose kernels take a few
# microseconds, so their checks are plain comparisons (messages are built only
# on failure) and their structures are packed bytes, passed by address. All of them
# take a keyword `stream`.
_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_pack_view, _pack_rows = struct.Struct("=Qqqq").pack, struct.Struct("=Qqq").pack  # fm_view, fm_rows
_pack_qk = struct.Struct("=8i2fQqQQQ").pack  # fm_qk_problem
_fast = {}


def _fast_fn(name):
    """A library function that takes every pointer as an address or packed bytes."""
    f = _fast.get(name)
    if f is None:
        f = lib()[name]  # a function object of its own
        res, args = _SIGS[name]
        simple = (ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float)
        f.restype, f.argtypes = res, [t if t in simple else _P for t in args]
        _fast[name] = f
    return f


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_given = threading.local()  # .stream: the running call was given one


def _enqueue(name, dev, *args):
    """Call a library function whose last argument is the stream: the current stream
    of device `dev` (an index), with that device current."""
    if dev < 0:
        raise ValueError("the tensors must be CUDA tensors: the library computes on the GPU only")
    if dev != torch.cuda.current_device():
        if getattr(_given, "stream", False):
            raise ValueError("stream belongs to another device than the tensors")
        with torch.cuda.device(dev):
            return _enqueue(name, dev, *args)
    s = _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    st = _fast_fn(name)(*args, s)
    if st != FM_OK:
        raise FMError(st, name)


def _streamed(f):
    """f with a `stream` argument: everything it does, new tensors and workspaces
    included, belongs to that stream (None: the current one)."""

    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            _given.stream = True
            try:
                return f(*args, **kw)
            finally:
                _given.stream = False

    return call


def _tensor(t, name, dims):
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"{name} must be a torch tensor of {dims} dimensions")


def _expect(t, name, shape, dtype, dev):
    """t is a contiguous tensor of this shape, dtype and device."""
    if (type(t) is torch.Tensor and t.shape == shape and t.dtype is dtype and t.get_device() == dev
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        _like(t, name, shape, dtype)  # raises, saying which
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device than the other tensors")


def _bf16_rows(t, name, shape, dev):
    """Address and element strides of a bf16 tensor whose rows (last dimension) are
    read in 16-byte pieces; 0 for the stride of a dimension of size 1."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != _BF16:
        _need(isinstance(t, torch.Tensor), f"{name} must be a torch tensor")
        _need(t.shape == shape, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    at, st, bits = t.data_ptr(), list(t.stride()), 0
    for i in range(len(st) - 1):
        if shape[i] == 1:
            st[i] = 0
        bits |= st[i]
    if at & 15 or bits & 7 or st[-1] != 1:
        raise ValueError(f"{name}: rows must be contiguous and start on 16-byte boundaries (strides {t.stride()})")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device than the other tensors")
    return at, st


def _view(t, name, shape, dev, out=False):
    """fm_view of a bf16 (B, H, N, d) tensor."""
    if type(t) is torch.Tensor and t.shape == shape and t.dtype is _BF16 and t.get_device() == dev:
        at, (sb, sh, sn, one) = t.data_ptr(), t.stride()
        if one == 1 and not (at & 15 or (sb | sh | sn) & 7) and (sb and sh and sn or not out):
            return _pack_view(at, sb, sh, sn)  # nothing to look at more closely
    at, (sb, sh, sn, _) = _bf16_rows(t, name, shape, dev)
    if out and not ((sb or shape[0] <= 1) and (sh or shape[1] <= 1) and (sn or shape[2] <= 1)):
        raise ValueError(f"{name}: an output cannot be a broadcast view")
    return _pack_view(at, sb, sh, sn)


def _new_view(shape, device):
    """A new contiguous bf16 (B, H, N, d) tensor and its fm_view."""
    t = torch.empty(shape, dtype=_BF16, device=device)
    _, H, N, d = shape
    return t, _pack_view(t.data_ptr(), H * N * d, N * d, d)


def _new_token_view(shape, device):
    """The same, laid out (B, N, H, d)."""
    _, H, N, d = shape
    t = torch.empty_strided(shape, (H * N * d, d, H * d, 1), dtype=_BF16, device=device)
    return t, _pack_view(t.data_ptr(), H * N * d, d, H * d)


def _rows(t, name, shape, dev, out=False):
    """fm_rows of a bf16 (T, H, d) tensor."""
    if type(t) is torch.Tensor and t.shape == shape and t.dtype is _BF16 and t.get_device() == dev:
        at, (st, sh, one) = t.data_ptr(), t.stride()
        if one == 1 and not (at & 15 or (st | sh) & 7) and (st and sh or not out):
            return _pack_rows(at, st, sh)
    at, (st, sh, _) = _bf16_rows(t, name, shape, dev)
    if out and not ((st or shape[0] <= 1) and (sh or shape[1] <= 1)):
        raise ValueError(f"{name}: an output cannot be a broadcast view")
    return _pack_rows(at, st, sh)


_ROPE_KINDS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}


def fm_rope_freqs(rot: int, *, base: float = 10000.0, kind: str = "plain", factor: float = 1.0, orig_len: int = 0,
                  beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """(inv_freq fp32 (rot / 2,), rot_scale): a rotation's inverse frequencies and
    the factor of its cos and sin. kind: "plain", or for contexts `factor` times
    longer than the trained ones "linear", "ntk" or "yarn" (orig_len: the trained length)."""
    _need(kind in _ROPE_KINDS, f"kind must be one of {sorted(_ROPE_KINDS)}, got {kind!r}")
    _need(int(rot) <= _MOST and int(orig_len) <= 1 << 62, f"rot={rot} or orig_len={orig_len} is too large")
    f = np.empty(max(1, int(rot) // 2), dtype=np.float32)
    sc = ctypes.c_float()
    _check(lib().fm_rope_freqs(int(rot), float(base), _ROPE_KINDS[kind], float(factor), int(orig_len),
                               float(beta_fast), float(beta_slow), f.ctypes.data, ctypes.byref(sc)), "fm_rope_freqs")
    return torch.from_numpy(f).to("cpu" if device is None else device), sc.value


def _norm_weights(q_weight, k_weight, d, dev):
    """Addresses of the norms' weights (0: no norm), and whether they are fp32."""
    w, f32 = [0, 0], 0
    for i, t in enumerate((q_weight, k_weight)):
        if t is not None:
            name = "k_weight" if i else "q_weight"
            if not isinstance(t, torch.Tensor) or t.dtype not in (_F32, _BF16):
                raise ValueError(f"{name} must be a float32 or bfloat16 tensor")
            _expect(t, name, (d,), t.dtype, dev)
            w[i], f32 = t.data_ptr(), 1 if t.dtype == _F32 else 0
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise ValueError("q_weight and k_weight must have one dtype")
    return w, f32


def _qk_args(q, k, positions, inv_freq, interleaved, rot_scale, q_weight, k_weight, eps):
    """The packed problem of a norm-and-rotation call, its shapes, dtypes and devices checked."""
    _tensor(q, "q", 4)
    _tensor(k, "k", 4)
    B, Hq, N, d = q.shape
    Hkv, dev = k.shape[1], q.get_device()
    if k.shape != (B, Hkv, N, d):
        raise ValueError(f"k has shape {tuple(k.shape)}, expected (B={B}, H_kv, N={N}, d={d})")
    rot = pos = sb = fr = 0
    if inv_freq is not None:
        _tensor(inv_freq, "inv_freq", 1)
        _expect(inv_freq, "inv_freq", inv_freq.shape, _F32, dev)
        if not isinstance(positions, torch.Tensor) or positions.shape not in ((N,), (B, N)):
            raise ValueError(f"positions must be an int32 tensor of shape (N={N},) or (B={B}, N={N})")
        _expect(positions, "positions", positions.shape, _I32, dev)
        rot, pos, fr = 2 * inv_freq.shape[0], positions.data_ptr(), inv_freq.data_ptr()
        sb = N if positions.dim() == 2 else 0
    w, f32 = _norm_weights(q_weight, k_weight, d, dev)
    return _pack_qk(B, N, Hq, Hkv, d, rot, 1 if interleaved else 0, f32, eps, rot_scale, pos, sb, fr, *w), dev


@_streamed
def fm_qk_norm_rope(q, k, v=None, *, positions=None, inv_freq=None, interleaved: bool = False, rot_scale: float = 1.0,
                    q_weight=None, k_weight=None, eps: float = 1e-6, out=None):
    """Per-head norm and rotation of queries and keys in one pass: q (B, H_q, N, d),
    k, v (B, H_kv, N, d) bf16 views of any strides (rows contiguous), e.g. of a
    fused projection's output, to (q', k') or (q', k', v') contiguous (B, H, N, d),
    or into the tensors `out` (views of any strides; an input itself is allowed).
    positions: int32 (N,) or (B, N); inv_freq: fp32 (rot / 2,), None: no rotation;
    q_weight / k_weight: (d,), None: no norm."""
    p, dev = _qk_args(q, k, positions, inv_freq, interleaved, rot_scale, q_weight, k_weight, eps)
    qs, ks = q.shape, k.shape
    qi, ki = _view(q, "q", qs, dev), _view(k, "k", ks, dev)
    vi = None if v is None else _view(v, "v", ks, dev)
    if dev < 0:
        raise ValueError("q must be a CUDA tensor: the library computes on the GPU only")
    if out is None:
        on = q.device
        (qo, qv), (ko, kv) = _new_view(qs, on), _new_view(ks, on)
        out, vv = (qo, ko), None
        if v is not None:
            vo, vv = _new_view(ks, on)
            out = (qo, ko, vo)
    else:
        if len(out) != (2 if v is None else 3):
            raise ValueError("out must hold one tensor per input")
        qv, kv = _view(out[0], "output q", qs, dev, True), _view(out[1], "output k", ks, dev, True)
        vv = None if v is None else _view(out[2], "output v", ks, dev, True)
        out = tuple(out)
    _enqueue("fm_qk_norm_rope", dev, p, qi, ki, vi, qv, kv, vv)
    return out


@functools.lru_cache(maxsize=256)
def _qk_bwd_bytes(dev, *sizes):
    """Workspace of a backward pass with normed sides: it goes by the sizes (B, N, H_q, H_kv, d) alone."""
    with torch.cuda.device(dev):
        return lib().fm_qk_norm_rope_bwd_workspace_bytes(fm_qk_problem(*sizes, q_weight=16, k_weight=16))


@_streamed
def fm_qk_norm_rope_bwd(dqo, dko, dvo, q, k, *, positions=None, inv_freq=None, interleaved: bool = False,
                        rot_scale: float = 1.0, q_weight=None, k_weight=None, eps: float = 1e-6, out=None):
    """Backward of fm_qk_norm_rope: the gradients dqo, dko, dvo (or None) of its
    outputs and its inputs q, k give (dq, dk, dv, dq_weight, dk_weight); None
    where there is no such input. dq, dk, dv are (B, H, N, d) views of contiguous
    (B, N, H, d) tensors (a projection's own layout), or the views `out` (dq, dk[, dv])."""
    p, dev = _qk_args(q, k, positions, inv_freq, interleaved, rot_scale, q_weight, k_weight, eps)
    qs, ks = q.shape, k.shape
    gq, gk = _view(dqo, "dqo", qs, dev), _view(dko, "dko", ks, dev)
    gv = None if dvo is None else _view(dvo, "dvo", ks, dev)
    qi, ki = _view(q, "q", qs, dev), _view(k, "k", ks, dev)
    if dev < 0:
        raise ValueError("q must be a CUDA tensor: the library computes on the GPU only")
    on = q.device
    dv = vv = None
    if out is None:
        (dq, qv), (dk, kv) = _new_token_view(qs, on), _new_token_view(ks, on)
        if dvo is not None:
            dv, vv = _new_token_view(ks, on)
    else:
        if len(out) != (2 if dvo is None else 3):
            raise ValueError("out must hold one tensor per gradient")
        dq, dk = out[0], out[1]
        qv, kv = _view(dq, "output dq", qs, dev, True), _view(dk, "output dk", ks, dev, True)
        if dvo is not None:
            dv = out[2]
            vv = _view(dv, "output dv", ks, dev, True)
    dwq = None if q_weight is None else torch.empty_like(q_weight)
    dwk = None if k_weight is None else torch.empty_like(k_weight)
    ws, wsb = None, 0
    if dwq is not None or dwk is not None:
        wsb = _qk_bwd_bytes(dev, qs[0], qs[2], qs[1], ks[1], qs[3])
        ws = torch.empty(max(16, wsb), dtype=_U8, device=on)
    _enqueue("fm_qk_norm_rope_bwd", dev, p, gq, gk, gv, qi, ki, qv, kv, vv,
             None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(),
             None if ws is None else ws.data_ptr(), wsb)
    return dq, dk, dv, dwq, dwk


class KVCache:
    """The paged cache: k, v (n_pages, H_kv, page_size, d) bf16, or float8_e4m3fn with
    exponent bytes k_exp, v_exp (n_pages, H_kv, page_size) uint8 (value = stored *
    2^(exponent - 127)). Checked once; holds the tensors it was given."""

    __slots__ = ("k", "v", "k_exp", "v_exp", "n_pages", "H_kv", "page_size", "d", "device", "index", "c", "at")

    def __init__(self, k, v, k_exp=None, v_exp=None):
        _need(isinstance(k, torch.Tensor) and k.dim() == 4, "k must be (n_pages, H_kv, page_size, d)")
        _need((k_exp is None) == (v_exp is None), "k_exp and v_exp go together")
        dt = torch.bfloat16 if k_exp is None else torch.float8_e4m3fn
        _like(k, "k", k.shape, dt)
        _like(v, "v", k.shape, dt)
        if k_exp is not None:
            _like(k_exp, "k_exp", k.shape[:3], torch.uint8)
            _like(v_exp, "v_exp", k.shape[:3], torch.uint8)
        n, h, page, d = k.shape
        _need(n > 0 and h > 0, "a cache needs pages and heads")
        _need(page in (16, 32, 64, 128), f"page_size must be 16, 32, 64 or 128, got {page}")
        _need(d in (64, 128, 256), f"d must be 64, 128 or 256, got {d}")
        for name, t in (("k", k), ("v", v), ("k_exp", k_exp), ("v_exp", v_exp)):
            _need(t is None or t.data_ptr() & 15 == 0, f"{name} must start on a 16-byte boundary")
        _same_cuda(k=k, v=v, k_exp=k_exp, v_exp=v_exp)
        self.k, self.v, self.k_exp, self.v_exp, self.device, self.index = k, v, k_exp, v_exp, k.device, k.get_device()
        self.n_pages, self.H_kv, self.page_size, self.d = n, h, page, d
        self.c = fm_kv_cache(k.data_ptr(), v.data_ptr(), 0 if k_exp is None else k_exp.data_ptr(),
                             0 if v_exp is None else v_exp.data_ptr(), n, h, page, d)
        self.at = ctypes.addressof(self.c)


def fm_cache_new(n_pages: int, H_kv: int, page_size: int, d: int, *, dtype=torch.bfloat16, device="cuda") -> KVCache:
    """A cache of n_pages pages, its contents undefined. dtype: torch.bfloat16 or torch.float8_e4m3fn."""
    _need(dtype in (torch.bfloat16, torch.float8_e4m3fn), f"dtype must be bfloat16 or float8_e4m3fn, got {dtype}")
    shape = (n_pages, H_kv, page_size, d)
    kv = [torch.empty(shape, dtype=dtype, device=device) for _ in range(2)]
    ex = [None, None]
    if dtype == torch.float8_e4m3fn:
        ex = [torch.empty(shape[:3], dtype=torch.uint8, device=device) for _ in range(2)]
    return KVCache(*kv, *ex)


_MOST = 1 << 30  # counts are handed to the library as 32 bits, which keep the low ones of more


class PagedBatch:
    """A batch of R sequences over a cache, int32 CUDA tensors: q_off (R + 1,) first new
    token of each among a call's packed tokens, kv_len (R,) keys of each (new ones
    included), page_table (R, width) page of each page_size keys. Checked once; the
    tensors' values may change between calls (their addresses may not)."""

    __slots__ = ("q_off", "kv_len", "page_table", "R", "width", "index", "c", "at")

    def __init__(self, q_off, kv_len, page_table):
        _need(isinstance(page_table, torch.Tensor) and page_table.dim() == 2, "page_table must be (R, width)")
        R, width = page_table.shape
        _need(R > 0 and width > 0, "a batch needs sequences and pages")
        _need(R <= _MOST and width <= _MOST, f"a batch has at most 2^30 sequences and pages of each, got {R} and {width}")
        _like(page_table, "page_table", (R, width), torch.int32)
        _like(q_off, "q_off", (R + 1,), torch.int32)
        _like(kv_len, "kv_len", (R,), torch.int32)
        _same_cuda(q_off=q_off, kv_len=kv_len, page_table=page_table)
        self.q_off, self.kv_len, self.page_table, self.index = q_off, kv_len, page_table, q_off.get_device()
        self.R, self.width = R, width
        self.c = fm_paged_batch(q_off.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), R, width)
        self.at = ctypes.addressof(self.c)


def _serve_args(cache, batch):
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    if not isinstance(batch, PagedBatch):
        raise ValueError("batch must be a PagedBatch")
    if batch.index != cache.index:
        raise ValueError("the batch is on another device than the cache")
    return cache.index


@_streamed
def fm_cache_write(k, v, cache: KVCache, batch: PagedBatch):
    """Put the rows of T new tokens, k and v (T, H_kv, d) bf16 views, in their places
    in the cache (rounded to e4m3 with a scale a row where the cache is e4m3)."""
    dev = _serve_args(cache, batch)
    _tensor(k, "k", 3)
    shape = (k.shape[0], cache.H_kv, cache.d)
    if shape[0] > _MOST:
        raise ValueError(f"a call takes at most 2^30 tokens, got {shape[0]}")
    kr, vr = _rows(k, "k", shape, dev), _rows(v, "v", shape, dev)
    _enqueue("fm_cache_write", dev, cache.at, batch.at, shape[0], kr, vr)


@_streamed
def fm_cache_read(cache: KVCache, kv_off, page_table, n_rows: int, *, k=None, v=None):
    """Keys and values as packed bf16 rows (1, H_kv, n_rows, d): sequence r's keys from 0
    on become rows [kv_off[r], kv_off[r + 1]). kv_off (R + 1,) and page_table (R, width)
    int32, kv_off[R] at most n_rows. Rows that no sequence has are left as they were
    (undefined in new tensors)."""
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    dev = cache.index
    _tensor(page_table, "page_table", 2)
    R, width = page_table.shape
    _expect(page_table, "page_table", (R, width), _I32, dev)
    _expect(kv_off, "kv_off", (R + 1,), _I32, dev)
    shape = (1, cache.H_kv, int(n_rows), cache.d)
    if not (0 <= shape[2] <= _MOST and R <= _MOST and width <= _MOST):
        raise ValueError(f"n_rows must be in [0, 2^30], and so must the table's sizes, got {n_rows}, {R}, {width}")
    if k is None:
        k = torch.empty(shape, dtype=_BF16, device=cache.device)
    else:
        _expect(k, "k", shape, _BF16, dev)
    if v is None:
        v = torch.empty(shape, dtype=_BF16, device=cache.device)
    else:
        _expect(v, "v", shape, _BF16, dev)
    _enqueue("fm_cache_read", dev, cache.at, kv_off.data_ptr(), page_table.data_ptr(), R, width, shape[2],
             k.data_ptr(), v.data_ptr())
    return k, v


@_streamed
def fm_cache_append(q, k, v, cache: KVCache, batch: PagedBatch, *, positions=None, inv_freq=None,
                    interleaved: bool = False, rot_scale: float = 1.0, q_weight=None, k_weight=None, eps: float = 1e-6,
                    out=None):
    """fm_qk_norm_rope and fm_cache_write in one pass: T new tokens' q (T, H_q, d) and
    k, v (T, H_kv, d), bf16 views of any strides (rows contiguous), e.g. of a fused
    projection's output; keys and values go to their places in the cache, the queries
    to q' (T, H_q, d), or to `out` (a view; q itself is allowed). positions: int32 (T,),
    None: each token's position in its sequence; inv_freq: fp32 (rot / 2,), None: no
    rotation; q_weight / k_weight: (d,), None: no norm. Rows of tokens past q_off[R] are
    left as they were (undefined in a new tensor)."""
    dev = _serve_args(cache, batch)
    _tensor(q, "q", 3)
    T, Hq, d = shape = q.shape
    if d != cache.d:
        raise ValueError(f"q has d={d}, the cache d={cache.d}")
    if T > _MOST:
        raise ValueError(f"a call takes at most 2^30 tokens, got {T}")
    if not 0 < Hq <= 1 << 20:
        raise ValueError(f"H_q must be in [1, 2^20], got {Hq}")
    rot = pos = fr = 0
    if inv_freq is not None:
        _tensor(inv_freq, "inv_freq", 1)
        _expect(inv_freq, "inv_freq", inv_freq.shape, _F32, dev)
        rot, fr = 2 * inv_freq.shape[0], inv_freq.data_ptr()
    if positions is not None:
        _expect(positions, "positions", (T,), _I32, dev)
        pos = positions.data_ptr()
    w, f32 = _norm_weights(q_weight, k_weight, d, dev)
    p = _pack_qk(1, T, Hq, cache.H_kv, d, rot, 1 if interleaved else 0, f32, eps, rot_scale, pos, 0, fr, *w)
    kv = (T, cache.H_kv, d)
    qr, kr, vr = _rows(q, "q", shape, dev), _rows(k, "k", kv, dev), _rows(v, "v", kv, dev)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=cache.device)
        orow = _pack_rows(out.data_ptr(), Hq * d, d)
    else:
        orow = _rows(out, "out", shape, dev, True)
    _enqueue("fm_cache_append", dev, cache.at, batch.at, p, qr, kr, vr, orow)
    return out


@_streamed
def fm_cache_copy(cache: KVCache, src, dst):
    """Make page dst[i] a copy of page src[i] (int32 CUDA (n,); a pair of two -1 copies
    nothing). A page that is copied to may be in no other pair (pairs are copied in no order):
    pages that change places go by way of free ones."""
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    dev = cache.index
    _tensor(src, "src", 1)
    n = src.shape[0]
    if n > _MOST:
        raise ValueError(f"a call copies at most 2^30 pages, got {n}")
    _expect(src, "src", (n,), _I32, dev)
    _expect(dst, "dst", (n,), _I32, dev)
    _enqueue("fm_cache_copy", dev, cache.at, src.data_ptr(), dst.data_ptr(), n)


@functools.lru_cache(maxsize=1024)
def _paged_bytes(dev, T, Hq, R, width, n_pages, H_kv, page, d, f8):
    """Workspace of an attention call (it goes by sizes alone; the addresses only have to be set)."""
    c = fm_kv_cache(16, 16, 16 if f8 else 0, 16 if f8 else 0, n_pages, H_kv, page, d)
    with torch.cuda.device(dev):
        return lib().fm_attn_paged_workspace_bytes(c, fm_paged_batch(16, 16, 16, R, width), T, Hq)


def fm_attn_paged_workspace_bytes(cache: KVCache, batch: PagedBatch, T: int, H_q: int) -> int:
    """Bytes of workspace an fm_attn_paged call of these shapes needs."""
    if not (0 <= T <= _MOST and 0 < H_q <= _MOST):
        raise ValueError(f"T must be in [0, 2^30], H_q in [1, 2^30], got {T} and {H_q}")
    return _paged_bytes(_serve_args(cache, batch), T, H_q, batch.R, batch.width, cache.n_pages, cache.H_kv,
                        cache.page_size, cache.d, cache.k_exp is not None)


@_streamed
def fm_attn_paged(q, cache: KVCache, batch: PagedBatch, *, scale: float, causal: bool = True, window: int = 0,
                  sinks: int = 0, o=None, lse=None, ws=None):
    """Attention of T new tokens q (T, H_q, d) over the paged cache, their own keys and
    values written before (fm_cache_write): (O bf16 (T, H_q, d), LSE fp32 (T, H_q)).
    Position p sees key j < kv_len iff j <= p (when causal) and, with a window,
    j > p - window or j < sinks. Rows of tokens past q_off[R] are left as they
    were (undefined in new tensors). ws: a uint8 workspace of
    fm_attn_paged_workspace_bytes, one for each call that may run at once."""
    dev = _serve_args(cache, batch)
    _tensor(q, "q", 3)
    T, Hq, d = shape = q.shape
    if d != cache.d:
        raise ValueError(f"q has d={d}, the cache d={cache.d}")
    if Hq <= 0 or Hq % cache.H_kv:
        raise ValueError(f"H_q={Hq} must be a multiple of H_kv={cache.H_kv}")
    if not (0 <= window and 0 <= sinks):
        raise ValueError(f"window and sinks must not be negative, got {window} and {sinks}")
    window, sinks = min(window, 1 << 30), min(sinks, 1 << 30)  # (all positions are below)
    qr = _rows(q, "q", shape, dev)
    wsb = fm_attn_paged_workspace_bytes(cache, batch, T, Hq)
    if o is None:
        o = torch.empty(shape, dtype=_BF16, device=cache.device)
        orow = _pack_rows(o.data_ptr(), Hq * d, d)
    else:
        orow = _rows(o, "o", shape, dev, True)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=_F32, device=cache.device)
    else:
        _expect(lse, "lse", (T, Hq), _F32, dev)
    if ws is None:
        ws = torch.empty(max(16, wsb), dtype=_U8, device=cache.device)
    elif (not isinstance(ws, torch.Tensor) or not ws.is_contiguous() or ws.dtype != _U8 or ws.numel() < wsb
          or ws.get_device() != dev):
        raise ValueError(f"ws must be a contiguous uint8 tensor of at least {wsb} bytes on the cache's device")
    _enqueue("fm_attn_paged", dev, cache.at, batch.at, T, Hq, qr, scale, 1 if causal else 0, window, sinks,
             orow, lse.data_ptr(), ws.data_ptr(), wsb)
    return o, lse


class SharedPrefix:
    """Groups of a batch's sequences that share their first keys, int32 CUDA tensors:
    sequences [seq_off[g], seq_off[g + 1]) hold the same first prefix_len[g] keys, the
    whole pages of them as the same pages. seq_off (S + 1,) ascends from 0 to R. Checked
    once; the tensors' values may change between calls (their addresses may not).
    max_prefix: how long prefixes are at most in such calls, by which a call decides
    whether sharing them pays (0: not known, then what the page table has room for; a
    longer one is no error)."""

    __slots__ = ("seq_off", "prefix_len", "S", "index", "c", "at", "__dict__")
    max_prefix = 0

    def __init__(self, seq_off, prefix_len, max_prefix: int = 0):
        _need(isinstance(prefix_len, torch.Tensor) and prefix_len.dim() == 1, "prefix_len must be (S,)")
        S = prefix_len.shape[0]
        _need(0 < S <= _MOST, f"there must be 1 to 2^30 groups, got {S}")
        _need(0 <= max_prefix <= _MOST, f"max_prefix must be in [0, 2^30], got {max_prefix}")
        _like(prefix_len, "prefix_len", (S,), torch.int32)
        _like(seq_off, "seq_off", (S + 1,), torch.int32)
        _same_cuda(seq_off=seq_off, prefix_len=prefix_len)
        self.seq_off, self.prefix_len, self.S, self.index = seq_off, prefix_len, S, seq_off.get_device()
        self.max_prefix = int(max_prefix)
        self.c = fm_shared_prefix(seq_off.data_ptr(), prefix_len.data_ptr(), S, self.max_prefix)
        self.at = ctypes.addressof(self.c)


@functools.lru_cache(maxsize=1024)
def _shared_bytes(dev, T, Hq, R, width, S, max_prefix, n_pages, H_kv, page, d, f8):
    c = fm_kv_cache(16, 16, 16 if f8 else 0, 16 if f8 else 0, n_pages, H_kv, page, d)
    with torch.cuda.device(dev):
        return lib().fm_attn_shared_workspace_bytes(c, fm_paged_batch(16, 16, 16, R, width),
                                                    fm_shared_prefix(16, 16, S, max_prefix), T, Hq)


def fm_attn_shared_workspace_bytes(cache: KVCache, batch: PagedBatch, shared: SharedPrefix, T: int, H_q: int) -> int:
    """Bytes of workspace an fm_attn_shared call of these shapes needs."""
    if not (0 <= T <= _MOST and 0 < H_q <= _MOST):
        raise ValueError(f"T must be in [0, 2^30], H_q in [1, 2^30], got {T} and {H_q}")
    dev = _serve_args(cache, batch)
    if not isinstance(shared, SharedPrefix):
        raise ValueError("shared must be a SharedPrefix")
    if shared.index != dev:
        raise ValueError("the groups are on another device than the cache")
    return _shared_bytes(dev, T, H_q, batch.R, batch.width, shared.S, shared.max_prefix, cache.n_pages, cache.H_kv,
                         cache.page_size, cache.d, cache.k_exp is not None)


@_streamed
def fm_attn_shared(q, cache: KVCache, batch: PagedBatch, shared: SharedPrefix, *, scale: float, causal: bool = True,
                   o=None, lse=None, ws=None):
    """fm_attn_paged of a batch whose sequences share prefixes, as `shared` says: each
    group's shared keys are read once for all of its new tokens. (O bf16 (T, H_q, d),
    LSE fp32 (T, H_q)). Rows of tokens past q_off[R] are left as they were (undefined in
    new tensors). ws: a uint8 workspace of fm_attn_shared_workspace_bytes, one for each
    call that may run at once."""
    dev = _serve_args(cache, batch)
    _tensor(q, "q", 3)
    T, Hq, d = shape = q.shape
    if d != cache.d:
        raise ValueError(f"q has d={d}, the cache d={cache.d}")
    if Hq <= 0 or Hq % cache.H_kv:
        raise ValueError(f"H_q={Hq} must be a multiple of H_kv={cache.H_kv}")
    qr = _rows(q, "q", shape, dev)
    wsb = fm_attn_shared_workspace_bytes(cache, batch, shared, T, Hq)
    if o is None:
        o = torch.empty(shape, dtype=_BF16, device=cache.device)
        orow = _pack_rows(o.data_ptr(), Hq * d, d)
    else:
        orow = _rows(o, "o", shape, dev, True)
    if lse is None:
        lse = torch.empty((T, Hq), dtype=_F32, device=cache.device)
    else:
        _expect(lse, "lse", (T, Hq), _F32, dev)
    if ws is None:
        ws = torch.empty(max(16, wsb), dtype=_U8, device=cache.device)
    elif (not isinstance(ws, torch.Tensor) or not ws.is_contiguous() or ws.dtype != _U8 or ws.numel() < wsb
          or ws.get_device() != dev):
        raise ValueError(f"ws must be a contiguous uint8 tensor of at least {wsb} bytes on the cache's device")
    _enqueue("fm_attn_shared", dev, cache.at, batch.at, shared.at, T, Hq, qr, scale, 1 if causal else 0, orow,
             lse.data_ptr(), ws.data_ptr(), wsb)
    return o, lse


@dataclass
class QKNormRope:
    """Norm and rotation of a flashmask_attention call's queries and keys
    (the arguments of fm_qk_norm_rope). Gradients reach q_weight and k_weight."""
    positions: torch.Tensor | None = None
    inv_freq: torch.Tensor | None = None
    interleaved: bool = False
    rot_scale: float = 1.0
    q_weight: torch.Tensor | None = None
    k_weight: torch.Tensor | None = None
    eps: float = 1e-6


class _FirstOnly(torch.autograd.Function):
    """n gradients, and the tensors that they depend on: passes the gradients on, so
    that a gradient of theirs raises instead of missing the library calls' part.
    (once_differentiable goes by the incoming gradients alone.)"""

    @staticmethod
    def forward(ctx, n, *tensors):
        ctx.mark_dirty(*(t for t in tensors[:n] if t is not None))  # the same tensors, no views of them
        return tensors[:n]

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("flashmask_attention has no second derivatives: its gradients cannot be differentiated")


def _first_only(grads, *depends_on):
    return _FirstOnly.apply(len(grads), *grads, *depends_on) if torch.is_grad_enabled() else grads


class _QKNormRopeFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, wq, wk, positions, inv_freq, interleaved, rot_scale, eps):
        how = dict(interleaved=interleaved, rot_scale=rot_scale, eps=eps)
        ctx.save_for_backward(q, k, wq, wk, positions, inv_freq)
        ctx.how = how
        return fm_qk_norm_rope(q, k, v, positions=positions, inv_freq=inv_freq, q_weight=wq, k_weight=wk, **how)

    @staticmethod
    def backward(ctx, dqo, dko, dvo):
        q, k, wq, wk, positions, inv_freq = ctx.saved_tensors
        grads = fm_qk_norm_rope_bwd(dqo.contiguous(), dko.contiguous(), dvo.contiguous(), q, k, positions=positions,
                                    inv_freq=inv_freq, q_weight=wq, k_weight=wk, **ctx.how)
        grads = _first_only(grads, dqo, dko, dvo, q, k, wq, wk)
        return (*grads, None, None, None, None, None)


class _FlashMaskFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, lts, lte, uts, ute, scale, causal):
        bm, bn = attn_tiling()
        queues = fm_classify_tiles(lts, lte, uts, ute, causal=causal, block_m=bm, block_n=bn, n_rows=q.shape[2])
        o, lse = fm_attn_fwd(q, k, v, lts, lte, uts, ute, queues, scale=scale, causal=causal)
        ctx.save_for_backward(q, k, v, o, lse, lts, lte, uts, ute)
        ctx.queues, ctx.scale, ctx.causal = queues, scale, causal
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, lts, lte, uts, ute = ctx.saved_tensors
        dq, dk, dv = fm_attn_bwd(q, k, v, o, lse, do.contiguous(), lts, lte, uts, ute, ctx.queues, scale=ctx.scale,
                                 causal=ctx.causal)
        dq, dk, dv = _first_only((dq, dk, dv), do, q, k, v)
        return dq, dk, dv, None, None, None, None, None, None


def flashmask_attention(q, k, v, lts, lte, uts, ute, *, causal: bool, scale: float | None = None,
                        qk: QKNormRope | None = None):
    """Masked SDPA with the FlashMask column-wise mask; differentiable in q, k, v, once
    (a gradient of its gradients is refused).

    qk: norm and rotate the queries and keys first (fm_qk_norm_rope, in one pass
    that also lays q, k, v out): q, k, v may then be strided views, e.g. of a fused
    projection's output, and gradients reach the norms' weights too."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    if qk is not None:
        q, k, v = _QKNormRopeFn.apply(q, k, v, qk.q_weight, qk.k_weight, qk.positions, qk.inv_freq,
                                      bool(qk.interleaved), float(qk.rot_scale), float(qk.eps))
    return _FlashMaskFn.apply(q, k, v, lts, lte, uts, ute, float(scale), bool(causal))
