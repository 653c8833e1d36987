"""ctypes binding of libupf (include/upf.h): argument marshalling only.

Every function here has the name of the C entry point it calls and passes
plain integers (device pointers, sizes, the CUDA stream handle) through.  All
computation happens in libupf's CUDA kernels; if the library is missing or
cannot be loaded, every call raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_char_p, c_double, c_float, c_int, c_int32, c_int64, c_size_t, c_uint64, c_void_p
from typing import Optional, Sequence

import numpy as np

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("UPF_LIBRARY", os.path.join(_PKG_DIR, "libupf.so"))

UPF_OK = 0
STATUS_NAMES = {0: "UPF_OK", 1: "UPF_ERR_INVALID_ARG", 2: "UPF_ERR_UNSUPPORTED", 3: "UPF_ERR_CUDA",
                4: "UPF_ERR_CAPACITY", 5: "UPF_ERR_NONFINITE", 6: "UPF_ERR_TIMEOUT"}


class UpfError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


class UpfBatch(ctypes.Structure):
    _fields_ = [("num_reqs", c_int32), ("cu_seqlens_dev", c_void_p), ("cu_seqlens_host", POINTER(c_int32)),
                ("num_q_heads", c_int32), ("num_kv_heads", c_int32), ("head_dim", c_int32),
                ("kv_of_q", POINTER(c_int32))]


class UpfParams(ctypes.Structure):
    _fields_ = [("n_tail", c_int32), ("block", c_int32), ("sink_keep", c_int32), ("tail_keep", c_int32),
                ("top_p", c_float), ("softmax_scale", c_float)]


class UpfCompactIO(ctypes.Structure):
    _fields_ = [("row_bytes", c_int64), ("hidden_in", c_void_p), ("hidden_out", c_void_p),
                ("pos_in", c_void_p), ("pos_out", c_void_p), ("slot_in", c_void_p), ("slot_out", c_void_p),
                ("kept_index", c_void_p), ("cu_seqlens_out", c_void_p), ("total_kept", c_void_p),
                ("layer_id", c_int32), ("history_cap", c_int32), ("history", c_void_p), ("history_len", c_void_p)]


class UpfKvCache(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("num_slots", c_int64), ("num_kv_heads", c_int32), ("head_dim", c_int32),
                ("k_exp", c_int32), ("v_exp", c_int32)]


class UpfKvQuery(ctypes.Structure):
    _fields_ = [("num_reqs", c_int32), ("num_q_heads", c_int32), ("kv_of_q", POINTER(c_int32)),
                ("num_q_tokens", c_int32), ("max_q_len", c_int32), ("cu_q", c_void_p), ("kv_len", c_void_p),
                ("page_table", c_void_p), ("page_stride", c_int64), ("max_pages", c_int32), ("page_size", c_int32),
                ("window", c_int32), ("sinks", c_int32), ("softmax_scale", c_float)]


class UpfKvEviction(ctypes.Structure):
    _fields_ = [("num_reqs", c_int32), ("kv_len", c_void_p), ("kv_len_out", c_void_p), ("page_table", c_void_p),
                ("page_stride", c_int64), ("max_pages", c_int32), ("page_size", c_int32), ("page_table_out", c_void_p),
                ("page_stride_out", c_int64), ("max_pages_out", c_int32), ("budget", c_int32), ("trigger", c_int32),
                ("sinks", c_int32), ("recent", c_int32), ("weights", c_void_p), ("weights_stride", c_int64),
                ("weights_cols", c_int32), ("weights_out_cols", c_int32), ("weights_out", c_void_p),
                ("weights_out_stride", c_int64), ("kept", c_void_p), ("kept_stride", c_int64)]


class UpfRope(ctypes.Structure):
    _fields_ = [("head_dim", c_int32), ("rotary_dim", c_int32), ("interleaved", c_int32), ("scaling", c_int32),
                ("base", c_double), ("factor", c_double), ("original_len", c_double), ("low", c_double),
                ("high", c_double), ("divisors", POINTER(c_double)), ("magnitude", c_double)]


UPF_BF16, UPF_F16 = 0, 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "yarn": 3, "bands": 4}
UPF_KV_FEW_TOKENS = 1024

_SIGNATURES = {
    "upf_version": ([], c_int),
    "upf_default_params": ([POINTER(UpfParams)], None),
    "upf_status_name": ([c_int], c_char_p),
    "upf_last_error": ([], c_char_p),
    "upf_create": ([POINTER(c_void_p), c_int], c_int),
    "upf_destroy": ([c_void_p], c_int),
    "upf_sync_status": ([c_void_p, c_void_p], c_int),
    "upf_workspace_bytes": ([POINTER(UpfBatch), POINTER(UpfParams)], c_size_t),
    "upf_score": ([c_void_p, POINTER(UpfBatch), POINTER(UpfParams), c_void_p, c_int64, c_void_p, c_int64,
                   c_void_p, c_void_p, c_size_t, c_void_p], c_int),
    "upf_score_shard": ([c_void_p, POINTER(UpfBatch), POINTER(UpfParams), c_int32, c_void_p, c_int64, c_void_p,
                         c_int64, c_void_p, c_void_p, c_size_t, c_void_p], c_int),
    "upf_set_wait_limit": ([c_void_p, c_int64], c_int),
    "upf_plan_info": ([POINTER(UpfBatch), POINTER(UpfParams), POINTER(c_int32), POINTER(c_int32), POINTER(c_int64),
                       POINTER(c_int64), POINTER(c_int32), POINTER(c_int32)], c_int),
    "upf_select": ([c_void_p, POINTER(UpfBatch), POINTER(UpfParams), c_void_p, c_void_p, c_void_p, c_void_p,
                    c_void_p, c_size_t, c_void_p], c_int),
    "upf_compact": ([c_void_p, POINTER(UpfBatch), c_void_p, POINTER(UpfCompactIO), c_void_p, c_size_t, c_void_p],
                    c_int),
    "upf_select_noalloc": ([POINTER(UpfBatch), POINTER(UpfParams), c_void_p, c_void_p, c_void_p, c_void_p,
                            c_void_p, c_void_p], c_int),
    "upf_revive": ([c_void_p, POINTER(UpfBatch), c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p], c_int),
    "upf_history_kv_len": ([c_void_p, POINTER(UpfBatch), c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_void_p],
                           c_int),
    "upf_kv_cache_bytes": ([POINTER(UpfKvCache)], c_size_t),
    "upf_kv_write_workspace_bytes": ([POINTER(UpfKvCache), c_int32], c_size_t),
    "upf_kv_write": ([c_void_p, POINTER(UpfKvCache), c_int32, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int32,
                      c_void_p, c_void_p, c_size_t, c_void_p], c_int),
    "upf_kv_read": ([c_void_p, POINTER(UpfKvCache), c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_int64, c_void_p,
                     c_int64, c_void_p], c_int),
    "upf_kv_attend_workspace_bytes": ([POINTER(UpfKvCache), POINTER(UpfKvQuery)], c_size_t),
    "upf_kv_attend": ([c_void_p, POINTER(UpfKvCache), POINTER(UpfKvQuery), c_int32, c_void_p, c_int64, c_void_p,
                       c_int64, c_void_p, c_void_p, c_size_t, c_void_p], c_int),
    "upf_kv_accumulate_workspace_bytes": ([POINTER(UpfKvCache), POINTER(UpfKvQuery)], c_size_t),
    "upf_kv_accumulate": ([c_void_p, POINTER(UpfKvCache), POINTER(UpfKvQuery), c_int32, c_void_p, c_int64, c_void_p,
                           c_float, c_void_p, c_void_p, c_int64, c_int32, c_void_p, c_size_t, c_void_p], c_int),
    "upf_kv_evict_workspace_bytes": ([POINTER(UpfKvCache), POINTER(UpfKvEviction)], c_size_t),
    "upf_kv_evict": ([c_void_p, POINTER(UpfKvCache), POINTER(UpfKvEviction), c_void_p, c_size_t, c_void_p], c_int),
    "upf_rope_turns": ([POINTER(UpfRope), POINTER(c_uint64), POINTER(c_double)], c_int),
    "upf_rope_apply": ([c_void_p, POINTER(UpfRope), c_void_p, c_int32, c_int32, c_void_p, c_int32, c_void_p, c_void_p,
                        c_int64, c_void_p, c_int64, c_int32, c_void_p, c_int64, c_void_p, c_int64, c_int32, c_void_p],
                       c_int),
    "upf_stage_name": ([c_int32], c_char_p),
    "upf_profile_enable": ([c_void_p, c_int32], c_int),
    "upf_profile_read": ([c_void_p, c_void_p, c_void_p, c_int32], c_int),
    "upf_select_tokens": ([c_void_p, POINTER(UpfBatch), POINTER(UpfParams), c_void_p, c_int64, c_void_p, c_int64,
                           c_void_p, c_void_p, c_void_p, c_void_p, POINTER(UpfCompactIO), c_void_p, c_size_t,
                           c_void_p], c_int),
    "upf_select_tokens_check": ([c_void_p, POINTER(UpfBatch), POINTER(UpfParams), c_void_p, c_int64, c_void_p, c_int64,
                                 c_void_p, c_void_p, POINTER(UpfCompactIO), c_void_p, c_size_t], c_int),
}

_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libupf.so (built by ``sparse_long_context_tail_gb300.build``); raise if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libupf is not built ({p} missing): run __graft_entry__.build() or "
                           f"python -m sparse_long_context_tail_gb300.build")
    lib = ctypes.CDLL(p)
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


def _check(status: int) -> None:
    if status != UPF_OK:
        raise UpfError(status, load().upf_last_error().decode())


# ------------------------------------------------------------------ structs --

def _head_map(kv_of_q: Optional[Sequence[int]], num_q_heads: int) -> Optional[np.ndarray]:
    """The kv head of each q head for the library, which reads num_q_heads entries."""
    if kv_of_q is None:
        return None
    kv = np.ascontiguousarray(kv_of_q, dtype=np.int32)
    if kv.shape != (num_q_heads,):
        raise ValueError(f"kv_of_q has shape {kv.shape}, expected a kv head for each of {num_q_heads} q heads")
    return kv


def make_batch(cu_seqlens_dev: int, cu_seqlens_host: np.ndarray, num_q_heads: int, num_kv_heads: int,
               head_dim: int, kv_of_q: Optional[Sequence[int]] = None):
    """Build a upf_batch; returns (struct, keepalive) -- keep both alive during the call."""
    cu = np.ascontiguousarray(cu_seqlens_host, dtype=np.int32)
    kv = _head_map(kv_of_q, num_q_heads)
    b = UpfBatch(len(cu) - 1, ctypes.c_void_p(cu_seqlens_dev), cu.ctypes.data_as(POINTER(c_int32)),
                 num_q_heads, num_kv_heads, head_dim,
                 kv.ctypes.data_as(POINTER(c_int32)) if kv is not None else POINTER(c_int32)())
    return b, (cu, kv)


def make_params(n_tail: int = 128, block: int = 64, sink_keep: int = 128, tail_keep: int = 128,
                top_p: float = 0.99, softmax_scale: float = 0.0) -> UpfParams:
    return UpfParams(n_tail, block, sink_keep, tail_keep, top_p, softmax_scale)


def make_compact_io(row_bytes=0, hidden_in=0, hidden_out=0, pos_in=0, pos_out=0, slot_in=0, slot_out=0,
                    kept_index=0, cu_seqlens_out=0, total_kept=0, layer_id=0, history_cap=0, history=0,
                    history_len=0) -> UpfCompactIO:
    return UpfCompactIO(row_bytes, hidden_in or None, hidden_out or None, pos_in or None, pos_out or None,
                        slot_in or None, slot_out or None, kept_index or None, cu_seqlens_out or None,
                        total_kept or None, layer_id, history_cap, history or None, history_len or None)


def _check_int32(**sizes: int) -> None:
    """ctypes cuts a larger number down to its low bits without a word."""
    for name, value in sizes.items():
        if not -2 ** 31 <= value < 2 ** 31:
            raise ValueError(f"{name} {value} does not fit 32 bits")


def make_kv_cache(data: int, num_slots: int, num_kv_heads: int, head_dim: int, k_exp: int = 0,
                  v_exp: int = 0) -> UpfKvCache:
    _check_int32(num_kv_heads=num_kv_heads, head_dim=head_dim, k_exp=k_exp, v_exp=v_exp)
    return UpfKvCache(data or None, num_slots, num_kv_heads, head_dim, k_exp, v_exp)


def make_kv_query(num_reqs: int, num_q_heads: int, num_q_tokens: int, kv_len: int, page_table: int, page_stride: int,
                  max_pages: int, page_size: int, cu_q: int = 0, max_q_len: int = 1, window: int = 0, sinks: int = 0,
                  softmax_scale: float = 0.0, kv_of_q: Optional[Sequence[int]] = None):
    """Build a upf_kv_query; returns (struct, keepalive) -- keep both alive during the call."""
    if (max_q_len | page_size | window | sinks) >> 31:      # one is negative or too large
        _check_int32(max_q_len=max_q_len, page_size=page_size, window=window, sinks=sinks)
    kv = _head_map(kv_of_q, num_q_heads)
    x = UpfKvQuery(num_reqs, num_q_heads, kv.ctypes.data_as(POINTER(c_int32)) if kv is not None else None,
                   num_q_tokens, max_q_len, cu_q or None, kv_len or None, page_table or None, page_stride, max_pages,
                   page_size, window, sinks, softmax_scale)
    return x, kv


def make_kv_eviction(num_reqs: int, kv_len: int, kv_len_out: int, page_table: int, page_stride: int, max_pages: int,
                     page_size: int, weights: int, weights_stride: int, weights_cols: int, weights_out: int,
                     weights_out_stride: int, weights_out_cols: int, budget: int, trigger: int, sinks: int = 0,
                     recent: int = 0, page_table_out: int = 0, page_stride_out: int = 0, max_pages_out: int = 0,
                     kept: int = 0, kept_stride: int = 0) -> UpfKvEviction:
    if (page_size | budget | trigger | sinks | recent | weights_cols | weights_out_cols) >> 31:   # as in make_kv_query
        _check_int32(page_size=page_size, budget=budget, trigger=trigger, sinks=sinks, recent=recent,
                     weights_cols=weights_cols, weights_out_cols=weights_out_cols)
    return UpfKvEviction(num_reqs, kv_len or None, kv_len_out or None, page_table or None, page_stride, max_pages,
                         page_size, page_table_out or None, page_stride_out, max_pages_out, budget, trigger, sinks,
                         recent, weights or None, weights_stride, weights_cols, weights_out_cols, weights_out or None,
                         weights_out_stride, kept or None, kept_stride)


def make_rope(head_dim: int, rotary_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
              factor: float = 1.0, original_len: float = 0.0, low: float = 0.0, high: float = 0.0,
              divisors: Optional[Sequence[float]] = None, magnitude: float = 0.0):
    """Build a upf_rope; returns (struct, keepalive) -- keep both alive during the calls."""
    _check_int32(head_dim=head_dim, rotary_dim=rotary_dim)
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, not {scaling!r}")
    div = None
    if divisors is not None:
        div = np.ascontiguousarray(divisors, dtype=np.float64)
        if div.shape != (rotary_dim // 2,):
            raise ValueError(f"divisors has shape {div.shape}, expected one for each of {rotary_dim // 2} pairs")
    x = UpfRope(head_dim, rotary_dim, 1 if interleaved else 0, ROPE_SCALINGS[scaling], base, factor, original_len, low,
                high, div.ctypes.data_as(POINTER(c_double)) if div is not None else None, magnitude)
    return x, div


# ------------------------------------------------------- entry points (C ABI) --

def upf_version() -> int:
    return load().upf_version()


def upf_default_params() -> UpfParams:
    p = UpfParams()
    load().upf_default_params(ctypes.byref(p))
    return p


def upf_status_name(status: int) -> str:
    return load().upf_status_name(status).decode()


def upf_last_error() -> str:
    return load().upf_last_error().decode()


def upf_create(device: int = 0) -> int:
    h = c_void_p()
    _check(load().upf_create(ctypes.byref(h), device))
    return h.value


def upf_destroy(ctx: int) -> None:
    _check(load().upf_destroy(ctx))


def upf_sync_status(ctx: int, stream: int = 0) -> int:
    """Return the device status code (0 = OK) without raising."""
    return load().upf_sync_status(ctx, stream or None)


def upf_workspace_bytes(batch: UpfBatch, params: UpfParams) -> int:
    n = load().upf_workspace_bytes(ctypes.byref(batch), ctypes.byref(params))
    if n == 0:
        raise UpfError(1, upf_last_error())
    return n


def upf_score(ctx, batch, params, q, q_row_stride, k, k_row_stride, scores, ws, ws_bytes, stream=0):
    _check(load().upf_score(ctx, ctypes.byref(batch), ctypes.byref(params), q, q_row_stride, k, k_row_stride,
                            scores, ws, ws_bytes, stream or None))


def upf_score_shard(ctx, batch, params, num_q_heads_total, q, q_row_stride, k, k_row_stride, scores, ws, ws_bytes,
                    stream=0):
    _check(load().upf_score_shard(ctx, ctypes.byref(batch), ctypes.byref(params), num_q_heads_total, q, q_row_stride,
                                  k, k_row_stride, scores, ws, ws_bytes, stream or None))


def upf_plan_info(batch: UpfBatch, params: UpfParams):
    """(keys per split of pass 1, of pass 2, items of pass 1, items of pass 2,
    CTAs per item of pass 1, of pass 2)."""
    k1, k2, i1, i2, c1, c2 = c_int32(), c_int32(), c_int64(), c_int64(), c_int32(), c_int32()
    _check(load().upf_plan_info(ctypes.byref(batch), ctypes.byref(params), ctypes.byref(k1), ctypes.byref(k2),
                                ctypes.byref(i1), ctypes.byref(i2), ctypes.byref(c1), ctypes.byref(c2)))
    return k1.value, k2.value, i1.value, i2.value, c1.value, c2.value


def upf_set_wait_limit(ctx: int, cycles: int) -> None:
    _check(load().upf_set_wait_limit(ctx, cycles))


def upf_select(ctx, batch, params, scores, block_scores, keep_bits, kept_count, ws, ws_bytes, stream=0):
    _check(load().upf_select(ctx, ctypes.byref(batch), ctypes.byref(params), scores, block_scores or None,
                             keep_bits, kept_count, ws, ws_bytes, stream or None))


def upf_select_noalloc(batch, params, scores, block_scores, keep_bits, kept_count, status_dev=0, stream=0):
    """upf_select without a context or workspace (scratch in a fixed array inside the library)."""
    _check(load().upf_select_noalloc(ctypes.byref(batch), ctypes.byref(params), scores, block_scores or None,
                                     keep_bits, kept_count, status_dev or None, stream or None))


def upf_compact(ctx, batch, keep_bits, io: UpfCompactIO, ws, ws_bytes, stream=0):
    _check(load().upf_compact(ctx, ctypes.byref(batch), keep_bits, ctypes.byref(io), ws, ws_bytes, stream or None))


def upf_revive(ctx, batch, kept_index, total_kept, rows, row_bytes, full, stream=0):
    _check(load().upf_revive(ctx, ctypes.byref(batch), kept_index, total_kept, rows, row_bytes, full, stream or None))


def upf_history_kv_len(ctx, batch, history, history_len, history_cap, layer_id, kv_len, stream=0):
    _check(load().upf_history_kv_len(ctx, ctypes.byref(batch), history, history_len, history_cap, layer_id, kv_len,
                                     stream or None))


def upf_kv_cache_bytes(cache: UpfKvCache) -> int:
    n = load().upf_kv_cache_bytes(ctypes.byref(cache))
    if n == 0:
        raise UpfError(1, upf_last_error())
    return n


def upf_kv_write_workspace_bytes(cache: UpfKvCache, num_tokens: int) -> int:
    n = load().upf_kv_write_workspace_bytes(ctypes.byref(cache), num_tokens)
    if n == 0:
        raise UpfError(1, upf_last_error())
    return n


def upf_kv_write(ctx, cache, dtype, k, k_row_stride, v, v_row_stride, slots, num_tokens, num_tokens_dev, ws, ws_bytes,
                 stream=0):
    lib = _lib or load()
    _check(lib.upf_kv_write(ctx, ctypes.byref(cache), dtype, k, k_row_stride, v, v_row_stride, slots, num_tokens,
                            num_tokens_dev or None, ws or None, ws_bytes, stream or None))


def upf_kv_read(ctx, cache, dtype, slots, num_tokens, num_tokens_dev, k, k_row_stride, v, v_row_stride, stream=0):
    lib = _lib or load()
    _check(lib.upf_kv_read(ctx, ctypes.byref(cache), dtype, slots, num_tokens, num_tokens_dev or None, k or None,
                           k_row_stride, v or None, v_row_stride, stream or None))


def upf_kv_attend_workspace_bytes(cache: UpfKvCache, query: UpfKvQuery) -> int:
    n = load().upf_kv_attend_workspace_bytes(ctypes.byref(cache), ctypes.byref(query))
    if n == 0:
        raise UpfError(1, upf_last_error())
    return n


def upf_kv_attend(ctx, cache, query, dtype, q, q_row_stride, out, out_row_stride, lse, ws, ws_bytes, stream=0):
    lib = _lib or load()
    _check(lib.upf_kv_attend(ctx, ctypes.byref(cache), ctypes.byref(query), dtype, q, q_row_stride, out,
                             out_row_stride, lse or None, ws, ws_bytes, stream or None))


def upf_kv_accumulate_workspace_bytes(cache: UpfKvCache, query: UpfKvQuery) -> int:
    n = load().upf_kv_accumulate_workspace_bytes(ctypes.byref(cache), ctypes.byref(query))
    if n == 0:
        raise UpfError(1, upf_last_error())
    return n


def upf_kv_accumulate(ctx, cache, query, dtype, q, q_row_stride, lse, decay, weights_in, weights_out, weights_stride,
                      weights_cols, ws, ws_bytes, stream=0):
    lib = _lib or load()
    _check(lib.upf_kv_accumulate(ctx, ctypes.byref(cache), ctypes.byref(query), dtype, q, q_row_stride, lse, decay,
                                 weights_in or None, weights_out, weights_stride, weights_cols, ws, ws_bytes,
                                 stream or None))


def upf_kv_evict_workspace_bytes(cache: UpfKvCache, eviction: UpfKvEviction) -> int:
    n = load().upf_kv_evict_workspace_bytes(ctypes.byref(cache), ctypes.byref(eviction))
    if n == 0:
        raise UpfError(1, upf_last_error())
    return n


def upf_kv_evict(ctx, cache, eviction, ws, ws_bytes, stream=0):
    lib = _lib or load()
    _check(lib.upf_kv_evict(ctx, ctypes.byref(cache), ctypes.byref(eviction), ws, ws_bytes, stream or None))


def upf_rope_turns(rope: UpfRope):
    """(turns as numpy uint64 [rotary_dim / 2], magnitude)."""
    turns = np.zeros(max(1, rope.rotary_dim // 2), dtype=np.uint64)
    m = c_double()
    _check(load().upf_rope_turns(ctypes.byref(rope), turns.ctypes.data_as(POINTER(c_uint64)), ctypes.byref(m)))
    return turns, m.value


def upf_rope_apply(ctx, rope, turns_dev, inverse, dtype, positions, num_tokens, num_tokens_dev, q, q_row_stride, q_out,
                   q_out_row_stride, num_q_heads, k, k_row_stride, k_out, k_out_row_stride, num_kv_heads, stream=0):
    lib = _lib or load()
    _check(lib.upf_rope_apply(ctx, ctypes.byref(rope), turns_dev, inverse, dtype, positions, num_tokens,
                              num_tokens_dev or None, q or None, q_row_stride, q_out or None, q_out_row_stride,
                              num_q_heads, k or None, k_row_stride, k_out or None, k_out_row_stride, num_kv_heads,
                              stream or None))


NUM_STAGES = 8


def upf_stage_name(stage: int) -> str:
    return load().upf_stage_name(stage).decode()


def upf_profile_enable(ctx: int, on: bool = True) -> None:
    _check(load().upf_profile_enable(ctx, 1 if on else 0))


def upf_profile_read(ctx: int):
    """Per-stage (launches, device ms) since the previous read, as two lists."""
    launches = (c_int32 * NUM_STAGES)()
    ms = (ctypes.c_double * NUM_STAGES)()
    _check(load().upf_profile_read(ctx, ctypes.byref(launches), ctypes.byref(ms), NUM_STAGES))
    return list(launches), list(ms)


def upf_select_tokens(ctx, batch, params, q, q_row_stride, k, k_row_stride, scores, block_scores, keep_bits,
                      kept_count, io: UpfCompactIO, ws, ws_bytes, stream=0):
    _check(load().upf_select_tokens(ctx, ctypes.byref(batch), ctypes.byref(params), q, q_row_stride, k,
                                    k_row_stride, scores or None, block_scores or None, keep_bits, kept_count,
                                    ctypes.byref(io), ws, ws_bytes, stream or None))


def upf_select_tokens_check(ctx, batch, params, q, q_row_stride, k, k_row_stride, keep_bits, kept_count, io: UpfCompactIO,
                            ws, ws_bytes):
    _check(load().upf_select_tokens_check(ctx, ctypes.byref(batch), ctypes.byref(params), q, q_row_stride, k,
                                          k_row_stride, keep_bits, kept_count, ctypes.byref(io), ws, ws_bytes))
