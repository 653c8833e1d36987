"""Torch-tensor front end of the 4-bit KV cache: checks, output allocation and pointer passing.

``QuantKVCache`` holds one layer's keys and values as 4-bit floats (``include/upf.h``
has the format).  It takes what the selection hands out: ``write`` stores kept
tokens at their slot ids (``SelectOutputs.slot_out``, with ``total_kept`` as the
device-side count), ``read`` gives entries back, and ``attend`` runs the attention
of new tokens over ``kv_len`` entries per request (``upf_history_kv_len``), with or
without a sliding window beside a few first entries.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import _binding as B

_DTYPES = {torch.bfloat16: B.UPF_BF16, torch.float16: B.UPF_F16}


class AttendOutputs(NamedTuple):
    out: torch.Tensor    # [num_q_tokens, H_q, d], the type of q
    lse: torch.Tensor    # float32 [num_q_tokens, H_q], natural logarithm; -inf for a row that sees nothing


class QuantKVCache:
    """One layer's cache of ``num_slots`` slots on one GPU, with its own libupf context.

    ``storage``: uint8 tensor of ``upf_kv_cache_bytes`` bytes to use (any contiguous shape);
    by default one is allocated, its slots unwritten.  ``k_exp`` / ``v_exp`` scale the range
    by a power of two.  Calls run on the current stream of the cache's device; one
    cache must not be used by two streams at the same time, and has to outlive the graphs that
    captured calls on it."""

    def __init__(self, num_slots: int, num_kv_heads: int, head_dim: int, device: Optional[int] = None, k_exp: int = 0,
                 v_exp: int = 0, storage: Optional[torch.Tensor] = None):
        self.ctx = 0
        self.num_slots, self.num_kv_heads, self.head_dim = num_slots, num_kv_heads, head_dim
        self._cache = B.make_kv_cache(0, num_slots, num_kv_heads, head_dim, k_exp, v_exp)
        nbytes = B.upf_kv_cache_bytes(self._cache)
        if storage is not None:
            if storage.dtype != torch.uint8 or not storage.is_cuda or not storage.is_contiguous():
                raise ValueError("storage must be a contiguous uint8 CUDA tensor")
            if storage.numel() != nbytes:
                raise ValueError(f"storage has {storage.numel()} bytes, the cache needs {nbytes}")
            if device is not None and storage.device.index != device:
                raise ValueError(f"storage is on {storage.device}, not on device {device}")
            device = storage.device.index
        self.device = torch.device("cuda", device or 0)
        self.storage = torch.empty(nbytes, dtype=torch.uint8, device=self.device) if storage is None else storage
        self._cache.data = self.storage.data_ptr()
        self._ws_bytes = {}      # of attend, by (q heads, new tokens); of write, by None: they depend on these alone
        self.ctx = B.upf_create(self.device.index)

    def close(self) -> None:
        if self.ctx:
            torch.cuda.synchronize(self.device)
            B.upf_destroy(self.ctx)
            self.ctx = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def status(self) -> int:
        """Device status word of the context (0 = OK); waits for the current stream."""
        return B.upf_sync_status(self.ctx, self._stream())

    # ------------------------------------------------------------------
    # A call on a few tokens takes a few microseconds on the GPU, so the checks below ask each
    # tensor for its shape and strides once.
    def _stream(self) -> int:
        # the handle of torch.cuda.current_stream(self.device) without the object
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    def _rows(self, name: str, t: torch.Tensor, heads: int) -> int:
        """Check rows of `heads` heads; return the row stride in elements."""
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")
        if t.dtype not in _DTYPES:
            raise ValueError(f"{name} must be bfloat16 or float16, not {t.dtype}")
        shape, d = t.shape, self.head_dim
        if len(shape) != 3 or shape[1] != heads or shape[2] != d:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected [tokens, {heads}, {d}]")
        row, head, dim = t.stride()
        if dim != 1 or (heads > 1 and head != d):
            raise ValueError(f"{name}: the heads of a row must be contiguous (strides {t.stride()})")
        # the stride of a single row is never used and may be anything
        return row if shape[0] > 1 else heads * d

    def _ints(self, name: str, t: Optional[torch.Tensor], dtype: torch.dtype, n: int) -> int:
        if t is None:
            return 0
        if t.device != self.device or t.dtype != dtype or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {self.device}")
        return t.data_ptr()

    # ------------------------------------------------------------------
    def write(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
              num_tokens: Optional[torch.Tensor] = None) -> None:
        """Store ``k``, ``v`` [T, H_kv, d] (rows may be strided) at ``slots`` (int64 [T]; negative: skip).

        ``num_tokens``: device int32 [1]; only that many first tokens are stored (e.g. ``total_kept``)."""
        ks = self._rows("k", k, self.num_kv_heads)
        vs = self._rows("v", v, self.num_kv_heads)
        T = k.shape[0]
        if v.shape[0] != T or v.dtype != k.dtype:
            raise ValueError("k and v disagree on the token count or the type")
        sp = self._ints("slots", slots, torch.int64, T)
        np_ = self._ints("num_tokens", num_tokens, torch.int32, 1)
        wp = wn = 0
        if T > B.UPF_KV_FEW_TOKENS:      # fewer need no workspace
            wn = self._ws_bytes.get(None)
            if wn is None:
                wn = self._ws_bytes[None] = B.upf_kv_write_workspace_bytes(self._cache, T)
            ws = torch.empty(wn, dtype=torch.uint8, device=self.device)
            wp = ws.data_ptr()
        B.upf_kv_write(self.ctx, self._cache, _DTYPES[k.dtype], k.data_ptr(), ks, v.data_ptr(), vs, sp, T, np_, wp, wn,
                       self._stream())

    def read(self, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, num_tokens: Optional[torch.Tensor] = None,
             out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Keys and values [T, H_kv, d] held at ``slots`` (int64 [T]).

        ``out``: the two tensors to fill; rows of skipped tokens (negative slots, or past
        ``num_tokens``) keep what they hold (anything, in new tensors)."""
        T = slots.numel()
        sp = self._ints("slots", slots, torch.int64, T)
        np_ = self._ints("num_tokens", num_tokens, torch.int32, 1)
        if out is None:
            if dtype not in _DTYPES:
                raise ValueError(f"dtype must be bfloat16 or float16, not {dtype}")
            shape = (T, self.num_kv_heads, self.head_dim)
            k = torch.empty(shape, dtype=dtype, device=self.device)
            v = torch.empty(shape, dtype=dtype, device=self.device)
            ks = vs = self.num_kv_heads * self.head_dim
        else:
            k, v = out
            ks = self._rows("out[0]", k, self.num_kv_heads)
            vs = self._rows("out[1]", v, self.num_kv_heads)
            if k.shape[0] != T or v.shape[0] != T or k.dtype != v.dtype:
                raise ValueError("out disagrees with slots on the token count, or its two tensors on the type")
        B.upf_kv_read(self.ctx, self._cache, _DTYPES[k.dtype], sp, T, np_, k.data_ptr(), ks, v.data_ptr(), vs,
                      self._stream())
        return k, v

    def attend(self, q: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor, page_size: int,
               cu_q: Optional[torch.Tensor] = None, max_q_len: int = 1, window: int = 0, sinks: int = 0,
               softmax_scale: Optional[float] = None, kv_of_q: Optional[Sequence[int]] = None,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None) -> AttendOutputs:
        """Attention of ``q`` [tokens, H_q, d] over the cache.

        ``page_table``: int32 [R, max_pages]; ``kv_len``: int32 [R], the new tokens' own entries
        included; ``cu_q``: int32 [R + 1], or None for one new token per request; ``window`` 0: no
        window; ``sinks``: first entries that stay visible beside the window; ``softmax_scale``:
        positive, None for 1/sqrt(d).  Rows of no request keep what ``out`` and ``lse`` hold
        (anything, in new tensors); ``out`` must not overlap ``q`` or the cache."""
        if q.dim() != 3:
            raise ValueError(f"q has shape {tuple(q.shape)}, expected [tokens, H_q, {self.head_dim}]")
        N, Hq, d = q.shape
        qs = self._rows("q", q, Hq)
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.device != self.device:
            raise ValueError(f"page_table must be an int32 [requests, pages] tensor on {self.device}")
        R, pages = page_table.shape
        table_row, table_page = page_table.stride()
        if pages < 1 or (pages > 1 and table_page != 1):
            raise ValueError("page_table needs a page at least, and the pages of a request side by side")
        lp = self._ints("kv_len", kv_len, torch.int32, R)
        cp = self._ints("cu_q", cu_q, torch.int32, R + 1)
        if out is None:
            out = torch.empty((N, Hq, d), dtype=q.dtype, device=self.device)
            outs = Hq * d
        else:
            outs = self._rows("out", out, Hq)
            if out.shape[0] != N or out.dtype != q.dtype:
                raise ValueError("out disagrees with q on the token count or the type")
        if lse is None:
            lse = torch.empty((N, Hq), dtype=torch.float32, device=self.device)
        elif lse.dtype != torch.float32 or lse.shape != (N, Hq) or not lse.is_contiguous() or lse.device != self.device:
            raise ValueError(f"lse must be a contiguous float32 [{N}, {Hq}] tensor on {self.device}")
        if softmax_scale is not None:
            softmax_scale = ctypes.c_float(softmax_scale).value
            if not softmax_scale > 0:
                raise ValueError("softmax_scale must be positive in fp32, or None for 1/sqrt(head_dim)")
        query, keep = B.make_kv_query(R, Hq, N, lp, page_table.data_ptr(), table_row if R > 1 else pages, pages,
                                      page_size, cp, max_q_len, window, sinks, softmax_scale or 0.0, kv_of_q)
        nbytes = self._ws_bytes.get((Hq, max_q_len))
        if nbytes is None:
            nbytes = self._ws_bytes[Hq, max_q_len] = B.upf_kv_attend_workspace_bytes(self._cache, query)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        B.upf_kv_attend(self.ctx, self._cache, query, _DTYPES[q.dtype], q.data_ptr(), qs, out.data_ptr(), outs,
                        lse.data_ptr(), ws.data_ptr(), nbytes, self._stream())
        del keep
        return AttendOutputs(out, lse)
