"""Torch-tensor front end of the rotary positions: table, checks, output allocation and pointer passing.

``RotaryEmbedding`` turns queries and keys by their positions before
``TokenSelector.select_tokens`` scores them and ``QuantKVCache.write`` stores the keys
(``include/upf.h`` has the formulas).  After a selection the positions are those of the kept
tokens (``SelectOutputs.pos_out``, with ``total_kept`` as the device-side count).
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import numpy as np
import torch

from . import _binding as B

_DTYPES = {torch.bfloat16: B.UPF_BF16, torch.float16: B.UPF_F16}
# turns within the original length where the change begins and ends
_BANDS = {"yarn": (1.0, 32.0), "bands": (1.0, 4.0)}


class RotaryEmbedding:
    """The rotation of one attention layer's heads on one GPU, with its own libupf context.

    The first ``rotary_dim`` dims (None: all) of a head of ``head_dim`` turn, in pairs (i, i + rotary_dim / 2), or
    (2i, 2i + 1) if ``interleaved``; pair i by base^(-2i / rotary_dim) radians per position.
    ``scaling``: "none", or "linear", "base", "yarn", "bands" for contexts ``factor`` times as long as
    ``original_len``; ``low`` and ``high``: turns within ``original_len`` between which "yarn" (1, 32) and "bands"
    (1, 4) go from divided to kept frequencies.  ``divisors``: what each pair's frequency is divided by.
    ``magnitude``: what sines and cosines are multiplied by (None: 0.1 ln factor + 1 for "yarn", else 1).
    Calls run on the current stream of the device."""

    def __init__(self, head_dim: int, rotary_dim: Optional[int] = None, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, original_len: float = 0.0, low: Optional[float] = None,
                 high: Optional[float] = None, divisors: Optional[Sequence[float]] = None,
                 magnitude: Optional[float] = None, device: int = 0):
        self.ctx = 0
        if magnitude is not None and not magnitude > 0:
            raise ValueError("magnitude must be positive, or None")
        ends = _BANDS.get(scaling, (0.0, 0.0))
        self._rope, self._keep = B.make_rope(
            head_dim, head_dim if rotary_dim is None else rotary_dim, base, interleaved, scaling, factor, original_len,
            ends[0] if low is None else low, ends[1] if high is None else high, divisors, magnitude or 0.0)
        turns, self.magnitude = B.upf_rope_turns(self._rope)
        self.head_dim, self.rotary_dim = head_dim, self._rope.rotary_dim
        self.device = torch.device("cuda", device)
        self.turns = torch.from_numpy(turns.view(np.int64)).to(self.device)   # fractions of a turn, in units of 2^-64
        self.ctx = B.upf_create(device)

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

    def _rows(self, name: str, t: torch.Tensor) -> int:
        """Check rows of heads; return the row stride in elements."""
        shape, d = t.shape, self.head_dim
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the rotation on {self.device}")
        if len(shape) != 3 or shape[2] != d:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected [tokens, heads, {d}]")
        row, head, dim = t.stride()
        if dim != 1 or (shape[1] > 1 and head != d):
            raise ValueError(f"{name}: the heads of a row must be contiguous (strides {t.stride()})")
        # the stride of a single row is never used and may be anything
        return row if shape[0] > 1 else shape[1] * d

    def _side(self, name: str, t: Optional[torch.Tensor], out: Optional[torch.Tensor], T: int, dtype: torch.dtype):
        if t is None:
            if out is not None:
                raise ValueError(f"out has a tensor for {name}, which is None")
            return 0, 0, 0, 0, 0, None
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
        stride = self._rows(name, t)
        if t.shape[0] != T:
            raise ValueError(f"{name} has {t.shape[0]} tokens, positions {T}")
        if out is None:
            out = torch.empty_like(t, memory_format=torch.contiguous_format)
            out_stride = t.shape[1] * self.head_dim
        elif out is t:
            out_stride = stride
        else:
            out_stride = self._rows(f"out of {name}", out)
            if out.shape != t.shape or out.dtype != dtype:
                raise ValueError(f"out of {name} must have its shape and type")
        return t.data_ptr(), stride, out.data_ptr(), out_stride, t.shape[1], out

    def apply(self, q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: torch.Tensor,
              num_tokens: Optional[torch.Tensor] = None,
              out: Optional[Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]] = None,
              inverse: bool = False) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
        """``q`` [T, H_q, d] and ``k`` [T, H_kv, d] (either may be None; rows may be strided), turned by
        ``positions`` (int64 [T], any values).

        ``num_tokens``: device int32 [1]; only that many first tokens are done (e.g. ``total_kept``), rows past
        them keep what ``out`` holds (anything, in new tensors).  ``out``: the two tensors to fill; they may be
        ``q`` and ``k`` themselves, and must not overlap them otherwise.  ``inverse``: turn back, and divide by
        the magnitude."""
        some = k if q is None else q
        if some is None:
            raise ValueError("q or k must be given")
        dtype = some.dtype
        if dtype not in _DTYPES:
            raise ValueError(f"{'k' if q is None else 'q'} must be bfloat16 or float16, not {dtype}")
        if positions.device != self.device or positions.dtype != torch.int64 or positions.dim() != 1 or \
                not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous torch.int64 vector on {self.device}")
        T = positions.shape[0]
        count = 0
        if num_tokens is not None:
            if num_tokens.device != self.device or num_tokens.dtype != torch.int32 or num_tokens.numel() != 1:
                raise ValueError(f"num_tokens must be a torch.int32 tensor of one element on {self.device}")
            count = num_tokens.data_ptr()
        q_out, k_out = (None, None) if out is None else out
        qp, qs, qop, qos, hq, q_out = self._side("q", q, q_out, T, dtype)
        kp, ks, kop, kos, hk, k_out = self._side("k", k, k_out, T, dtype)
        B.upf_rope_apply(self.ctx, self._rope, self.turns.data_ptr(), 1 if inverse else 0, _DTYPES[dtype],
                         positions.data_ptr(), T, count, qp, qs, qop, qos, hq, kp, ks, kop, kos, hk,
                         torch._C._cuda_getCurrentRawStream(self.device.index))
        return q_out, k_out
