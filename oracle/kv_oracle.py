"""Float64 oracle of the 4-bit KV cache (test infrastructure only, like ``upf_oracle``).

Written from the definitions: a group of 16 values x is held as e2m1 codes and an
e4m3 scale s = e4m3(min(max|x| 2^-exp / 6, 448)), code = e2m1(x 2^-exp / s), both to
nearest with ties to even; a group with a non-finite value is 16 NaNs.  Attention of a
row at position p over the entries it sees is a plain softmax.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
# every e4m3 number of the codes 0x00 .. 0x7E
E4M3 = [(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)]


def _nearest_even(x: float, numbers: Sequence[float]) -> int:
    """Index of the number nearest to x >= 0; of two as near the one with the even index."""
    i = int(np.searchsorted(numbers, x))
    if i == 0:
        return 0
    if i == len(numbers):
        return i - 1
    lo, hi = x - numbers[i - 1], numbers[i] - x
    return i - 1 if lo < hi or (lo == hi and (i - 1) % 2 == 0) else i


def quantise_group(x: Sequence[float], exp: int) -> Tuple[List[int], int]:
    """(16 codes, scale byte) of 16 values."""
    if not np.all(np.isfinite(x)):
        return [0] * 16, 0x7F
    y = [float(v) * 2.0 ** -exp for v in x]
    sb = _nearest_even(min(max(abs(v) for v in y) / 6, 448.0), E4M3)
    if E4M3[sb] == 0:
        return [0] * 16, 0
    return [_nearest_even(abs(v) / E4M3[sb], E2M1) + (8 if v < 0 else 0) for v in y], sb


def group_values(codes: Sequence[int], sb: int, exp: int) -> np.ndarray:
    s = np.nan if sb == 0x7F else E4M3[sb]
    return np.array([(-1.0 if c & 8 else 1.0) * E2M1[c & 7] * s * 2.0 ** exp for c in codes])


def _nearest_even_all(x: np.ndarray, numbers: Sequence[float]) -> np.ndarray:
    """`_nearest_even` of every element (the midpoints are exact in float64)."""
    n = np.array(numbers)
    mid = (n[1:] + n[:-1]) / 2
    low, high = np.searchsorted(mid, x), np.searchsorted(mid, x, side="right")
    return np.where(low % 2 == 0, low, high)


def cache_values(x: np.ndarray, exp: int) -> np.ndarray:
    """What the cache stands for after x [..., d] was written: `quantise_group` of every group."""
    y = np.asarray(x, dtype=np.float64).reshape(-1, 16) * 2.0 ** -exp
    fine = np.isfinite(y).all(1)
    y = np.where(fine[:, None], y, 0.0)
    s = np.array(E4M3)[_nearest_even_all(np.minimum(np.abs(y).max(1, initial=0.0) / 6, 448.0), E4M3)]
    t = np.divide(np.abs(y), s[:, None], out=np.zeros_like(y), where=s[:, None] > 0)
    v = np.copysign(np.array(E2M1)[_nearest_even_all(t, E2M1)], y) * s[:, None] * 2.0 ** exp
    return np.where(fine[:, None], v, np.nan).reshape(x.shape)


def code_address(d: int, row: int, dim: int, values: bool) -> Tuple[int, int, int]:
    """(byte of the code, 0 or 1 for its low or high nibble, byte of the scale) in a record."""
    D = min(d, 128)
    part, j = divmod(dim, D)
    if not values:
        return part * 16 * (D // 2) + row * (D // 2) + j // 2, j % 2, 16 * d + row * (d // 16) + dim // 16
    half, pair, bit = row // 8, row % 8 // 2, row % 2
    chunk, rest = divmod(j, D // 8)
    code = (((part * 2 + half) * 8 + chunk) * 4 + pair) * 2 + bit
    scale = (((part * 2 + half) * (D // 16) + j // 16) * 4 + pair) * 2 + bit
    return 8 * d + code * (D // 16) + rest // 2, rest % 2, 17 * d + scale


def unpack(storage: np.ndarray, slots: Sequence[int], heads: int, d: int, exp: int, values: bool) -> np.ndarray:
    """[len(slots), heads, d] held in the packed bytes."""
    rec = np.asarray(storage, dtype=np.uint8).reshape(-1, heads, 18 * d)
    where = np.array([[code_address(d, row, j, values) for j in range(d)] for row in range(16)])
    e2m1 = np.array(E2M1 + [-v for v in E2M1])
    e4m3 = np.array(E4M3 + [np.nan])
    out = np.empty((len(slots), heads, d))
    for t, slot in enumerate(slots):
        byte, high, scale = where[slot % 16].T
        r = rec[slot // 16]
        out[t] = e2m1[r[:, byte] >> (4 * high) & 15] * e4m3[r[:, scale] & 0x7F] * 2.0 ** exp
    return out


def visible(n: int, q_len: int, i: int, window: int, sinks: int) -> np.ndarray:
    """Entries of n that new token i of q_len sees."""
    p = n - q_len + i
    e = np.arange(n)
    return e[(e <= p) & ((window == 0) | (p - e < window) | (e < sinks))]


def attend(q: np.ndarray, k: Sequence[np.ndarray], v: Sequence[np.ndarray], cu_q: Sequence[int], window: int = 0,
           sinks: int = 0, scale: Optional[float] = None, kv_of_q: Optional[Sequence[int]] = None):
    """out, lse and the row's bounds of the tolerances: q [N, H_q, d]; k[r], v[r]: [n_r, H_kv, d].

    ``spread`` [N, H_q, d] = sum_e p_e |v_e|; ``total`` [N, H_q, d] = sum_e |v_e|; ``reach`` [N, H_q] = scale * max_e sum |q| |k_e|;
    ``flat`` [N, H_q] = scale * max|q| * max_e sum |k_e|; ``seen`` [N]: entries."""
    q = np.asarray(q, dtype=np.float64)
    N, Hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    out, spread, total = (np.zeros((N, Hq, d)) for _ in range(3))
    lse, reach, flat = np.full((N, Hq), -np.inf), np.zeros((N, Hq)), np.zeros((N, Hq))
    seen = np.zeros(N, dtype=np.int64)
    for r in range(len(cu_q) - 1):
        n, a, b = len(k[r]), cu_q[r], cu_q[r + 1]
        for i in range(b - a):
            e = visible(n, b - a, i, window, sinks)
            seen[a + i] = len(e)
            for h in range(Hq):
                g = h // (Hq // k[r].shape[1]) if kv_of_q is None else kv_of_q[h]
                if not len(e):
                    continue
                ke, ve, row = k[r][e, g], v[r][e, g], q[a + i, h]
                x = ke @ row * scale
                top = x.max()
                w = np.exp(x - top)
                lse[a + i, h] = top + np.log(w.sum())
                w /= w.sum()
                out[a + i, h] = w @ ve
                spread[a + i, h] = w @ np.abs(ve)
                total[a + i, h] = np.abs(ve).sum(0)
                reach[a + i, h] = scale * (np.abs(ke) @ np.abs(row)).max()
                flat[a + i, h] = scale * np.abs(row).max() * np.abs(ke).sum(1).max()
    return out, lse, spread, total, reach, flat, seen
