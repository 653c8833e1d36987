"""Oracle of the rotary positions (test infrastructure only).

Frequencies come from the definitions in 60-digit decimals; an angle is position times frequency,
reduced to one turn exactly, in rational numbers.
"""
from __future__ import annotations

from decimal import Decimal, getcontext
from fractions import Fraction
from typing import List, Optional, Sequence

import numpy as np

getcontext().prec = 60
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def frequencies(rotary_dim: int, base: float, scaling: str = "none", factor: float = 1.0, original_len: float = 0.0,
                low: float = 0.0, high: float = 0.0, divisors: Optional[Sequence[float]] = None) -> List[Decimal]:
    """Radians per position of each pair."""
    n, b, s, length = rotary_dim, Decimal(base), Decimal(factor), Decimal(original_len)
    if scaling == "base" and n > 2:
        b *= s ** (Decimal(n) / (n - 2))
    out = []
    for i in range(n // 2):
        f = b ** (Decimal(-2 * i) / n)
        keep = Decimal(1)
        if scaling == "linear":
            keep = Decimal(0)
        elif scaling == "bands":
            keep = (length * f / TWO_PI - Decimal(low)) / (Decimal(high) - Decimal(low))
        elif scaling == "yarn":
            # the pair that makes t turns: length b^(-2 i / n) / 2 pi = t
            at = [n * (length / (Decimal(t) * TWO_PI)).ln() / (2 * b.ln()) for t in (high, low)]
            first = max(int(at[0].to_integral_value("ROUND_FLOOR")), 0)
            last = min(int(at[1].to_integral_value("ROUND_CEILING")), n - 1)
            keep = 1 - (Decimal(i - first) / max(Decimal(last - first), Decimal("0.001")))
        keep = min(max(keep, Decimal(0)), Decimal(1))
        f = f * keep + f / s * (1 - keep)
        out.append(f / Decimal(divisors[i]) if divisors is not None else f)
    return out


def angles(positions: Sequence[int], turns: Sequence[int]) -> np.ndarray:
    """Angles in [0, 2 pi) of positions times fractions of a turn in units of 2^-64."""
    return np.array([[float(Fraction(int(p) * int(t) % 2 ** 64, 2 ** 64)) * 2 * np.pi for t in turns] for p in positions])


def rotate(x: np.ndarray, angle: np.ndarray, rotary_dim: int, interleaved: bool, magnitude: float = 1.0,
           inverse: bool = False) -> np.ndarray:
    """x [T, H, d] float64, angle [T, rotary_dim / 2]."""
    y = np.array(x, dtype=np.float64)
    for i in range(rotary_dim // 2):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)
        c, s = np.cos(angle[:, None, i]), np.sin(angle[:, None, i])
        m = magnitude
        if inverse:
            s, m = -s, 1 / magnitude
        y[..., p], y[..., q] = m * (x[..., p] * c - x[..., q] * s), m * (x[..., q] * c + x[..., p] * s)
    return y
