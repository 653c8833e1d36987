"""Rotary positions without a GPU: pins of the oracle, the table, and refusals before any launch."""
import ctypes
import math
from decimal import Decimal

import numpy as np
import pytest

from oracle import rope_oracle as O
from sparse_long_context_tail_gb300 import _binding as B
from sparse_long_context_tail_gb300 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


KINDS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
         dict(scaling="yarn", factor=16.0, original_len=4096, low=1, high=32),
         dict(scaling="yarn", factor=0.5, original_len=300, low=2, high=3),
         dict(scaling="bands", factor=8.0, original_len=8192, low=1, high=4),
         dict(scaling="linear", factor=2.0, divisors=True), dict(divisors=True)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,base", [(2, 10000.0), (6, 10000.0), (64, 10000.0), (128, 500000.0), (256, 1e7)])
def test_table_is_the_frequencies_in_turns(n, base, kind):
    kind = dict(kind)
    if kind.get("divisors"):
        kind["divisors"] = 1.0 + 0.37 * np.arange(n // 2)
    rope, keep = B.make_rope(256, n, base, **kind)
    turns, magnitude = B.upf_rope_turns(rope)
    want = O.frequencies(n, base, **kind)
    assert len(turns) == len(want)
    for t, f in zip(turns, want):
        turn = f / O.TWO_PI % 1
        # a pow, a division, up to five more roundings of the frequency, and 2^-64 of the table itself
        assert abs(Decimal(int(t)) / 2 ** 64 - turn) <= f * Decimal(2) ** -49 + Decimal(2) ** -64, (n, base, kind)
    assert magnitude == (0.1 * math.log(kind["factor"]) + 1 if kind.get("scaling") == "yarn" and kind["factor"] > 1 else 1)


def test_frequency_rules_by_hand():
    assert [float(f) for f in O.frequencies(4, 100.0)] == pytest.approx([1, 0.1])
    assert [float(f) for f in O.frequencies(4, 100.0, "linear", 2.0)] == pytest.approx([0.5, 0.05])
    # a new base whose last pair is as if its positions were interpolated
    for n in (4, 64):
        assert float(O.frequencies(n, 1e4, "base", 8.0)[-1]) == pytest.approx(float(O.frequencies(n, 1e4)[-1]) / 8)
        assert float(O.frequencies(n, 1e4, "base", 8.0)[0]) == 1
    for scaling, high in (("yarn", 32), ("bands", 4)):   # the fastest pair is kept, the slowest divided
        f = O.frequencies(128, 5e5, scaling, 8.0, 8192, 1, high)
        g = O.frequencies(128, 5e5)
        assert f[0] == g[0] and abs(f[-1] - g[-1] / 8) < Decimal(10) ** -50
        assert all(b / 8 <= a * (1 + Decimal(10) ** -50) and a <= b for a, b in zip(f, g))
        assert all(a >= b for a, b in zip(f, f[1:]))
    # half way between one turn and four, half way between f and f / 8
    f = float(O.frequencies(2, 1e4, "bands", 8.0, 2.5 * 2 * math.pi, 1, 4)[0])
    assert f == pytest.approx((1 + 1 / 8) / 2)


def test_rotation_by_hand():
    x = np.arange(8.0).reshape(1, 1, 8)
    quarter = np.full((1, 2), np.pi / 2)
    assert np.allclose(O.rotate(x, quarter, 4, False)[0, 0], [-2, -3, 0, 1, 4, 5, 6, 7])
    assert np.allclose(O.rotate(x, quarter, 4, True)[0, 0], [-1, 0, -3, 2, 4, 5, 6, 7])
    assert np.allclose(O.rotate(x, quarter, 4, True, 3.0)[0, 0], [-3, 0, -9, 6, 4, 5, 6, 7])
    y = O.rotate(x, quarter * 0.3, 8 // 2, False, 3.0)
    assert np.allclose(O.rotate(y, quarter * 0.3, 4, False, 3.0, inverse=True), x)
    assert np.allclose(O.angles([1, -1, 5], [2 ** 62]), np.array([[0.5], [1.5], [0.5]]) * np.pi)


def test_frequencies_above_a_turn_and_magnitudes():
    rope, keep = B.make_rope(64, 2, 10000.0, divisors=[1 / (2 * np.pi * 2.25)])
    turns, m = B.upf_rope_turns(rope)
    assert abs(int(turns[0]) - 2 ** 62) <= 2 ** 13 and m == 1      # two turns and a quarter a position
    rope, keep = B.make_rope(64, 64, magnitude=1.25)
    assert B.upf_rope_turns(rope)[1] == 1.25


BAD = [(dict(head_dim=96), "head_dim"), (dict(rotary_dim=0), "rotary_dim"), (dict(rotary_dim=130), "rotary_dim"),
       (dict(rotary_dim=63), "rotary_dim"), (dict(base=0.0), "base"), (dict(base=-1.0), "base"),
       (dict(base=float("inf")), "base"), (dict(base=float("nan")), "base"), (dict(magnitude=-1.0), "magnitude"),
       (dict(magnitude=float("nan")), "magnitude"), (dict(scaling="linear", factor=0.0), "factor"),
       (dict(scaling="base", factor=float("nan")), "factor"), (dict(scaling="bands", factor=2.0, low=1, high=4), "original_len"),
       (dict(scaling="bands", factor=2.0, original_len=64, low=4, high=4), "low"),
       (dict(scaling="yarn", factor=2.0, original_len=64, low=0, high=4), "low"),
       (dict(scaling="yarn", factor=2.0, original_len=64, low=1, high=4, base=1.0), "base"),
       (dict(divisors=[0.0] * 64), "divisors"), (dict(divisors=[float("nan")] * 64), "divisors"),
       (dict(base=1e-300, rotary_dim=128, divisors=[1e-300] * 64), "frequency")]


@pytest.mark.parametrize("bad,word", BAD)
def test_rotations_that_are_refused(bad, word):
    a = dict(head_dim=128, rotary_dim=128)
    a.update(bad)
    rope, keep = B.make_rope(**a)
    with pytest.raises(B.UpfError) as e:
        B.upf_rope_turns(rope)
    assert word in e.value.message, e.value.message
    if word not in ("divisors", "frequency"):      # those of the table alone
        with pytest.raises(B.UpfError) as e:
            B.upf_rope_apply(None, rope, 256, 0, 0, 8, 1, 0, 256, 1024, 4096, 1024, 1, 0, 0, 0, 0, 0)
        assert word in e.value.message, e.value.message


def test_structs_that_the_binding_refuses():
    with pytest.raises(ValueError, match="scaling"):
        B.make_rope(128, 128, scaling="other")
    with pytest.raises(ValueError, match="divisors"):
        B.make_rope(128, 128, divisors=[1.0] * 63)
    with pytest.raises(ValueError, match="32 bits"):
        B.make_rope(128, 128 + 2 ** 32)
    assert B.load().upf_rope_turns(None, None, None) == 1 and "NULL" in B.upf_last_error()
    rope, keep = B.make_rope(128, 128)
    assert B.load().upf_rope_turns(ctypes.byref(rope), None, None) == 1 and "turns" in B.upf_last_error()


CALL = dict(turns=256, inverse=0, dtype=0, positions=8, num_tokens=16, count=0, q=0x10000, q_row_stride=512, q_out=0x80000,
            q_out_row_stride=512, num_q_heads=4, k=0x20000, k_row_stride=256, k_out=0x90000, k_out_row_stride=256,
            num_kv_heads=2)
BAD_CALLS = [(dict(), "context"), (dict(dtype=2), "dtype"), (dict(num_tokens=-1), "num_tokens"),
             (dict(num_tokens=2 ** 30 + 1), "num_tokens"), (dict(num_q_heads=-1), "heads"),
             (dict(num_kv_heads=65537), "heads"), (dict(num_q_heads=0, num_kv_heads=0), "heads"), (dict(q=0), "q"),
             (dict(q=0x10008), "aligned"), (dict(k_out=0x90004), "k_out"), (dict(q_row_stride=504), "stride"),
             (dict(q_row_stride=516), "stride"), (dict(k_out_row_stride=248), "stride"), (dict(positions=0), "positions"),
             (dict(turns=0), "turns"), (dict(turns=264), "turns"),
             # outputs over inputs of the other, over their own with another stride or a few rows on, over each other
             (dict(q_out=0x20000), "overlaps"), (dict(k_out=0x10000, k_out_row_stride=512), "overlaps"),
             (dict(q_out=0x10000, q_out_row_stride=520), "overlaps"), (dict(q_out=0x10400), "overlaps"),
             (dict(k_out=0x80000), "overlap"), (dict(k_out=0x80200, k_out_row_stride=512), "overlap")]


def _apply(**kw):
    a = dict(CALL)
    a.update(kw)
    rope, keep = B.make_rope(128, 128)
    B.upf_rope_apply(None, rope, a["turns"], a["inverse"], a["dtype"], a["positions"], a["num_tokens"], a["count"], a["q"],
                     a["q_row_stride"], a["q_out"], a["q_out_row_stride"], a["num_q_heads"], a["k"], a["k_row_stride"],
                     a["k_out"], a["k_out_row_stride"], a["num_kv_heads"])


@pytest.mark.parametrize("bad,word", BAD_CALLS)
def test_calls_that_are_refused(bad, word):
    with pytest.raises(B.UpfError) as e:
        _apply(**bad)
    assert word in e.value.message, e.value.message


# these get as far as the missing context
@pytest.mark.parametrize("good", [
    dict(num_tokens=0, q=0, positions=0), dict(num_q_heads=0, q=0, q_out=3), dict(num_kv_heads=0, k=0),
    dict(q_out=0x10000, k_out=0x20000),                                           # in place
    dict(num_tokens=1, q_out=0x10000, q_out_row_stride=1024),                     # one row: its stride says nothing
    # heads side by side in one projection's rows, in place and into another
    dict(q=0x10000, q_row_stride=1024, q_out=0x10000, q_out_row_stride=1024, k=0x10400, k_row_stride=1024, k_out=0x10400,
         k_out_row_stride=1024),
    dict(q_out=0x80000, q_out_row_stride=768, k_out=0x80400, k_out_row_stride=768)])
def test_calls_that_are_not_refused(good):
    with pytest.raises(B.UpfError) as e:
        _apply(**good)
    assert "context" in e.value.message, e.value.message


@pytest.mark.parametrize("n,base,kind", [(256, 1e7, dict(scaling="linear", factor=32.0)), (128, 5e5, dict(scaling="linear", factor=8.0)),
                                         (128, 5e5, dict(scaling="base", factor=8.0)), (128, 1e4, dict()),
                                         (128, 5e5, dict(scaling="bands", factor=32.0, original_len=8192, low=1, high=4)),
                                         (64, 1e6, dict(scaling="yarn", factor=40.0, original_len=32768, low=1, high=32))])
def test_angles_at_any_position_are_as_near_as_the_header_says(n, base, kind):
    """Positions times the table modulo a turn, against 60-digit decimals: |position| (2^-64 + 2^-50 f / 2 pi) of a turn."""
    rope, keep = B.make_rope(256, n, base, **kind)
    turns, _ = B.upf_rope_turns(rope)
    for t, f in zip(turns, O.frequencies(n, base, **kind)):
        for p in (1, 131071, 2 ** 31 - 1, 2 ** 40 + 7):
            off = (Decimal(p * int(t) % 2 ** 64) / 2 ** 64 - p * f / O.TWO_PI) % 1
            off = min(abs(off), abs(1 - abs(off)))
            assert off <= p * (Decimal(2) ** -64 + Decimal(2) ** -50 * f / O.TWO_PI), (p, f)


@pytest.mark.parametrize("bad,word", [(dict(positions=12), "positions"), (dict(positions=9), "positions"), (dict(count=6), "num_tokens_dev"),
                                      (dict(count=1), "num_tokens_dev")])
def test_misaligned_positions_and_counts_are_refused(bad, word):
    with pytest.raises(B.UpfError, match=f"{word} must be"):
        _apply(**bad)
