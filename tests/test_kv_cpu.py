"""The 4-bit KV cache without a GPU: pins of its oracle, sizes, and refusals before any launch."""
import itertools
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from sparse_long_context_tail_gb300 import _binding as B
from sparse_long_context_tail_gb300 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


# ------------------------------------------------------------------ oracle --

def test_number_tables():
    byte = torch.arange(127, dtype=torch.uint8)
    assert K.E4M3 == byte.view(torch.float8_e4m3fn).double().tolist()
    # a 4-bit float: two exponent bits (bias 1), one fraction bit
    assert K.E2M1 == [m / 2 if e == 0 else 2.0 ** (e - 1) * (1 + m / 2) for e, m in itertools.product(range(4), range(2))]


def test_codes_are_the_nearest_numbers_and_ties_are_even():
    rng = np.random.default_rng(0)
    for _ in range(200):
        x = (rng.standard_normal(16) * 2.0 ** rng.integers(-6, 6)).astype(np.float16).astype(float)
        codes, sb = K.quantise_group(x, 0)
        want = Fraction(max(abs(v) for v in x)) / 6
        assert abs(Fraction(K.E4M3[sb]) - want) == min(abs(Fraction(s) - want) for s in K.E4M3)
        if K.E4M3[sb] == 0:
            assert codes == [0] * 16
            continue
        for c, v in zip(codes, x):
            t = Fraction(v) / Fraction(K.E4M3[sb])
            near = [abs(abs(t) - Fraction(m)) for m in K.E2M1]
            assert near[c & 7] == min(near) and (c & 7 == 0 or (c >> 3 == 1) == (v < 0))
            if near.count(min(near)) == 2:
                assert (c & 7) % 2 == 0
    # amax 6: scale 1; the seven ties go to 0, 1, 1, 2, 2, 4, 4
    codes, sb = K.quantise_group([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0, 0, 0, 0, 0], 0)
    assert K.E4M3[sb] == 1 and K.group_values(codes, sb, 0)[:11].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -4]
    assert K.quantise_group([1.0] * 15 + [np.inf], 0) == ([0] * 16, 0x7F)
    assert K.quantise_group([0.0] * 16, 0) == ([0] * 16, 0)
    assert K.quantise_group([1e6] * 16, 0) == ([7] * 16, 0x7E) and K.group_values([7], 0x7E, 1)[0] == 6 * 448 * 2
    assert K.quantise_group([6.0 * 2.0 ** 5] * 16, 5) == K.quantise_group([6.0] * 16, 0)


def test_whole_arrays_are_quantised_group_by_group():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((200, 64)) * 2.0 ** rng.integers(-12, 12, (200, 1))).astype(np.float16).astype(float)
    x[0, 3], x[1, 20] = np.nan, np.inf
    x[2] = np.tile([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, 0], 4)
    for exp in (-3, 0, 5):
        want = [K.group_values(*K.quantise_group(g, exp), exp) for g in x.reshape(-1, 16)]
        np.testing.assert_array_equal(K.cache_values(x, exp), np.stack(want).reshape(x.shape))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_record_addresses_are_a_bijection(d):
    where = [K.code_address(d, row, j, of) for of in (False, True) for row in range(16) for j in range(d)]
    assert len({(b, h) for b, h, _ in where}) == 32 * d
    assert {b for b, _, _ in where} == set(range(16 * d))
    assert {s for _, _, s in where} == set(range(16 * d, 18 * d))
    for row in range(16):      # the sixteen dims of a group share a scale, other groups have others
        for of in (False, True):
            s = [K.code_address(d, row, j, of)[2] for j in range(d)]
            assert all(len(set(s[j:j + 16])) == 1 for j in range(0, d, 16)) and len(set(s)) == d // 16


def test_visible_entries():
    assert K.visible(5, 1, 0, 0, 0).tolist() == [0, 1, 2, 3, 4]
    assert K.visible(5, 2, 0, 0, 3).tolist() == [0, 1, 2, 3]
    assert K.visible(9, 1, 0, 2, 0).tolist() == [7, 8] and K.visible(9, 1, 0, 2, 3).tolist() == [0, 1, 2, 7, 8]
    assert K.visible(4, 1, 0, 3, 3).tolist() == [0, 1, 2, 3]
    assert K.visible(1, 3, 0, 0, 0).tolist() == [] and K.visible(1, 3, 2, 0, 0).tolist() == [0]
    assert K.visible(0, 1, 0, 4, 2).tolist() == []


def test_attention_closed_forms():
    v = np.arange(12.0).reshape(3, 1, 4)
    out, lse, *_ = K.attend(np.zeros((1, 2, 4)), [np.ones((3, 1, 4))], [v], [0, 1])
    assert np.allclose(out[0], v.mean(0)) and np.allclose(lse, np.log(3))
    out, lse, *_ = K.attend(np.ones((2, 1, 4)), [np.zeros((0, 1, 4))], [np.zeros((0, 1, 4))], [0, 2])
    assert not out.any() and np.isneginf(lse).all()
    k = np.array([[[1.0, 0]], [[0, 2.0]]])
    out, lse, *_ = K.attend(np.array([[[1.0, 1]]]), [k], [k], [0, 1], scale=1.0)
    assert np.allclose(lse, np.log(np.exp(1) + np.exp(2)))
    assert np.allclose(out[0, 0], [np.exp(1 - lse[0, 0]), 2 * np.exp(2 - lse[0, 0])])


# -------------------------------------------------------------- host refusals --

def _cache(**kw):
    a = dict(data=0x1000, num_slots=64, num_kv_heads=2, head_dim=128, k_exp=0, v_exp=0)
    a.update(kw)
    return B.make_kv_cache(**a)


def _query(**kw):
    a = dict(num_reqs=2, num_q_heads=4, num_q_tokens=2, kv_len=0x100, page_table=0x100, page_stride=4, max_pages=4,
             page_size=16)
    a.update(kw)
    return B.make_kv_query(**a)


def test_sizes():
    for d in (64, 128, 256):
        assert B.upf_kv_cache_bytes(_cache(head_dim=d)) == 64 // 16 * 2 * 18 * d
    assert B.upf_kv_write_workspace_bytes(_cache(), 0) > 0
    x, keep = _query()
    assert B.upf_kv_attend_workspace_bytes(_cache(), x) > 0


BAD_CACHES = [(dict(num_slots=0), "num_slots"), (dict(num_slots=40), "num_slots"), (dict(num_slots=-16), "num_slots"),
              (dict(num_slots=1 << 37), "num_slots"), (dict(num_kv_heads=0), "num_kv_heads"),
              (dict(num_kv_heads=257), "num_kv_heads"), (dict(head_dim=96), "head_dim"), (dict(k_exp=33), "k_exp"),
              (dict(v_exp=-33), "v_exp")]


@pytest.mark.parametrize("bad,word", BAD_CACHES)
def test_caches_that_are_refused(bad, word):
    c = _cache(**bad)
    x, keep = _query()
    for call in (lambda: B.upf_kv_cache_bytes(c), lambda: B.upf_kv_write_workspace_bytes(c, 1),
                 lambda: B.upf_kv_attend_workspace_bytes(c, x),
                 lambda: B.upf_kv_write(None, c, 0, 16, 256, 16, 256, 8, 1, 0, 256, 1 << 30),
                 lambda: B.upf_kv_read(None, c, 0, 8, 1, 0, 16, 256, 16, 256),
                 lambda: B.upf_kv_attend(None, c, x, 0, 16, 512, 16, 512, 0, 256, 1 << 30)):
        with pytest.raises(B.UpfError) as e:
            call()
        assert word in e.value.message, e.value.message


BAD_QUERIES = [(dict(num_reqs=0), "num_reqs"), (dict(num_q_heads=3), "H_q"), (dict(num_q_heads=0), "H_q"),
               (dict(num_q_heads=258), "num_q_heads"), (dict(kv_of_q=[0, 0, 0, 1]), "kv_of_q"),
               (dict(kv_of_q=[0, 0, 1, 2]), "kv_of_q"), (dict(num_q_tokens=-1), "num_q_tokens"),
               (dict(max_q_len=0), "max_q_len"), (dict(max_q_len=1025), "max_q_len"), (dict(page_size=8), "page_size"),
               (dict(page_size=48), "page_size"), (dict(page_size=1 << 17), "page_size"), (dict(max_pages=0), "max_pages"),
               (dict(max_pages=1 << 27), "max_pages"), (dict(window=-1), "window"), (dict(sinks=-1), "sinks"),
               (dict(softmax_scale=float("nan")), "softmax_scale"), (dict(softmax_scale=float("inf")), "softmax_scale")]


@pytest.mark.parametrize("bad,word", BAD_QUERIES)
def test_queries_that_are_refused(bad, word):
    x, keep = _query(**bad)
    for call in (lambda: B.upf_kv_attend_workspace_bytes(_cache(), x),
                 lambda: B.upf_kv_attend(None, _cache(), x, 0, 16, 512, 16, 512, 0, 256, 1 << 30)):
        with pytest.raises(B.UpfError) as e:
            call()
        assert word in e.value.message, e.value.message


@pytest.mark.parametrize("query,args,word", [
    (dict(kv_len=0), {}, "kv_len"), (dict(page_table=0), {}, "page_table"), (dict(page_stride=3), {}, "page_stride"),
    (dict(num_q_tokens=3), {}, "cu_q"), ({}, dict(dtype=2), "dtype"), ({}, dict(q=0), "q "), ({}, dict(q=24), "q "),
    ({}, dict(qs=511), "stride"), ({}, dict(qs=508), "stride"), ({}, dict(out=0), "out"), ({}, dict(out=8), "out"),
    ({}, dict(outs=256), "stride"), ({}, dict(ws=0), "workspace"), ({}, dict(ws=128), "workspace"),
    ({}, dict(nbytes=1), "workspace"), ({}, {}, "context")])
def test_attend_calls_that_are_refused(query, args, word):
    x, keep = _query(**query)
    a = dict(dtype=0, q=16, qs=512, out=16, outs=512, ws=256, nbytes=1 << 30)
    a.update(args)
    with pytest.raises(B.UpfError) as e:
        B.upf_kv_attend(None, _cache(), x, a["dtype"], a["q"] or None, a["qs"], a["out"] or None, a["outs"], 0,
                        a["ws"] or None, a["nbytes"])
    assert e.value.status == 1 and word in e.value.message, e.value.message


@pytest.mark.parametrize("args,word", [
    (dict(dtype=-1), "dtype"), (dict(k=0), "k "), (dict(k=8), "k "), (dict(ks=128), "stride"), (dict(ks=260), "stride"),
    (dict(v=0), "v "), (dict(vs=0), "stride"), (dict(slots=0), "slots"), (dict(T=-1), "num_tokens"),
    (dict(T=(1 << 30) + 1), "num_tokens"), (dict(T=2000, ws=0), "workspace"), (dict(T=2000, nbytes=0), "workspace"),
    (dict(T=2000, ws=64), "workspace"), (dict(T=0), "context"), (dict(ws=0, nbytes=0), "context"), ({}, "context")])
def test_write_calls_that_are_refused(args, word):
    a = dict(dtype=0, k=16, ks=256, v=16, vs=256, slots=8, T=4, ws=256, nbytes=1 << 20)
    a.update(args)
    with pytest.raises(B.UpfError) as e:
        B.upf_kv_write(None, _cache(), a["dtype"], a["k"] or None, a["ks"], a["v"] or None, a["vs"], a["slots"] or None,
                       a["T"], 0, a["ws"] or None, a["nbytes"])
    assert e.value.status == 1 and word in e.value.message, e.value.message


@pytest.mark.parametrize("args,word", [
    (dict(dtype=7), "dtype"), (dict(k=0, v=0), "both NULL"), (dict(k=8), "k "), (dict(ks=128), "stride"),
    (dict(v=8), "v "), (dict(vs=257), "stride"), (dict(slots=0), "slots"), (dict(T=-5), "num_tokens"),
    (dict(k=0, ks=0), "context"), (dict(v=0, vs=0), "context"), (dict(T=0), "context")])
def test_read_calls_that_are_refused(args, word):
    a = dict(dtype=1, k=16, ks=256, v=16, vs=256, slots=8, T=4)
    a.update(args)
    with pytest.raises(B.UpfError) as e:
        B.upf_kv_read(None, _cache(), a["dtype"], a["slots"] or None, a["T"], 0, a["k"], a["ks"], a["v"], a["vs"])
    assert e.value.status == 1 and word in e.value.message, e.value.message


def test_cache_data_is_checked():
    for data in (0, 64):
        with pytest.raises(B.UpfError) as e:
            B.upf_kv_read(None, _cache(data=data), 0, 8, 1, 0, 16, 256, 16, 256)
        assert "data" in e.value.message


# --------------------------------------------------------------- front end --

@pytest.fixture
def front():
    """A QuantKVCache without a context, on the CPU: its own checks run, then the library refuses."""
    from sparse_long_context_tail_gb300.kvcache import QuantKVCache
    c = QuantKVCache.__new__(QuantKVCache)
    c.ctx, c.num_slots, c.num_kv_heads, c.head_dim, c.device = 0, 64, 2, 128, torch.device("cpu")
    c._cache = _cache()
    return c


def _kv(T=3, H=2, d=128, dtype=torch.bfloat16):
    return torch.zeros(T, H, d, dtype=dtype)


def test_front_end_write_and_read_refusals(front):
    s = torch.zeros(3, dtype=torch.int64)
    for k, v, slots, n in ((_kv(), _kv(4), s, None), (_kv(), _kv(dtype=torch.float16), s, None),
                           (_kv(dtype=torch.float32), _kv(), s, None), (_kv(H=1), _kv(), s, None),
                           (_kv(d=64), _kv(), s, None), (_kv()[0], _kv(), s, None), (_kv(), _kv(), s.int(), None),
                           (_kv(), _kv(), s[:2], None), (_kv(), _kv(), torch.zeros(6, dtype=torch.int64)[::2], None),
                           (_kv(), _kv(), s, torch.zeros(1, dtype=torch.int64)),
                           (_kv(), _kv(), s, torch.zeros(2, dtype=torch.int32)),
                           (_kv(H=4)[:, ::2], _kv(), s, None), (_kv().transpose(1, 2).contiguous().transpose(1, 2), _kv(), s, None)):
        with pytest.raises(ValueError):
            front.write(k, v, slots, n)
    for kw in (dict(slots=s.int()), dict(slots=s, dtype=torch.float32), dict(slots=s, out=(_kv(), _kv(2))),
               dict(slots=s, out=(_kv(), _kv(dtype=torch.float16)))):
        with pytest.raises(ValueError):
            front.read(**kw)


def test_front_end_attend_refusals(front):
    good = dict(q=_kv(2, 4), page_table=torch.zeros(2, 4, dtype=torch.int32), kv_len=torch.zeros(2, dtype=torch.int32),
                page_size=16)
    for bad in (dict(q=_kv(2, 4)[0]), dict(q=_kv(2, 4, 64)), dict(q=_kv(2, 4, dtype=torch.float32)),
                dict(page_table=torch.zeros(2, 4, dtype=torch.int64)), dict(page_table=torch.zeros(8, dtype=torch.int32)),
                dict(page_table=torch.zeros(4, 2, dtype=torch.int32).t()), dict(page_table=torch.zeros(2, 0, dtype=torch.int32)),
                dict(kv_len=torch.zeros(3, dtype=torch.int32)), dict(kv_len=torch.zeros(2, dtype=torch.int64)),
                dict(cu_q=torch.zeros(2, dtype=torch.int32)), dict(out=_kv(1, 4)), dict(out=_kv(2, 4, dtype=torch.float16)),
                dict(lse=torch.zeros(2, 3)), dict(lse=torch.zeros(2, 4, dtype=torch.float64))):
        with pytest.raises(ValueError):
            front.attend(**{**good, **bad})


@pytest.mark.parametrize("heads", [[], [0, 0, 1], [0, 0, 1, 1, 1], [[0, 0], [1, 1]]])
def test_head_maps_of_another_length_are_refused(front, heads):
    """The library reads num_q_heads entries of the map: a shorter one would be read past its end."""
    with pytest.raises(ValueError, match="kv_of_q"):
        _query(kv_of_q=heads)
    with pytest.raises(ValueError, match="kv_of_q"):
        front.attend(_kv(2, 4), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 16, kv_of_q=heads)
    _query(kv_of_q=torch.tensor([0, 1, 0, 1]))


@pytest.mark.parametrize("scale", [0, 0.0, -0.125, float("nan"), 1e-60])
def test_scales_that_are_not_positive_are_refused(front, scale):
    """None selects 1/sqrt(head_dim), which the library takes from a scale that is not positive (1e-60 is 0 in fp32)."""
    args = _kv(2, 4), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 16
    front._ws_bytes = {(4, 1): 256}
    front._stream = lambda: 0
    with pytest.raises(ValueError, match="softmax_scale"):
        front.attend(*args, softmax_scale=scale)
    for good in (None, 0.5, 1e-40):
        with pytest.raises(B.UpfError) as e:      # past the front end's checks: the library refuses the null context
            front.attend(*args, softmax_scale=good)
        assert "softmax_scale" not in e.value.message


@pytest.mark.parametrize("name", ["max_q_len", "page_size", "window", "sinks"])
def test_sizes_past_32_bits_are_refused(front, name):
    """The C structure holds 32 bits: a larger number would be cut down to another one."""
    args = dict(q=_kv(2, 4), page_table=torch.zeros(2, 4, dtype=torch.int32), kv_len=torch.zeros(2, dtype=torch.int32), page_size=16)
    for value in (2 ** 32 + 16, -2 ** 32 + 16, 2 ** 31):
        with pytest.raises(ValueError, match=name):
            front.attend(**{**args, name: value})
        with pytest.raises(ValueError, match=name):
            _query(**{name: value})
    for field in ("num_kv_heads", "head_dim", "k_exp", "v_exp"):
        with pytest.raises(ValueError, match=field):
            _cache(**{field: 2 ** 32 + 64})
