"""Accumulated weights and eviction without a GPU: pins of the oracle, sizes, and refusals before any launch."""
import itertools

import numpy as np
import pytest

from oracle import kv_oracle as K
from sparse_long_context_tail_gb300 import _binding as B
from sparse_long_context_tail_gb300 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


# ------------------------------------------------------------------ oracle --

def test_drawn_weight_closed_forms():
    # equal logits: every visible entry draws the same from each row
    drawn, slack = K.accumulate(np.zeros((2, 3, 4)), np.log([[2.0] * 3, [3.0] * 3]), [np.ones((3, 1, 4))], [0, 2])
    assert np.allclose(drawn[0], [3 / 2 + 1, 3 / 2 + 1, 1])
    assert np.allclose(slack[0]["one"], drawn[0]) and not slack[0]["reach"].any()
    # the softmax of the attention: what a row gives adds up to one
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((5, 4, 8)), [rng.standard_normal((n, 2, 8)) for n in (7, 0, 9)]
    cu = [0, 2, 3, 5]
    lse = K.attend(q, k, k, cu, window=3, sinks=1)[1]
    drawn, _ = K.accumulate(q, lse, k, cu, window=3, sinks=1)
    assert [round(w.sum(), 9) for w in drawn] == [8, 0, 8] and np.isneginf(lse[2]).all()
    x = np.exp((k[0][:, 1] @ q[1, 3]) / np.sqrt(8))
    lone = np.full((5, 4), -np.inf)
    lone[1, 3] = np.log(x[[0, 4, 5, 6]].sum())
    w = K.accumulate(q, lone, k, cu, window=3, sinks=1)[0][0]
    want = x / x[[0, 4, 5, 6]].sum()
    want[1:4] = 0
    assert np.allclose(w, want)


def test_evicted_lists_by_hand_and_by_trial():
    assert K.evict([5, 1, 1, 4, 1, 9], 3, 3, 0, 0) == [0, 3, 5]
    assert K.evict([5, 1, 1, 4, 1, 9], 4, 4, 0, 0) == [0, 1, 3, 5]          # of equal ones the lower
    assert K.evict([0, 1, 1, 4, 1, 0], 4, 4, 1, 1) == [0, 1, 3, 5]          # the ends stay whatever they weigh
    assert K.evict([0, 1, 1, 4, 1, 0], 2, 2, 1, 1) == [0, 5]
    assert K.evict([1] * 6, 4, 6, 0, 0) == list(range(6)) and K.evict([1] * 7, 4, 6, 0, 1) == [0, 1, 2, 6]
    assert K.evict([], 4, 6, 2, 1) == []
    for w in itertools.product([0, 1, 2], repeat=6):
        got = K.evict(w, 3, 3, 1, 1)
        best = max(itertools.combinations(range(1, 5), 1), key=lambda c: (sum(w[e] for e in c), [-e for e in c]))
        assert got == [0, *best, 5]


# ------------------------------------------------------------- host refusals --

def _cache(**kw):
    a = dict(data=0x1000, num_slots=64, num_kv_heads=2, head_dim=128)
    a.update(kw)
    return B.make_kv_cache(**a)


def _eviction(**kw):
    a = dict(num_reqs=2, kv_len=0x100, kv_len_out=0x100, page_table=0x200, page_stride=4, max_pages=4, page_size=16,
             weights=0x10000, weights_stride=64, weights_cols=64, weights_out=0x10000, weights_out_stride=64,
             weights_out_cols=64, budget=32, trigger=40, sinks=2, recent=8)
    a.update(kw)
    return B.make_kv_eviction(**a)


SIZES = [(dict(num_reqs=0), "num_reqs"), (dict(num_reqs=2 ** 20 + 1), "num_reqs"), (dict(page_size=8), "page_size"),
         (dict(page_size=40), "page_size"), (dict(page_size=1 << 17), "page_size"), (dict(max_pages=0), "max_pages"),
         (dict(max_pages=1 << 27), "max_pages"), (dict(budget=0), "budget"), (dict(budget=41), "budget"),
         (dict(trigger=31), "trigger"), (dict(sinks=-1), "sinks"), (dict(recent=-1), "recent"),
         (dict(sinks=25, recent=8), "sinks"), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), "sinks"),
         (dict(num_reqs=2 ** 20, max_pages=2 ** 20, trigger=2 ** 24), "too many")]
POINTERS = [(dict(kv_len=0), "kv_len"), (dict(kv_len_out=0), "kv_len_out"), (dict(page_table=0), "page_table"),
            (dict(page_stride=3), "page_stride"), (dict(page_table_out=0x300), "max_pages_out"),
            (dict(page_table_out=0x300, max_pages_out=4, page_stride_out=3), "page_stride_out"),
            (dict(page_table_out=0x300, max_pages_out=1 << 27, page_stride_out=1 << 28), "max_pages_out"),
            (dict(weights=0), "weights"), (dict(weights=0x10002), "weights"), (dict(weights_cols=0), "cols"),
            (dict(weights_cols=65), "cols"), (dict(weights_out=0), "weights_out"), (dict(weights_out_cols=65), "cols"),
            (dict(weights_out_stride=80), "weights_out"), (dict(weights_out=0x10004), "weights_out"),
            (dict(weights_out=0x10000 + 256), "weights_out"), (dict(kv_len_out=0x104), "kv_len_out"),
            (dict(kv_len_out=0xFE), "kv_len_out"), (dict(kept=0x400, kept_stride=31), "kept_stride")]


@pytest.mark.parametrize("bad,word", SIZES)
def test_sizes_that_are_refused(bad, word):
    x = _eviction(**bad)
    for call in (lambda: B.upf_kv_evict_workspace_bytes(_cache(), x), lambda: B.upf_kv_evict(None, _cache(), x, 256, 1 << 40)):
        with pytest.raises(B.UpfError) as e:
            call()
        assert word in e.value.message, e.value.message


@pytest.mark.parametrize("bad,word", POINTERS + [(dict(), "context")])
def test_evictions_that_are_refused(bad, word):
    x = _eviction(**bad)
    need = B.upf_kv_evict_workspace_bytes(_cache(), x)
    with pytest.raises(B.UpfError) as e:
        B.upf_kv_evict(None, _cache(), x, 256, need)
    assert word in e.value.message, e.value.message


def test_eviction_workspaces():
    need = B.upf_kv_evict_workspace_bytes(_cache(), _eviction())
    for ws, have in ((0, need), (128, need), (256, need - 1)):
        with pytest.raises(B.UpfError, match="workspace"):
            B.upf_kv_evict(None, _cache(), _eviction(), ws, have)
    # by what can stay, not by what a table could hold
    assert B.upf_kv_evict_workspace_bytes(_cache(), _eviction(max_pages=1 << 20, page_stride=1 << 20)) == need
    with pytest.raises(B.UpfError):
        B.upf_kv_evict_workspace_bytes(_cache(num_slots=40), _eviction())
    assert B.load().upf_kv_evict_workspace_bytes(None, None) == 0 and "NULL" in B.upf_last_error()


# rows side by side in one array, and another array: these get as far as the missing context
@pytest.mark.parametrize("good", [dict(weights_stride=200, weights_out_stride=200, weights_out=0x10000 + 400),
                                  dict(weights_out=0x20000, weights_out_stride=90), dict(num_reqs=1, weights_out_stride=100),
                                  dict(kv_len_out=0x108), dict(kv_len_out=0xF8),
                                  dict(page_table_out=0x200, page_stride_out=4, max_pages_out=4)])
def test_evictions_that_are_not_refused(good):
    with pytest.raises(B.UpfError, match="context"):
        B.upf_kv_evict(None, _cache(), _eviction(**good), 256, 1 << 20)


def _query(**kw):
    a = dict(num_reqs=2, num_q_heads=4, num_q_tokens=2, kv_len=0x100, page_table=0x100, page_stride=4, max_pages=4,
             page_size=16)
    a.update(kw)
    return B.make_kv_query(**a)


CALLS = [(dict(), "context"), (dict(dtype=7), "dtype"), (dict(q=0), "q"), (dict(q=0x20008), "aligned"), (dict(qs=504), "stride"),
         (dict(lse=0), "lse"), (dict(lse=0x30002), "lse"), (dict(decay=-1e-9), "decay"), (dict(decay=1.001), "decay"),
         (dict(decay=float("nan")), "decay"), (dict(w_out=0), "weights_out"), (dict(w_out=0x50001), "weights_out"),
         (dict(w_in=0x40002), "weights_in"), (dict(cols=0), "cols"), (dict(cols=65), "cols"), (dict(w_in=0x50004), "weights_out"),
         (dict(w_in=0x50100), "weights_out")]


def _accumulate(query=None, **kw):
    a = dict(dtype=0, q=0x20000, qs=512, lse=0x30000, decay=1.0, w_in=0x40000, w_out=0x50000, stride=64, cols=64, ws=256,
             have=1 << 20)
    a.update(kw)
    x, keep = query or _query()
    B.upf_kv_accumulate(None, _cache(), x, a["dtype"], a["q"], a["qs"], a["lse"], a["decay"], a["w_in"], a["w_out"],
                        a["stride"], a["cols"], a["ws"], a["have"])


@pytest.mark.parametrize("bad,word", CALLS)
def test_accumulations_that_are_refused(bad, word):
    with pytest.raises(B.UpfError) as e:
        _accumulate(**bad)
    assert word in e.value.message, e.value.message


@pytest.mark.parametrize("good", [dict(w_in=0), dict(w_in=0x50000), dict(w_in=0x50000 + 400, stride=200), dict(decay=0.0)])
def test_accumulations_that_are_not_refused(good):
    with pytest.raises(B.UpfError, match="context"):
        _accumulate(**good)


@pytest.mark.parametrize("bad,word", [(dict(num_q_heads=3), "H_q"), (dict(max_q_len=1025), "max_q_len"),
                                      (dict(page_size=24), "page_size"), (dict(window=-1), "window"), (dict(kv_len=0), "kv_len"),
                                      (dict(num_q_tokens=3), "cu_q"), (dict(softmax_scale=float("nan")), "softmax_scale")])
def test_accumulations_with_bad_queries_are_refused(bad, word):
    with pytest.raises(B.UpfError) as e:
        _accumulate(query=_query(**bad))
    assert word in e.value.message, e.value.message


@pytest.mark.parametrize("name", ["kv_len", "kv_len_out", "page_table", "page_table_out", "kept"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_evictions_with_misaligned_arrays_are_refused(name, off):
    a = dict(kv_len=0x100, kv_len_out=0x200, page_table=0x300, page_table_out=0x400, page_stride_out=4, max_pages_out=4, kept=0x500,
             kept_stride=32)
    with pytest.raises(B.UpfError, match="context"):
        B.upf_kv_evict(None, _cache(), _eviction(**a), 256, 1 << 20)
    a[name] += off
    with pytest.raises(B.UpfError, match=f"{name} must be 4-byte aligned"):
        B.upf_kv_evict(None, _cache(), _eviction(**a), 256, 1 << 20)


@pytest.mark.parametrize("name", ["kv_len", "page_table", "cu_q"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_accumulations_with_misaligned_arrays_are_refused(name, off):
    a = dict(kv_len=0x100, page_table=0x300, cu_q=0x400)
    with pytest.raises(B.UpfError, match="context"):
        _accumulate(query=_query(**a))
    a[name] += off
    with pytest.raises(B.UpfError, match=f"{name} must be 4-byte aligned"):
        _accumulate(query=_query(**a))
