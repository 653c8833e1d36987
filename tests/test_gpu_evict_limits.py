"""Accumulated weights and eviction where numbers are at the ends of their range, against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from sparse_long_context_tail_gb300 import _binding as B
from test_gpu_evict import BF16, DEV, F16, Batch, check_evict, f64, queries
from test_gpu_kv import peaked

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


# ------------------------------------------------------- logits of any size --

FAR = 2.0 ** 23     # of |lse| log2 e: from there on a weight is held at 1


def accumulated(b, q, lse, old, **kw):
    return b.cache.accumulate(q, lse, b.table, b.kv_len, b.page, old, out=torch.full_like(old, 7.0), **kw)


def most_drawn(q, lse, k, window=0, sinks=0):
    """What the entries of one request draw at most, from q [rows, H_q, d] and lse [rows, H_q]; 0 where nothing is for certain.

    The exponent x - lse is off by the product's error (d + 8 terms of 2^-23 of sum |q_j k_j|), 2^-22 of x and of lse, and
    2^-20; from FAR on a weight is 1 at most; 2^-150 is below fp32's least number."""
    news, Hq, d = q.shape
    total = np.zeros(len(k))
    for i in range(news):
        seen = np.zeros(len(k), bool)
        seen[K.visible(len(k), news, i, window, sinks)] = True
        for h in range(Hq):
            if not np.isfinite(lse[i, h]):
                continue
            key = k[:, h // (Hq // k.shape[1])]
            x, reach = key @ q[i, h] * d ** -0.5, np.abs(key) @ np.abs(q[i, h]) * d ** -0.5
            u = x - lse[i, h] + reach * (d + 8) * 2.0 ** -23 + (np.abs(x) + abs(lse[i, h])) * 2.0 ** -22 + 2.0 ** -20
            if abs(lse[i, h]) * np.log2(np.e) >= FAR:
                u = np.minimum(u, 0)
            total += np.where(seen & (u > -104), np.exp(np.clip(u, -104, 700)), 0)
    return total


@pytest.mark.parametrize("Hq,d", [(4, 64), (12, 64), (4, 128), (12, 128), (4, 256), (12, 256)])
@pytest.mark.parametrize("logit", [1e5, 1e7, 1e9, 1e10, 2.0 ** 34, 1e12, 1e30, 1.2 * 2.0 ** 126])
def test_weights_of_peaked_rows(logit, Hq, d):
    """One entry (or two) far above all others, four rows a kv head and twelve: no NaN, no infinity, and what is far below or
    not seen keeps exactly what it had."""
    for twice in (False, True):
        for window, sinks in ((0, 0), (37, 5)):
            b, q, cu_q, top = peaked([1, 40, 700], Hq, 1, d, logit, twice=twice)
            b.page = 16
            lse = b.cache.attend(q, b.table, b.kv_len, 16, window=window, sinks=sinks).lse
            assert b.cache.status() == 0 and torch.isfinite(lse).all()
            old = torch.rand(3, 704, generator=torch.Generator().manual_seed(1)).to(DEV)
            got = accumulated(b, q, lse, old, window=window, sinks=sinks)
            assert b.cache.status() == 0
            for r, n in enumerate(b.lens):
                most = most_drawn(f64(q[r:r + 1]), f64(lse[r:r + 1]), b.k[r], window, sinks)
                none = torch.from_numpy(most == 0).to(DEV)
                assert torch.equal(got[r, :n][none], old[r, :n][none]) and (got[r, n:] == 7).all()
                drew = f64(got[r, :n]) - f64(old[r, :n])
                # the sum of the rows and of the old weight: its roundings
                assert (drew >= -2.0 ** -22).all() and (drew <= most * (1 + 2.0 ** -20) + 2.0 ** -22).all()
            kept = b.cache.evict(got, b.table, b.kv_len, 16, 20)
            assert b.cache.status() == 0 and (kept[2] >= 0).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,news", [(2, [1, 3]), (4, [1, 2]), (24, [1, 1]), (8, [7, 40])])
@pytest.mark.parametrize("size", [1e3, 1e6, 1e9])
def test_rows_of_large_logits_beside_ordinary_ones(size, Hq, news, dtype):
    """Every third row is multiplied by `size`; the others' weights are right within their arithmetic, and the large rows add
    what they may, nothing where their weight is 0 for certain."""
    if dtype == F16:
        size = min(size, 1e3)
    b = Batch([150, 333], 2, 128, seed=70)
    q, cu = queries(news, Hq, 128, dtype, 71)
    big = torch.zeros(q.shape[:2], dtype=torch.bool)
    big.view(-1)[::3] = True
    q = torch.where(big[:, :, None].to(DEV), (q.float() * size).to(dtype), q)
    assert torch.isfinite(q).all()
    kw = dict(cu_q=cu, max_q_len=max(news))
    lse = b.cache.attend(q, b.table, b.kv_len, 16, **kw).lse
    old = torch.zeros(2, 352, device=DEV)
    got = accumulated(b, q, lse, old, **kw)
    assert b.cache.status() == 0
    q64, l64, at = f64(q), f64(lse), cu.tolist()
    plain, slack = K.accumulate(q64, np.where(big.numpy(), -np.inf, l64), b.keys(), at)
    for r, n in enumerate(b.lens):
        mine = slice(at[r], at[r + 1])
        rows = news[r] * Hq
        large = most_drawn(q64[mine], np.where(big.numpy(), l64, -np.inf)[mine], b.keys()[r])
        s = slack[r]
        # as for all weights: products, the rounding of the row, logit factor and lse, the sum of all rows
        bound = (s["reach"] * 136 * 2.0 ** -23 + s["flat"] * 2.0 ** -25 + s["far"] * 2.0 ** -22 + s["one"] * 2.0 ** -21
                 + (rows + 2) * 2.0 ** -24 * (plain[r] + large) + 2.0 ** -125 * rows)
        over = f64(got[r, :n]) - plain[r]
        assert (over >= -bound).all() and (over <= bound + large).all()


def test_lse_whose_binary_logarithm_is_past_fp32_adds_nothing():
    """No attention gives such an lse back: it is reported as an infinite one is."""
    b = Batch([40, 50, 60], 2, 64, seed=12)
    for Hq in (4, 32):
        q, _ = queries([1, 1, 1], Hq, 64, BF16, 13)
        lse = b.cache.attend(q, b.table, b.kv_len, 16).lse
        old = torch.zeros(3, 64, device=DEV)
        base = accumulated(b, q, lse, old)
        for far, status in ((2.4e38, 5), (3.4e38, 5), (-2.4e38, 5), (2.3e38, 0)):
            l2 = lse.clone()
            l2[1] = far
            got = accumulated(b, q, l2, old)
            assert b.cache.status() == status
            assert not got[1, :50].any() and torch.equal(got[0], base[0]) and torch.equal(got[2], base[2])


@pytest.mark.parametrize("Hq", [1, 12])
def test_how_exactly_lse_is_taken(Hq):
    """Zero queries, so that a weight is exp(-lse) by itself.  Few rows: lse log2 e in two parts, so that two powers of two (2^-22
    each), their product and the sum are all; its rounding as one number would be 2^-18 at |lse| = 80.  Many rows have it as
    one: 2^-24 |lse|, one power and the sum."""
    R = 64
    b = Batch([5] * R, 1, 64, seed=87)
    q = torch.zeros(R, Hq, 64, dtype=BF16, device=DEV)
    at = np.linspace(-80, 80, R) + 0.1 * np.sin(np.arange(R))
    lse = torch.full((R, Hq), -float("inf"), device=DEV)
    lse[:, Hq // 2] = torch.from_numpy(at).float().to(DEV)
    got = f64(accumulated(b, q, lse, torch.zeros(R, 8, device=DEV))[:, :5])
    assert b.cache.status() == 0
    l64 = f64(lse[:, Hq // 2])[:, None]
    want = np.exp(-l64)
    error = 2.0 ** -21 + 2.0 ** -23 if Hq == 1 else np.abs(l64) * 2.0 ** -24 + 2.0 ** -21
    assert (np.abs(got / want - 1) <= error).all(), np.abs(got / want - 1).max()


# ----------------------------------------------------- keys that hold a NaN --

@pytest.mark.parametrize("Hq,news", [(2, 5), (8, 5), (8, 1), (32, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 20)])
def test_a_key_with_a_nan_marks_its_entry_wherever_it_is_seen(Hq, news, window, sinks):
    """Rows that count and rows that do not, tiles that are seen whole and in part: NaN where a row sees the entry, and
    nowhere else."""
    n, H = 300, 2
    b = Batch([n], H, 64, seed=72)
    odd = [3, 17, 130, 200, 257, 262, 297, 299]
    k = b.k.clone()
    k[odd, 1, 5] = float("nan")
    b.cache.write(k, b.v, b.slots[0])
    q, cu = queries([news], Hq, 64, BF16, 73)
    kw = dict(cu_q=cu, max_q_len=news, window=window, sinks=sinks)
    lse = b.cache.attend(q, b.table, b.kv_len, 16, **kw).lse
    assert lse[:, Hq // 2:].isnan().all() and lse[:, :Hq // 2].isfinite().all()
    seen = np.zeros(n, bool)
    for i in range(news):
        seen[K.visible(n, news, i, window, sinks)] = True
    want = np.zeros(n, bool)
    want[odd] = True
    want &= seen
    assert 0 < want.sum() < len(odd) or not window
    other = lse.clone()
    other[:, Hq // 2:] = -float("inf")
    drawn = K.accumulate(f64(q), f64(other), [K.cache_values(f64(k), 0)], cu.tolist(), window, sinks)[0][0]
    for x, status in ((lse, 5), (other, 0)):
        got = f64(accumulated(b, q, x, torch.zeros(1, n, device=DEV), **kw)[0])
        assert b.cache.status() == status
        np.testing.assert_array_equal(np.isnan(got), want)
        assert np.allclose(got[~want], drawn[~want], rtol=1e-4)


# ------------------------------------------- rows that two requests begin with --

@pytest.mark.parametrize("Hq", [2, 9, 128])
def test_requests_whose_rows_begin_before_an_earlier_one_ends_are_skipped(Hq):
    """cu_q that goes back: each request by itself may make sense, but a row has one place in the call."""
    b = Batch([40, 50, 60, 200], 1, 64, seed=77)
    q, _ = queries([12], Hq, 64, BF16, 78)
    lse = torch.full((12, Hq), 2.0, device=DEV)
    old = torch.rand(4, 208, generator=torch.Generator().manual_seed(79)).to(DEV)
    keys = b.keys()
    for cu, first_len, good in (([0, 8, 0, 8, 12], 40, [0, 3]), ([0, 5, 2, 9, 12], 40, [0, 3]), ([4, 9, 0, 4, 8], 40, [0]),
                                ([0, 8, 2, 6, 12], -1, [2, 3]), ([7, 7, 2, 5, 6], 40, [2, 3]), ([0, 3, 3, 2, 4], 40, [0]),
                                ([0, 4, 8, 8, 12], 40, [0, 1, 3])):
        kv_len = b.kv_len.clone()
        kv_len[0] = first_len
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        got = b.cache.accumulate(q, lse, b.table, kv_len, 16, old, cu_q=c, max_q_len=8, out=old.clone())
        fine = all(x <= y for x, y in zip(cu, cu[1:])) and first_len >= 0
        assert b.cache.status() == (0 if fine else 1), cu
        for r, n in enumerate(b.lens):
            if r not in good:
                assert torch.equal(got[r], old[r]), (cu, r)
                continue
            mine = slice(cu[r], cu[r + 1])
            drawn = K.accumulate(f64(q[mine]), f64(lse[mine]), [keys[r]], [0, cu[r + 1] - cu[r]])[0][0]
            assert np.allclose(f64(got[r, :n]), f64(old[r, :n]) + drawn, rtol=1e-4), (cu, r)
            assert torch.equal(got[r, n:], old[r, n:])


@pytest.mark.parametrize("Hq", [5, 18])
def test_many_requests_whose_rows_go_back(Hq):
    """2500 requests of a row: from the thousandth on they begin again at row 500, and count again from row 1000 on."""
    R = 2500
    b = Batch([(5 * i) % 23 for i in range(R)], 1, 64, seed=80)
    N = 2000
    q, _ = queries([N], Hq, 64, BF16, 81)
    lse = torch.full((N, Hq), 3.0, device=DEV)
    old = torch.rand(R, 32, generator=torch.Generator().manual_seed(82)).to(DEV)
    back = torch.cat([torch.arange(1001), torch.arange(500, 2000)]).int()         # [1000, 500) is no request's range
    assert back.numel() == R + 1
    got = b.cache.accumulate(q, lse, b.table, b.kv_len, 16, old, cu_q=back.to(DEV), max_q_len=2, out=old.clone())
    assert b.cache.status() == 1
    level = torch.cummax(back, 0).values          # the same without those that are skipped: they are empty
    want = b.cache.accumulate(q, lse, b.table, b.kv_len, 16, old, cu_q=level.to(DEV), max_q_len=2, out=old.clone())
    assert b.cache.status() == 0
    assert torch.equal(got[1000:1501], old[1000:1501])
    assert torch.allclose(got, want, rtol=1e-5) and not torch.equal(got[1501:], old[1501:])


# ------------------------------------------- requests that cannot be evicted --

def test_a_refused_request_keeps_its_length_when_lengths_are_rewritten_in_place():
    """Into other pages with kv_len itself as the new lengths: a request that is skipped is marked as not there, and its
    length can be had back."""
    b = Batch([100, 90, 80, 0], 2, 64, seed=74, spare=40)
    was = [b.contents(s) for s in b.slots]
    w = torch.rand(4, 120, generator=torch.Generator().manual_seed(75)).to(DEV)
    fine, want = w.clone(), K.evict(w[1, :90].tolist(), 50, 50, 0, 5)
    w[1, 40] = float("nan")
    out = b.free[:16].view(4, 4).to(DEV)
    kept = b.cache.evict(w, b.table, b.kv_len, 16, 50, recent=5, page_table_out=out)
    assert b.cache.status() == 5 and (kept[1] == -1).all()
    assert b.kv_len.tolist() == [50, -1 - 90, 50, 0]
    # the new table says so to whoever reads it, and a second call leaves it
    q, cu = queries([1] * 4, 4, 64, BF16, 76)
    got = b.cache.attend(q, out, b.kv_len, 16)
    assert b.cache.status() == 1 and not got.out[1].any() and torch.isneginf(got.lse[1]).all()
    again = torch.tensor([-1 - 90, -2 ** 31, 2 ** 31 - 1, -1], dtype=torch.int32, device=DEV)
    b.cache.evict(fine, b.table, again, 16, 50, recent=5, page_table_out=out)
    assert b.cache.status() == 1 and again.tolist() == [-1 - 90, -2 ** 31, -2 ** 31, -1]
    # the old pages hold its entries as before
    n = -1 - int(b.kv_len[1])
    assert n == 90 and all(torch.equal(x, y) for x, y in zip(b.contents(b.slots[1]), was[1]))
    lens = torch.tensor([0, n, 0, 0], dtype=torch.int32, device=DEV)
    kept = b.cache.evict(fine, b.table, lens, 16, 50, recent=5, page_table_out=out)
    assert b.cache.status() == 0 and lens.tolist() == [0, 50, 0, 0] and kept[1].tolist() == want


# --------------------------------------------------------- waits that run out --

@pytest.mark.parametrize("elsewhere", [False, True])
def test_a_wait_of_an_eviction_that_runs_out(elsewhere):
    """With a limit of one cycle, as often as it takes until some chunk looks for another one before that has been read: it
    is reported, lists, lengths and weights are those of a whole eviction, and what was not to be moved is as it was."""
    lens, budget, trigger = [20000, 500, 20000, 900, 20000, 0, 20000], 19000, 19500
    b = Batch(lens, 2, 64, seed=83, spare=len(lens) * 1250 if elsewhere else 20)
    w0 = torch.rand(7, 20000, generator=torch.Generator().manual_seed(84)).to(DEV)
    storage, want = b.cache.storage.clone(), [K.evict(w0[r, :n].tolist(), budget, trigger, 3, 40) for r, n in enumerate(lens)]
    kw, slots = {}, b.slots
    if elsewhere:          # the first pages are the request's own
        out = b.free[:7 * 1250].view(7, 1250).to(DEV).clone()
        own = min(600, b.table.shape[1])
        long = [0, 2, 4, 6]
        out[long, :own] = b.table[long, :own]
        kw["page_table_out"] = out
        slots = [b.slot_list(out[r], len(want[r])) for r in range(7)]
    mine = torch.zeros(b.cache.num_slots, dtype=torch.bool, device=DEV)
    for r, n in enumerate(lens):
        if elsewhere or n > trigger:
            mine[slots[r]] = True
        if not elsewhere and n > trigger:
            mine[b.slots[r]] = True
    others = (~mine).nonzero().flatten()
    before = b.contents(others)
    B.upf_set_wait_limit(b.cache.ctx, 1)
    for _ in range(100):
        b.cache.storage.copy_(storage)
        w, n2 = w0.clone(), b.kv_len.clone()
        kept = b.cache.evict(w, b.table, n2, b.page, budget, trigger=trigger, sinks=3, recent=40, **kw)
        status = b.cache.status()
        assert n2.tolist() == [len(x) for x in want]
        if status:
            break
    assert status == 6
    for r, n in enumerate(lens):
        assert kept[r].tolist() == (want[r] + [-1] * budget)[:budget]
        at = torch.tensor(want[r], dtype=torch.long, device=DEV)
        assert torch.equal(w[r, :len(at)], w0[r, at]) and not w[r, len(at):n].any() and torch.equal(w[r, n:], w0[r, n:])
    assert all(torch.equal(x, y) for x, y in zip(b.contents(others), before))
    B.upf_set_wait_limit(b.cache.ctx, 0)
    b.cache.storage.copy_(storage)
    was = [b.contents(s) for s in b.slots]
    kept = b.cache.evict(w0.clone(), b.table, b.kv_len, b.page, budget, trigger=trigger, sinks=3, recent=40, **kw)
    assert b.cache.status() == 0
    for r in range(7):
        at = torch.tensor(want[r], dtype=torch.long, device=DEV)
        assert all(torch.equal(x, y[at]) for x, y in zip(b.contents(b.slot_list(kw["page_table_out"][r] if elsewhere else b.table[r], len(at))), was[r]))


# ----------------------------------------- clusters and shared memory in full --

@pytest.mark.parametrize("kind", ["mixed", "equal", "near"])
@pytest.mark.parametrize("lens,budget", [([50000], 11111),                       # a cluster of eight
                                         ([40000, 900, 33000, 0, 17], 800),      # of eight, for more than four requests
                                         ([700000], 200000),                     # of sixteen, weights past shared memory
                                         ([350000, 10, 5000, 20, 30], 4000)])    # of eight, weights past shared memory
def test_requests_whose_weights_do_not_fit_a_cluster(lens, budget, kind):
    check_evict(Batch(lens, 1, 64, page=256, seed=85), budget, sinks=3, recent=50, kind=kind)


def test_bad_weights_past_shared_memory_are_found():
    """The last weights of a warp, and of the last one; a tie across the whole request."""
    n = 700000
    b = Batch([n], 1, 64, page=256, seed=86)
    storage = b.cache.storage.clone()
    w = torch.full((1, n), 0.25, device=DEV)
    w[0, 1000::7] = 0.5
    for at in (1300, 1405, n - 60, n - 55, n - 1, 0):
        for bad in (float("nan"), -1.0):
            x = w.clone()
            x[0, at] = bad
            kept = b.cache.evict(x, b.table, b.kv_len, 256, 150000, sinks=3, recent=50)
            assert b.cache.status() == 5 and (kept == -1).all() and b.kv_len.tolist() == [n]
            assert torch.equal(b.cache.storage, storage)
    kept = b.cache.evict(w.clone(), b.table, b.kv_len.clone(), 256, 150000, sinks=3, recent=50)
    assert b.cache.status() == 0 and kept[0].tolist() == K.evict(w[0].tolist(), 150000, 150000, 3, 50)


# ------------------------------------------------- one table with two strides --

def test_places_in_the_same_table_with_another_stride():
    """page_table_out begins where page_table does, but its second row is another one: entries of requests that are not cut
    are copied there all the same."""
    b = Batch([60, 50], 2, 64, seed=88, spare=12)
    was = [b.contents(s) for s in b.slots]
    P = b.table.shape[1]
    room = torch.full((4 * P,), -7, dtype=torch.int32, device=DEV)
    room[:2 * P] = b.table.flatten()
    room[3 * P:] = b.free[:P].to(DEV)
    table, out = room.as_strided((2, P), (P, 1)), room.as_strided((2, P), (3 * P, 1))
    w = torch.rand(2, 64, device=DEV)
    old = w.clone()
    for budget in (64, 55):        # none cut, the first one cut
        kept = b.cache.evict(w, table, b.kv_len, 16, budget, page_table_out=out)
        assert b.cache.status() == 0
        for r, n in enumerate(b.lens):
            want = K.evict(old[r, :n].tolist(), budget, budget, 0, 0)
            assert kept[r].tolist() == want + [-1] * (budget - len(want)) and int(b.kv_len[r]) == len(want)
            at = torch.tensor(want, device=DEV)
            assert all(torch.equal(x, y[at]) for x, y in zip(b.contents(b.slot_list(out[r], len(want))), was[r]))
