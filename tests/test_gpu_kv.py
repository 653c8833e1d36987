"""The 4-bit KV cache on the GPU against the float64 oracle.

Writing and reading back are exact: every code and scale is the definition's, so
what is read in bf16 equals the oracle's values bit for bit, and in fp16 its
rounding.  Attention is compared with a tolerance derived from the arithmetic (`_bound`).
"""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from sparse_long_context_tail_gb300 import _binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def make(num_slots, H, d, fill=0xA5, **kw):
    from sparse_long_context_tail_gb300.kvcache import QuantKVCache
    c = QuantKVCache(num_slots, H, d, **kw)
    c.storage.fill_(fill)          # unwritten slots hold rubbish: 0xFF is a NaN scale
    return c


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    x *= torch.exp2(torch.randint(-3, 4, shape[:-1] + (1,), generator=g).float())
    return x.to(dtype).to(DEV)


def f64(t):
    return t.cpu().double().numpy()


# ------------------------------------------------------------ write and read --

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H,d", [(1, 64), (2, 64), (3, 128), (8, 128), (2, 256)])
@pytest.mark.parametrize("T", [1, 2, 17, 131])
def test_what_is_written_is_read_back(T, H, d, dtype):
    c = make(16 * 20, H, d, k_exp=1, v_exp=-2)
    before = c.storage.clone()
    k, v = rand((T, H, d), dtype, 1), rand((T, H, d), dtype, 2)
    slots = torch.randperm(c.num_slots, generator=torch.Generator().manual_seed(3))[:T]
    c.write(k, v, slots.to(DEV))
    want = [K.cache_values(f64(k), 1), K.cache_values(f64(v), -2)]
    got = [f64(x) for x in c.read(slots.to(DEV))]
    packed = c.storage.cpu().numpy()
    for of in range(2):
        np.testing.assert_array_equal(got[of], want[of])
        np.testing.assert_array_equal(K.unpack(packed, slots.tolist(), H, d, (1, -2)[of], bool(of)), want[of])
    for x, w in zip(c.read(slots.to(DEV), dtype=F16), want):
        np.testing.assert_array_equal(x.cpu().numpy(), w.astype(np.float16))
    others = torch.ones(c.num_slots, dtype=torch.bool)
    others[slots] = False
    rest = others.nonzero().flatten().to(DEV)
    now = c.storage.clone()
    c.storage.copy_(before)
    was = c.read(rest)
    c.storage.copy_(now)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(was, c.read(rest)))
    assert c.status() == 0


def test_every_tie_and_border_is_the_definitions():
    """All 7-bit values against every 4-bit scale: x = m 2^e around each tie and each e4m3 border."""
    rows = []
    for top in list(range(64, 128)):                      # amax = top / 16 * 2^e
        for e in (-9, -6, -1, 0, 3, 7):
            g = torch.arange(0, 128, 8) * top / 128.0 / 16.0
            g[0] = top / 16.0
            rows.append(g * 2.0 ** e * torch.where(torch.arange(16) % 3 == 0, -1.0, 1.0))
    for sb in range(1, 0x7F):                              # amax = 6 s: the ties themselves
        s = K.E4M3[sb]
        rows.append(torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0]) * s)
        if sb > 1:                                         # amax / 6 midway between two scales
            rows.append(torch.cat([torch.tensor([3 * (s + K.E4M3[sb - 1])]), torch.linspace(-1, 1, 15) * s]))
    x = torch.stack(rows)
    x = torch.cat([x, torch.zeros(-len(x) % 8, 16)]).view(-1, 1, 128)
    for dtype in (BF16, F16):
        y = x.to(dtype).to(DEV)
        y = torch.where(torch.isfinite(y), y, torch.zeros_like(y))
        c = make((len(y) + 15) // 16 * 16, 1, 128)
        slots = torch.arange(len(y), device=DEV)
        c.write(y, -y, slots)
        k, v = c.read(slots)
        np.testing.assert_array_equal(f64(k), K.cache_values(f64(y), 0))
        np.testing.assert_array_equal(f64(v), -K.cache_values(f64(y), 0))


def test_non_finite_extreme_and_tiny_groups():
    x = torch.ones(6, 1, 64)
    x[0, 0, 3], x[1, 0, 17], x[2, 0, 63] = float("nan"), float("inf"), float("-inf")
    x[3] *= 3e38
    x[4] *= 1e-39
    x[5] = 0
    for exp in (-32, 0, 32):
        c = make(16, 1, 64, k_exp=exp, v_exp=exp)
        slots = torch.arange(6, device=DEV)
        y = x.to(BF16).to(DEV)
        c.write(y, y, slots)
        want = K.cache_values(f64(y), exp)
        assert np.isnan(want).sum() == 48
        for got in c.read(slots):
            np.testing.assert_array_equal(f64(got), want)
        # in fp16 values past its range become infinite, as any rounding to it does
        with np.errstate(over="ignore"):
            np.testing.assert_array_equal(c.read(slots, dtype=F16)[0].cpu().numpy(), want.astype(np.float16))


@pytest.mark.parametrize("T", [40, 3000])
def test_a_slot_given_twice_holds_the_last_token(T):
    H, d = 2, 128
    c = make(16 * 64, H, d)
    k, v = rand((T, H, d), BF16, 5), rand((T, H, d), BF16, 6)
    slots = torch.randint(0, 30 if T == 40 else 1000, (T,), generator=torch.Generator().manual_seed(7))
    for _ in range(3):
        c.write(k, v, slots.to(DEV))
        last = {int(s): t for t, s in enumerate(slots)}
        at, own = list(last), list(last.values())
        got = c.read(torch.tensor(at, device=DEV))
        np.testing.assert_array_equal(f64(got[0]), K.cache_values(f64(k[own]), 0))
        np.testing.assert_array_equal(f64(got[1]), K.cache_values(f64(v[own]), 0))
        slots = slots.flip(0)
    # a slot may be read any number of times
    many = torch.tensor([at[0]] * 5 + [at[1]], device=DEV)
    r = c.read(many)[0]
    assert torch.equal(r[0], r[4]) and c.status() == 0


@pytest.mark.parametrize("T", [33, 2000])
def test_skipped_tokens_and_device_counts(T):
    H, d, n = 2, 64, T - 7
    c = make(16 * 200, H, d, fill=0)
    k, v = rand((T, H, d), F16, 8), rand((T, H, d), F16, 9)
    slots = torch.randperm(c.num_slots, generator=torch.Generator().manual_seed(1))[:T]
    used = slots.clone()
    used[3] = -1
    used[5] = -(1 << 40)
    c.write(k, v, used.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV))
    want = K.cache_values(f64(k), 0)
    want[[3, 5]] = 0
    want[n:] = 0
    np.testing.assert_array_equal(f64(c.read(slots.to(DEV))[0]), want)
    out = (torch.full_like(k, 7.0), torch.full_like(v, 7.0))
    c.read(used.to(DEV), out=out, num_tokens=torch.tensor([n], dtype=torch.int32, device=DEV))
    want[[3, 5]] = 7
    want[n:] = 7
    np.testing.assert_array_equal(f64(out[0]), want)
    for count in (0, -4):
        c.write(-k, -v, slots.to(DEV), torch.tensor([count], dtype=torch.int32, device=DEV))
    c.write(k[:0], v[:0], slots[:0].to(DEV))
    assert c.read(slots[:0].to(DEV))[0].shape == (0, H, d)
    want[[3, 5]] = 0
    want[n:] = 0
    np.testing.assert_array_equal(f64(c.read(slots.to(DEV))[0]), want)
    # a count above the tokens given is cut down to them
    c.write(k, v, slots.to(DEV), torch.tensor([T + 100], dtype=torch.int32, device=DEV))
    np.testing.assert_array_equal(f64(c.read(slots.to(DEV))[0]), K.cache_values(f64(k), 0))
    assert c.status() == 0


@pytest.mark.parametrize("T", [4, 1500])
def test_slots_past_the_cache_are_reported_and_skipped(T):
    c = make(1600, 1, 64, fill=0)
    k = rand((T, 1, 64), BF16, 1)
    slots = torch.arange(T, device=DEV)
    slots[2] = 1600
    c.write(k, k, slots)
    assert c.status() == 1 and c.status() == 0
    out = (torch.zeros_like(k), torch.zeros_like(k))
    c.read(slots, out=out)
    assert c.status() == 1 and not out[0][2].any()
    want = K.cache_values(f64(k), 0)
    want[2] = 0
    np.testing.assert_array_equal(f64(out[0]), want)


def test_strided_rows_and_outputs():
    T, H, d = 50, 2, 128
    rows = rand((T, 3 * H, d), BF16, 4)          # one projection's rows: [q | k | v]
    k, v = rows[:, H:2 * H], rows[:, 2 * H:]
    c = make(64, H, d)
    slots = torch.arange(T, device=DEV)
    c.write(k, v, slots)
    wide = torch.zeros(T, 3 * H, d, dtype=BF16, device=DEV)
    c.read(slots, out=(wide[:, :H], wide[:, 2 * H:]))
    np.testing.assert_array_equal(f64(wide[:, :H]), K.cache_values(f64(k), 0))
    np.testing.assert_array_equal(f64(wide[:, 2 * H:]), K.cache_values(f64(v), 0))
    assert not wide[:, H:2 * H].any()
    with pytest.raises(B.UpfError):              # rows that do not start on 16 bytes
        off = torch.zeros(T * H * d + 1, dtype=BF16, device=DEV)[1:].view(T, H, d)
        c.write(off, off, slots)


# ------------------------------------------------------------------ attention --

class Batch:
    """Requests of given lengths in shuffled pages, written through the operator itself."""

    def __init__(self, lens, Hq, H, d, page=16, dtype=BF16, seed=0, k_exp=0, v_exp=0, spare=2, scale=1.0):
        self.lens, self.page, self.H = list(lens), page, H
        need = [-(-n // page) for n in lens]
        total = sum(need) + spare
        self.cache = make(total * page, H, d, fill=0xFF, k_exp=k_exp, v_exp=v_exp)
        order = torch.randperm(total, generator=torch.Generator().manual_seed(seed))
        width = max(max(need), 1)
        self.table = torch.full((len(lens), width + 1), -1, dtype=torch.int32)
        at = 0
        for r, m in enumerate(need):
            self.table[r, :m] = order[at:at + m].int()
            at += m
        slots = [[int(self.table[r, e // page]) * page + e % page for e in range(n)] for r, n in enumerate(lens)]
        self.slots = torch.tensor(sum(slots, []), dtype=torch.int64)
        T = len(self.slots)
        k, v = rand((T, H, d), dtype, seed + 1, 0.5 * scale), rand((T, H, d), dtype, seed + 2)
        if T:
            self.cache.write(k, v, self.slots.to(DEV))
        cut = np.cumsum([0] + self.lens)
        kk, vv = K.cache_values(f64(k), k_exp), K.cache_values(f64(v), v_exp)
        self.k = [kk[cut[r]:cut[r + 1]] for r in range(len(lens))]
        self.v = [vv[cut[r]:cut[r + 1]] for r in range(len(lens))]
        self.table, self.kv_len = self.table.to(DEV), torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.Hq, self.d, self.dtype = Hq, d, dtype

    def queries(self, news, seed=9, scale=1.0):
        cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        return rand((int(cu[-1]), self.Hq, self.d), self.dtype, seed, scale), cu


def _bound(dtype, ref):
    """Tolerances (out, lse) per element, from the arithmetic:

    * one rounding to the output type: eps / 2 of the value;
    * each softmax weight is rounded to f16 once, as 2^12 times its ratio to a reference that
      is at most the row's largest weight: half a step is 2^-11 of it, or, under the smallest
      normal number 2^-14, half of the fixed step 2^-24, which is 2^-25 / 2^12 = 2^-37 of the
      reference.  A normalised weight is thus off by 2^-11 of itself and 2^-37, and the sum by
      2^-11 sum p |v| + 2^-37 sum |v| (the second shows where the heavy entries hold zeros);
    * a logit sums d products in at most 16 matrix steps, each of which may drop 2^-22 of
      the sum of magnitudes; a query element under 2^-14 of its row's largest may lose
      2^-25 of that largest; the factor and the exponential add 2^-21 of the logit and of
      the weight.  delta bounds the logit's error, and weights are off by 2 delta;
    * the weighted sum takes seen / 16 matrix steps and up to 64 joins of parts, 2^-22 each.
    """
    out, lse, spread, total, reach, flat, seen = ref
    delta = reach * 2.0 ** -18 + flat * 2.0 ** -24 + reach * 2.0 ** -21 + 2.0 ** -21
    rel = 2.0 ** -11 + 2 * delta + (seen[:, None] / 16 + 64) * 2.0 ** -22
    finite = np.where(np.isfinite(lse), lse, 0)
    return (np.abs(out) * (torch.finfo(dtype).eps / 2) * (1 + rel[..., None]) + rel[..., None] * spread + 2.0 ** -37 * total
            + float(torch.finfo(dtype).smallest_normal) * float(torch.finfo(dtype).eps),
            delta + 2.0 ** -20 + (seen[:, None] / 16 + 64) * 2.0 ** -22 + np.abs(finite) * 2.0 ** -22)


def compare(got, ref, dtype):
    out, lse = f64(got[0]), f64(got[1])
    b_out, b_lse = _bound(dtype, ref)
    np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(ref[1]))
    over = np.abs(out - ref[0]) / b_out
    bad = np.argwhere(~(over <= 1))
    assert len(bad) == 0, f"{len(bad)} of {over.size} outputs, first {bad[:4].tolist()}, up to {np.nanmax(over):.3g} of the bound"
    see = np.isfinite(ref[1])
    over = np.abs(lse[see] - ref[1][see]) / b_lse[see]
    assert (over <= 1).all(), f"lse: {np.nanmax(over):.3g} of the bound"


def check(batch, news, window=0, sinks=0, scale=None, kv_of_q=None, q_scale=1.0, cu=True):
    q, cu_q = batch.queries(news, scale=q_scale)
    ref = K.attend(f64(q), batch.k, batch.v, cu_q, window, sinks, scale, kv_of_q)
    got = batch.cache.attend(q, batch.table, batch.kv_len, batch.page,
                             cu_q=torch.from_numpy(cu_q).to(DEV) if cu else None, max_q_len=max(max(news), 1),
                             window=window, sinks=sinks, softmax_scale=scale, kv_of_q=kv_of_q)
    assert batch.cache.status() == 0
    compare(got, ref, batch.dtype)
    return q, got, ref


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,H,d", [(8, 2, 64), (5, 1, 64), (4, 4, 128), (8, 2, 128), (12, 1, 128), (20, 1, 128),
                                    (16, 2, 256), (4, 2, 256)])
def test_one_new_token_each(Hq, H, d, dtype):
    b = Batch([1, 2, 15, 16, 17, 31, 32, 33, 0, 100, 257, 700], Hq, H, d, dtype=dtype, k_exp=1, v_exp=-1)
    check(b, [1] * 12, cu=False)


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_page_sizes(page, d):
    check(Batch([1, page - 1, page, page + 1, 3 * page + 5], 4, 2, d, page=page), [1] * 5)


@pytest.mark.parametrize("Hq,H,d", [(8, 2, 64), (8, 2, 128), (3, 3, 128), (16, 2, 256)])
@pytest.mark.parametrize("news", [[1, 3, 0, 7, 2], [2, 2, 2, 2, 2], [33, 1, 5, 40, 9]])
def test_several_new_tokens(news, Hq, H, d):
    b = Batch([40, 3, 9, 130, 2], Hq, H, d)      # request 4: more new tokens than entries leave rows empty
    check(b, news)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (33, 4), (64, 16), (100, 300), (5000, 3), (0, 7)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_windows_and_sinks(window, sinks, d):
    check(Batch([1, 20, 64, 333, 600], 4, 2, d), [1, 1, 2, 3, 1], window=window, sinks=sinks)


def test_pages_behind_the_window_may_be_gone():
    b = Batch([500, 300], 8, 2, 128)
    news, window, sinks = [2, 1], 40, 3
    lost = b.table.clone()
    for r, n in enumerate(b.lens):
        first = (n - news[r] - window + 1) // 16
        lost[r, 1:first] = -7
    b.table = lost
    check(b, news, window=window, sinks=sinks)


def test_scales_head_maps_and_large_and_small_queries():
    b = Batch([77, 200], 6, 3, 128)
    check(b, [1, 1], scale=0.5, kv_of_q=[0, 1, 2, 0, 1, 2])
    check(b, [1, 2], kv_of_q=[2, 2, 1, 1, 0, 0])
    check(b, [1, 2], q_scale=2.0 ** -60)         # logits of nothing: the mean of the values
    check(b, [1, 2], q_scale=64.0)               # a few entries take all the weight


def test_zero_logits_stay_zero_where_their_factor_passes_fp32():
    """Keys of zeros with the largest exponent under huge queries: 2^k_exp times the row's power of two is past 2^128."""
    for d, Hq in ((64, 4), (256, 20)):
        check(Batch([1, 40, 700], Hq, 1, d, k_exp=32, scale=0.0), [1, 2, 1], q_scale=2.0 ** 100)


@pytest.mark.parametrize("Hq,d", [(4, 64), (8, 128), (16, 256)])
def test_a_row_of_nan_stays_by_itself(Hq, d):
    """One head of one query is NaN or infinite: the heads and queries that share its unit are as without it."""
    b = Batch([90, 3000], Hq, 1, d)
    q, cu_q = b.queries([2, 2])
    ask = lambda x: b.cache.attend(x, b.table, b.kv_len, b.page, cu_q=torch.from_numpy(cu_q).to(DEV), max_q_len=2)
    want = ask(q)
    for x in (float("nan"), float("inf")):
        odd = q.clone()
        odd[1, 2, 5], odd[2, 0, d - 1] = x, x
        got = ask(odd)
        for g, w in zip(got, want):
            same = torch.ones_like(g, dtype=torch.bool)
            same[1, 2] = same[2, 0] = False
            assert torch.equal(g[same], w[same])
        if x != x:
            assert got.out[1, 2].isnan().all() and got.out[2, 0].isnan().all() and got.lse[1, 2].isnan()
    assert b.cache.status() == 0


def test_one_entry_is_given_back_exactly():
    b = Batch([1, 1], 4, 2, 128)
    q, got, ref = check(b, [1, 1])
    np.testing.assert_array_equal(f64(got[0]), ref[0])


def test_a_long_request_and_many_requests():
    check(Batch([30000], 8, 2, 64, page=64), [1])
    rng = np.random.default_rng(5)
    check(Batch(rng.integers(0, 60, 300).tolist(), 2, 1, 64), [1] * 300)


def test_rows_of_no_request_are_left_alone():
    b = Batch([40, 50], 4, 2, 128)
    q, cu = b.queries([1, 2])
    q = torch.cat([q, rand((3, 4, 128), BF16, 1)])
    out, lse = torch.full_like(q, 5.0), torch.full((6, 4), 5.0, device=DEV)
    b.cache.attend(q, b.table, b.kv_len, 16, cu_q=torch.from_numpy(cu).to(DEV), max_q_len=2, out=out, lse=lse)
    assert (out[3:] == 5).all() and (lse[3:] == 5).all()
    compare((out[:3], lse[:3]), K.attend(f64(q[:3]), b.k, b.v, cu), BF16)


def test_padded_tables_and_strided_rows():
    b = Batch([40, 50, 9], 4, 2, 64)
    q, cu = b.queries([1, 1, 1])
    wide = torch.zeros(3, 12, 64, dtype=BF16, device=DEV)
    wide[:, 4:8] = q
    table = torch.full((3, 40), -1, dtype=torch.int32, device=DEV)
    table[:, :b.table.shape[1]] = b.table
    o = torch.zeros(3, 12, 64, dtype=BF16, device=DEV)
    got = b.cache.attend(wide[:, 4:8], table[:, :b.table.shape[1]], b.kv_len, 16, out=o[:, 8:])
    compare(got, K.attend(f64(q), b.k, b.v, cu), BF16)
    assert not o[:, :8].any()


def test_non_finite_entries_show_only_where_they_are_seen():
    b = Batch([60, 60], 4, 2, 128)
    bad = rand((1, 2, 128), BF16, 3)
    bad[0, 0, 5] = float("nan")
    b.cache.write(bad, bad, b.slots[20:21].to(DEV))       # entry 20 of request 0, kv head 0
    q, cu = b.queries([1, 1])
    got = b.cache.attend(q, b.table, b.kv_len, 16)
    assert torch.isnan(got.out[0, :2]).all() and torch.isnan(got.lse[0, :2]).all()
    got2 = b.cache.attend(q, b.table, b.kv_len, 16, window=39, sinks=20)
    b.k[0][20] = b.v[0][20] = 0
    compare(got2, K.attend(f64(q), b.k, b.v, cu, 39, 20), BF16)
    inf = q.clone()
    inf[1, 0, 0] = float("inf")
    got3 = b.cache.attend(inf, b.table, b.kv_len, 16, window=39, sinks=20)
    assert torch.isnan(got3.out[1, 0]).all() and torch.equal(got3.out[1, 1:], got2.out[1, 1:])


def test_bad_tables_are_reported_and_touch_nothing_else():
    b = Batch([40, 50, 60], 4, 2, 128)
    q, cu = b.queries([1, 1, 1])
    good = K.attend(f64(q), b.k, b.v, cu)
    for page in (-1, 10 ** 6, 2 ** 31 - 1):
        t = b.table.clone()
        t[1, 1] = page                           # entries 16..31 of request 1 are not seen
        got = b.cache.attend(q, t, b.kv_len, 16)
        assert b.cache.status() == 1 and b.cache.status() == 0
        cut = [b.k[0], np.delete(b.k[1], range(16, 32), 0), b.k[2]], [b.v[0], np.delete(b.v[1], range(16, 32), 0), b.v[2]]
        compare(got, K.attend(f64(q), *cut, cu), BF16)
    for n in (-1, 16 * b.table.shape[1] + 1, 2 ** 31 - 1):
        kv = b.kv_len.clone()
        kv[1] = n                                # an empty row
        got = b.cache.attend(q, b.table, kv, 16)
        assert b.cache.status() == 1
        ref = [x.copy() for x in good]
        ref[0][1], ref[1][1] = 0, -np.inf
        compare(got, ref, BF16)
    for wrong in ([0, 2, 1, 3], [0, -1, 2, 3], [0, 1, 2, 9], [0, 0, 3, 3]):
        out, lse = torch.full_like(q, 5.0), torch.full((3, 4), 5.0, device=DEV)
        b.cache.attend(q, b.table, b.kv_len, 16, cu_q=torch.tensor(wrong, dtype=torch.int32, device=DEV), max_q_len=2,
                       out=out, lse=lse)
        assert b.cache.status() == 1


@pytest.mark.parametrize("lens,Hq,H,d", [
    ([60000] + [100] * 19, 1, 1, 64),        # one unit over most of the CTAs, among others: parts added up in two steps
    ([6000] + [20] * 100, 4, 1, 128),        # short units, teams as workers, one of them over many teams
    ([9000] + [33] * 60, 12, 1, 256),        # the same with teams of four warps
    ([20000, 20000], 4, 1, 128),             # few units over many CTAs: added up by the second launch
    ([5000, 17, 4000, 900], 32, 2, 128),     # two chunks of rows a kv head
])
def test_units_over_many_workers(lens, Hq, H, d):
    b = Batch(lens, Hq, H, d, page=64)
    q, cu_q = b.queries([1] * len(lens))
    ref = K.attend(f64(q), b.k, b.v, cu_q)
    first = None
    for _ in range(3):                       # the counters are back at zero after each call
        got = b.cache.attend(q, b.table, b.kv_len, 64)
        compare(got, ref, BF16)
        assert first is None or (torch.equal(first.out, got.out) and torch.equal(first.lse, got.lse))
        first = got
    # another shape in between, on the same counters
    half = b.kv_len // 2
    got = b.cache.attend(q, b.table, half, 64)
    n = half.tolist()
    compare(got, K.attend(f64(q), [k[:m] for k, m in zip(b.k, n)], [v[:m] for v, m in zip(b.v, n)], cu_q), BF16)
    assert torch.equal(b.cache.attend(q, b.table, b.kv_len, 64).out, first.out) and b.cache.status() == 0


def test_requests_that_do_not_begin_at_row_zero():
    b = Batch([70, 30], 4, 2, 128)
    q, cu = b.queries([2, 1])
    shifted = torch.cat([rand((3, 4, 128), BF16, 2), q])
    out, lse = torch.full_like(shifted, 5.0), torch.full((6, 4), 5.0, device=DEV)
    b.cache.attend(shifted, b.table, b.kv_len, 16, cu_q=torch.from_numpy(cu + 3).to(DEV), max_q_len=2, out=out, lse=lse)
    assert (out[:3] == 5).all() and (lse[:3] == 5).all() and b.cache.status() == 0
    compare((out[3:], lse[3:]), K.attend(f64(q), b.k, b.v, cu), BF16)


def test_two_caches_on_two_streams():
    """Each cache has its own context: their calls may overlap."""
    work = []
    for i, (Hq, H, d) in enumerate([(8, 2, 128), (16, 2, 256)]):
        b = Batch([3000, 500, 40], Hq, H, d, seed=20 + i)
        q, cu = b.queries([1, 1, 1])
        work.append((b, q, K.attend(f64(q), b.k, b.v, cu), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for b, q, ref, stream in work:
            with torch.cuda.stream(stream):
                outs.append((b.cache.attend(q, b.table, b.kv_len, 16), ref))
    torch.cuda.synchronize()
    for got, ref in outs:
        compare(got, ref, BF16)


def test_results_repeat_bit_for_bit():
    b = Batch([3000, 17, 900], 8, 2, 128)
    q, cu = b.queries([2, 1, 2])
    cu = torch.from_numpy(cu).to(DEV)
    first = b.cache.attend(q, b.table, b.kv_len, 16, cu_q=cu, max_q_len=2)
    for _ in range(5):
        again = b.cache.attend(q, b.table, b.kv_len, 16, cu_q=cu, max_q_len=2)
        assert torch.equal(first.out, again.out) and torch.equal(first.lse, again.lse)


def test_two_captured_steps_and_an_eager_one():
    """Write and attend captured twice on one cache's stream; lengths change between replays."""
    b = Batch([300, 40], 8, 2, 128)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q, cu = b.queries([1, 1])
    k, v = rand((2, 2, 128), BF16, 31), rand((2, 2, 128), BF16, 32)
    slots = torch.full((2,), -1, dtype=torch.int64, device=DEV)
    graphs, outs = [], []
    with torch.cuda.stream(stream):
        for _ in range(2):
            b.cache.write(k, v, slots)
            b.cache.attend(q, b.table, b.kv_len, 16)
        for window in (0, 33):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                b.cache.write(k, v, slots)
                outs.append(b.cache.attend(q, b.table, b.kv_len, 16, window=window))
            graphs.append(g)
    torch.cuda.synchronize()
    for step in range(3):
        # replace the last entry of each request, then look at fewer entries every step
        lens = [300 - 7 * step, 40 - step]
        b.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        k.copy_(rand((2, 2, 128), BF16, 40 + step))
        cut = [0, 300]
        at = [cut[r] + lens[r] - 1 for r in range(2)]
        slots.copy_(b.slots[at])
        for r in range(2):
            b.k[r][lens[r] - 1] = K.cache_values(f64(k[r]), 0)
            b.v[r][lens[r] - 1] = K.cache_values(f64(v[r]), 0)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        kk, vv = [b.k[r][:lens[r]] for r in range(2)], [b.v[r][:lens[r]] for r in range(2)]
        for out, window in zip(outs, (0, 33)):
            compare(out, K.attend(f64(q), kk, vv, cu, window), BF16)
        compare(b.cache.attend(q, b.table, b.kv_len, 16), K.attend(f64(q), kk, vv, cu), BF16)


def test_entries_far_into_a_large_cache():
    """Byte offsets past 2^32: 4.8 GB of slots, the pages at its end."""
    from sparse_long_context_tail_gb300.kvcache import QuantKVCache
    H, d = 8, 256
    c = QuantKVCache(2 ** 21, H, d)
    T = 40
    slots = c.num_slots - 64 + torch.arange(T, device=DEV)
    k, v = rand((T, H, d), BF16, 1), rand((T, H, d), BF16, 2)
    c.write(k, v, slots)
    np.testing.assert_array_equal(f64(c.read(slots)[0]), K.cache_values(f64(k), 0))
    q = rand((1, 16, d), BF16, 3)
    table = torch.arange(c.num_slots // 16 - 4, c.num_slots // 16, device=DEV, dtype=torch.int32)[None]
    got = c.attend(q, table, torch.tensor([T], dtype=torch.int32, device=DEV), 16)
    compare(got, K.attend(f64(q), [K.cache_values(f64(k), 0)], [K.cache_values(f64(v), 0)], [0, 1]), BF16)


# ---------------------------------------------------- after the selection path --

def test_selected_tokens_are_written_at_their_slots_and_attended():
    """select_tokens -> the kept rows' K and V into the cache at slot_out -> the history's KV lengths -> attention."""
    from sparse_long_context_tail_gb300 import workload as wl
    from sparse_long_context_tail_gb300.selector import TokenSelector
    spec = wl.WorkloadSpec("kv", [900, 0, 1500], 8, 2, 128, 256, planted=[2, 0, 3], seed=31)
    w = wl.generate(spec)
    cu = w.cu_seqlens
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    k_full = up(w.k_bits.view(np.int16)).view(BF16)
    hidden = rand((w.total_tokens, 2 * 128), BF16, 3)          # stands for the rows the next layer projects V from
    R, cap = 3, 2
    hist, hlen = torch.zeros((R, cap, 2), dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int32, device=DEV)
    # every request has its own run of pages; a kept token's slot is where its page and offset are
    page = 32
    start = np.cumsum([0] + [-(-int(n) // page) for n in np.diff(cu)])
    table = torch.full((R, int(np.diff(start).max())), -1, dtype=torch.int32)
    perm = torch.randperm(int(start[-1]), generator=torch.Generator().manual_seed(2))
    for r in range(R):
        table[r, :start[r + 1] - start[r]] = perm[start[r]:start[r + 1]].int()
    sel = TokenSelector(0)
    out = sel.select_tokens(up(w.q_full_bits().view(np.int16)).view(BF16), k_full, cu, up(cu), 8, 2, 128, hidden,
                            layer_id=4, history=hist, history_len=hlen,
                            params=B.make_params(128, 64, 128, 128, 0.9))
    cu2 = out.cu_seqlens_out.cpu().numpy()
    total = int(out.total_kept)
    kept = out.kept_index.long()
    kept[total:] = 0
    slots = torch.full((w.total_tokens,), 1, dtype=torch.int64)      # rows past total_kept: a slot that must not change
    for r in range(R):
        e = torch.arange(int(cu2[r + 1] - cu2[r]))
        slots[cu2[r]:cu2[r + 1]] = table[r, e // page].long() * page + e % page
    c = make(int(start[-1]) * page, 2, 128)
    k, v = k_full[kept], out.hidden_out.view(-1, 2, 128)
    c.write(k, v, slots.to(DEV), out.total_kept)                    # no host read of the count
    kv = torch.empty(R, dtype=torch.int32, device=DEV)
    cu_dev = up(cu)
    batch, keep = B.make_batch(cu_dev.data_ptr(), cu, 8, 2, 128)
    B.upf_history_kv_len(sel.ctx, batch, hist.data_ptr(), hlen.data_ptr(), cap, 4, kv.data_ptr(),
                         torch.cuda.current_stream().cuda_stream)
    q = rand((R, 8, 128), BF16, 8)
    got = c.attend(q, table.to(DEV), kv, page, window=256, sinks=128)
    assert sel.status() == 0 and c.status() == 0
    assert kv.tolist() == np.diff(cu2).tolist() and total < w.total_tokens
    kk, vv = K.cache_values(f64(k[:total]), 0), K.cache_values(f64(v[:total]), 0)
    ref = K.attend(f64(q), [kk[cu2[r]:cu2[r + 1]] for r in range(R)], [vv[cu2[r]:cu2[r + 1]] for r in range(R)],
                   [0, 1, 2, 3], 256, 128)
    compare(got, ref, BF16)
    back = c.read(slots[:total].to(DEV))
    np.testing.assert_array_equal(f64(back[0]), kk)
    sel.close()


def test_a_wait_that_runs_out_is_reported_and_the_cache_recovers():
    """The copies' waits limited to one SM cycle, over a 300 MB cache (more than L2 holds), until some record is not
    there that soon.  The kernel reports it, waits for its own copies and returns, and the next calls are right."""
    n = 1 << 17
    big = make(n, 8, 128, fill=0)
    q = rand((1, 8, 128), BF16, 1)
    table = torch.randperm(n // 16, generator=torch.Generator().manual_seed(1)).int()[None].to(DEV)
    kv = torch.full((1,), n, dtype=torch.int32, device=DEV)
    B.upf_set_wait_limit(big.ctx, 1)
    for _ in range(200):
        big.attend(q, table, kv, 16)
        status = big.status()
        if status:
            break
    assert status == 6
    B.upf_set_wait_limit(big.ctx, 0)
    got = big.attend(q, table, kv, 16)
    assert big.status() == 0 and not got.out.any() and (got.lse - np.log(n)).abs().max() < 1e-5
    check(Batch([500, 300], 8, 4, 128), [1, 1])


# ------------------------------------------------------- logits of any size --

def peaked(lens, Hq, H, d, logit, twice=False, sign=1.0, dtype=BF16, page=16):
    """Requests in each of which one entry (`twice`: two, with the same keys) has a logit of about `logit` for every head
    and all others are far below: positive queries, its keys +6, the others' negative.  `sign` -1: every entry's
    keys are -6 instead.  Returns (batch, q, cu_q, entries that take all the weight)."""
    b = Batch(lens, Hq, H, d, page=page, dtype=dtype)
    cut = np.cumsum([0] + b.lens)
    T = int(cut[-1])
    k = -rand((T, H, d), dtype, 3).abs().clamp(2.0 ** -4, 6.0)
    if sign < 0:
        k = torch.full_like(k, -6.0)
    top = [sorted({n // 3, max(n - 2, 0)} if twice else {n // 3}) for n in b.lens]
    for r, at in enumerate(top):
        for e in at:
            k[cut[r] + e] = 6.0 * sign
    v = rand((T, H, d), dtype, 4)
    b.cache.write(k, v, b.slots.to(DEV))
    kk, vv = K.cache_values(f64(k), 0), K.cache_values(f64(v), 0)
    b.k, b.v = [kk[x:y] for x, y in zip(cut, cut[1:])], [vv[x:y] for x, y in zip(cut, cut[1:])]
    g = torch.Generator().manual_seed(5)
    q = (1 + torch.rand((len(lens), Hq, d), generator=g)) * (logit / (9 * d ** 0.5))     # scale sum q 6 = 9 sqrt(d) each
    return b, q.to(dtype).to(DEV), np.arange(len(lens) + 1), top


LAYOUTS = [([1, 40, 700], "teams"), ([6000] + [20] * 100, "a unit over many teams"), ([30000], "a second launch"),
           ([60000] + [100] * 19, "parts added up in two steps")]


@pytest.mark.parametrize("Hq,d", [(4, 64), (12, 64), (4, 128), (12, 128), (4, 256), (12, 256)])
@pytest.mark.parametrize("logit", [1e5, 1e7, 1e9, 1e12, 1e30])
def test_the_heaviest_entry_is_given_back_whatever_the_logits_size(logit, Hq, d):
    """Weights come from differences of logits: the entry with the largest one takes all the weight and its values come out
    exactly; two entries with the same keys share it, wherever they are."""
    for lens, _ in LAYOUTS if logit == 1e9 else LAYOUTS[:2] if logit == 1e7 else LAYOUTS[:1]:
        b, q, cu_q, top = peaked(lens, Hq, 1, d, logit)
        ref = K.attend(f64(q), b.k, b.v, cu_q)
        got = b.cache.attend(q, b.table, b.kv_len, 16)
        for r, at in enumerate(top):
            np.testing.assert_array_equal(f64(got.out[r]), np.broadcast_to(b.v[r][at[0]], (Hq, d)))
        assert (np.abs(f64(got.lse) - ref[1]) <= _bound(BF16, ref)[1]).all() and b.cache.status() == 0
        b, q, cu_q, top = peaked(lens, Hq, 1, d, logit, twice=True)
        got = b.cache.attend(q, b.table, b.kv_len, 16)
        for r, at in enumerate(top):
            # equal weights, an fp32 sum of two products and one rounding to bf16
            mean, size = b.v[r][at].mean(0), np.abs(b.v[r][at]).sum(0)
            assert (np.abs(f64(got.out[r]) - mean) <= np.abs(mean) * 2.0 ** -8 * (1 + 2.0 ** -10) + size * 2.0 ** -22).all()


@pytest.mark.parametrize("Hq,d", [(4, 64), (12, 128), (4, 256), (12, 256)])
def test_logits_past_fp32_are_nan_and_stay_by_themselves(Hq, d):
    """The largest logit of one head is past fp32's range, on either side: that row is NaN, the others are as without it,
    and a row that sees nothing is empty all the same."""
    for lens, _ in LAYOUTS[:3]:
        for sign in (1.0, -1.0):
            b, q, cu_q, top = peaked(lens, Hq, 1, d, 4.0, sign=sign)
            want = b.cache.attend(q, b.table, b.kv_len, 16)
            odd = q.clone()
            odd[0, 2] = 1e38 * (1.0 if sign > 0 else 1.5)
            got = b.cache.attend(odd, b.table, b.kv_len, 16)
            assert got.out[0, 2].isnan().all() and got.lse[0, 2].isnan()
            for g, w in zip(got, want):
                same = torch.ones_like(g, dtype=torch.bool)
                same[0, 2] = False
                assert torch.equal(g[same], w[same])
    b = Batch([1, 5], Hq, 1, d, k_exp=32, scale=2.0 ** 32)            # 2^k_exp takes the factor past fp32 before any product
    q, cu_q = b.queries([2, 1], scale=2.0 ** 110)
    got = b.cache.attend(q, b.table, b.kv_len, 16, cu_q=torch.from_numpy(cu_q).to(DEV), max_q_len=2)
    assert not got.out[0].any() and torch.isneginf(got.lse[0]).all()
    assert got.out[1:].isnan().all() and got.lse[1:].isnan().all() and b.cache.status() == 0


def test_scales_at_the_ends_of_fp32():
    """softmax_scale below the smallest normal fp32 number under large queries, and a large one over small ones."""
    for scale, size, k_exp in ((2.0 ** -140, 2.0 ** 120, 17), (2.0 ** 120, 2.0 ** -100, -21), (2.0 ** 127, 2.0 ** -126, -2)):
        b = Batch([77, 200, 1], 6, 3, 128, k_exp=k_exp, scale=2.0 ** k_exp)
        check(b, [1, 1, 1], scale=scale, q_scale=size)


@pytest.mark.parametrize("Hq,d", [(4, 64), (12, 128), (16, 256)])
def test_an_infinite_query_is_nan_wherever_it_sees_something(Hq, d):
    """Keys of one sign where the query is infinite: every logit is -inf (or +inf), and their softmax is 0 / 0."""
    b = Batch([1, 300], Hq, 1, d)
    k = rand((301, 1, d), BF16, 3)
    k[..., 7] = -k[..., 7].abs().clamp(min=2.0)
    k[..., 0] = 12.0
    b.cache.write(k, k, b.slots.to(DEV))
    assert (b.cache.read(b.slots.to(DEV))[0][..., 7] < 0).all()
    q, cu_q = b.queries([2, 1])                      # the first query sees nothing
    ask = lambda x: b.cache.attend(x, b.table, b.kv_len, 16, cu_q=torch.from_numpy(cu_q).to(DEV), max_q_len=2)  # noqa: E731
    want = ask(q)
    for x in (float("inf"), float("-inf")):
        odd = q.clone()
        odd[0, 1, 7] = odd[1, 2, 7] = odd[2, 3, 7] = x
        got = ask(odd)
        assert not got.out[0].any() and torch.isneginf(got.lse[0]).all()
        for at in ((1, 2), (2, 3)):
            assert got.out[at].isnan().all() and got.lse[at].isnan()
        for g, w in zip(got, want):
            same = torch.ones_like(g, dtype=torch.bool)
            same[1, 2] = same[2, 3] = False
            assert torch.equal(g[same], w[same])
    assert b.cache.status() == 0


def test_a_cache_made_and_used_on_one_stream_while_another_is_busy():
    """Its device words are zero before the first call on any stream, and its status is read and cleared in order with the
    caller's stream alone: half a second of work on the default stream neither delays nor undoes anything."""
    from sparse_long_context_tail_gb300.kvcache import QuantKVCache
    b = Batch([20000, 20000], 4, 1, 128, page=64)    # units that are added up by their last worker and by a second launch
    s = Batch([6000] + [20] * 100, 4, 1, 128)
    work = [(x, x.queries([1] * len(x.lens))[0], x.page) for x in (b, s)]
    refs = [K.attend(f64(q), x.k, x.v, np.arange(len(x.lens) + 1)) for x, q, _ in work]
    bad = s.table.clone()
    bad[5, 0] = -3
    for x, q, p in work:                             # a kernel's first launch in a process waits for the device
        x.cache.attend(q, x.table, x.kv_len, p)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(10 ** 9)
    with torch.cuda.stream(side):
        made = [QuantKVCache(x.cache.num_slots, 1, 128, storage=x.cache.storage) for x, _, _ in work]
        got = [[c.attend(q, x.table, x.kv_len, p) for _ in range(3)] for c, (x, q, p) in zip(made, work)]
        made[1].attend(work[1][1], bad, s.kv_len, 16)
        reported = made[1].status(), made[1].status(), made[0].status()
        got[1].append(made[1].attend(work[1][1], s.table, s.kv_len, 16))
        side.synchronize()
        busy = not torch.cuda.default_stream().query()
    torch.cuda.synchronize()
    assert reported == (1, 0, 0)
    for outs, ref in zip(got, refs):
        for x in outs:
            compare(x, ref, BF16)
    assert busy, "the calls waited for the default stream"


@pytest.mark.parametrize("Hq,H,d", [(4, 4, 256), (64, 4, 256), (128, 8, 128)])
def test_a_wait_that_runs_out_in_teams_of_several_warps(Hq, H, d):
    """As above, where two or four warps work on a tile: the warps of a team give up together, whichever lane's wait ran out,
    and so they do where the cache's units are short and each team is its own worker."""
    n = (1 << 20) // (H * d // 128)                  # 151 MB
    big = make(n, H, d, fill=0)
    table = torch.randperm(n // 16, generator=torch.Generator().manual_seed(1)).int().to(DEV)
    for R in (1, n // 1024):
        q = rand((R, Hq, d), BF16, 1)
        kv = torch.full((R,), n // R, dtype=torch.int32, device=DEV)
        ask = lambda: big.attend(q, table.view(R, -1), kv, 16)  # noqa: E731
        B.upf_set_wait_limit(big.ctx, 1)
        for _ in range(200):
            ask()
            status = big.status()
            if status:
                break
        assert status == 6
        B.upf_set_wait_limit(big.ctx, 0)
        got = ask()
        assert big.status() == 0 and not got.out.any() and (got.lse - np.log(n // R)).abs().max() < 1e-5


# ----------------------------------------------------------- more of the above --

def test_inconsistent_row_ranges_touch_only_the_good_requests():
    """cu_q that is not ascending, leaves the rows or holds more than max_q_len rows: such a request is skipped, its rows are
    left as they are and the others are right."""
    b = Batch([40, 50, 60], 4, 2, 128)
    q, _ = b.queries([1, 1, 1])
    lone = [K.attend(f64(q[r:r + 1]), b.k[r:r + 1], b.v[r:r + 1], [0, 1]) for r in range(3)]
    # the rows of each good request, with the oracle's view of it
    two = K.attend(f64(q[:2]), b.k[:1], b.v[:1], [0, 2])
    tail = K.attend(f64(q[2:3]), b.k[2:], b.v[2:], [0, 1])
    for wrong, kept, good in (([0, 0, 3, 3], [0, 1, 2], []), ([0, -1, 2, 3], [0, 1], [(2, 3, tail)]),
                              ([0, 1, 2, 9], [2], [(0, 1, lone[0]), (1, 2, lone[1])]),
                              ([0, 2, 1, 3], [], [(0, 1, [x[:1] for x in two])]),   # row 1 is given to two requests
                              ([0, 1, 2 ** 31 - 1, 3], [1, 2], [(0, 1, lone[0])]), ([3, 3, 3, 3], [0, 1, 2], [])):
        out, lse = torch.full_like(q, 5.0), torch.full((3, 4), 5.0, device=DEV)
        b.cache.attend(q, b.table, b.kv_len, 16, cu_q=torch.tensor(wrong, dtype=torch.int32, device=DEV), max_q_len=2,
                       out=out, lse=lse)
        assert b.cache.status() == (0 if wrong == [3, 3, 3, 3] else 1)
        assert (out[kept] == 5).all() and (lse[kept] == 5).all(), wrong
        for x, y, ref in good:
            compare((out[x:y], lse[x:y]), ref, BF16)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,d", [(12, 64), (4, 256), (12, 128), (4, 64)])
@pytest.mark.parametrize("lens", [[60000] + [100] * 19, [6000] + [20] * 100, [20000, 20000]])
def test_units_over_many_workers_at_every_shape(lens, Hq, d, dtype):
    """Eight and sixteen rows of each head size: parts added up in two steps, by teams, and by the second launch."""
    b = Batch(lens, Hq, 1, d, page=64, dtype=dtype)
    q, got, ref = check(b, [1] * len(lens))
    again = b.cache.attend(q, b.table, b.kv_len, 64)
    assert torch.equal(got.out, again.out) and torch.equal(got.lse, again.lse)


@pytest.mark.parametrize("seed", range(60))
def test_random_batches(seed):
    r = np.random.default_rng(1000 + seed)
    pick = lambda *x: x[r.integers(len(x))]  # noqa: E731
    Hq, H, d = pick((8, 2, 64), (5, 1, 64), (40, 2, 64), (8, 2, 128), (28, 4, 128), (4, 4, 128), (32, 2, 128), (16, 2, 256),
                    (9, 1, 256), (24, 2, 256))
    R = pick(1, 2, 3, 8, 20, 60, 300)
    top = pick(1, 16, 40, 200, 1000, 3000) if R < 60 else pick(1, 20, 100)
    lens = r.integers(0, top + 1, R)
    if r.random() < 0.2:
        lens[r.integers(R)] = r.integers(2000, 9000)
    q_len = pick(1, 1, 2, 5, 17, 60) if R <= 20 else pick(1, 2)
    news = r.integers(0 if q_len > 1 else 1, q_len + 1, R)
    news[0] = max(news[0], 1)
    window = int(pick(0, 0, 1, 5, 33, 64, 300, 5000))
    b = Batch(lens.tolist(), Hq, H, d, page=int(pick(16, 32, 64, 128)), dtype=pick(BF16, F16), seed=seed,
              k_exp=int(r.integers(-3, 4)), v_exp=int(r.integers(-3, 4)), scale=pick(0.2, 1, 3))
    check(b, news.tolist(), window=window, sinks=int(pick(0, 1, 4, 17, 100)) if window else 0, q_scale=pick(0.1, 1, 4))


# ------------------------------------------- calls at the ends of what is allowed --

def test_outputs_that_may_be_left_out():
    """upf_kv_read of keys or values alone, and upf_kv_attend without lse, give what the full calls give."""
    b = Batch([300, 40], 8, 2, 128)
    c, slots = b.cache, b.slots.to(DEV)
    T, width = len(slots), 2 * 128
    k, v = c.read(slots)
    for of in range(2):
        out = [torch.full_like(k, 3.0), torch.full_like(v, 3.0)]
        ptr = [x.data_ptr() if i == of else 0 for i, x in enumerate(out)]
        B.upf_kv_read(c.ctx, c._cache, B.UPF_BF16, slots.data_ptr(), T, 0, ptr[0], width, ptr[1], width, c._stream())
        assert torch.equal(out[of], (k, v)[of]) and (out[1 - of] == 3).all()
    q, _ = b.queries([1, 1])
    want = c.attend(q, b.table, b.kv_len, 16)
    query, keep = B.make_kv_query(2, 8, 2, b.kv_len.data_ptr(), b.table.data_ptr(), b.table.shape[1], b.table.shape[1], 16)
    ws = torch.empty(B.upf_kv_attend_workspace_bytes(c._cache, query), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    B.upf_kv_attend(c.ctx, c._cache, query, B.UPF_BF16, q.data_ptr(), 8 * 128, out.data_ptr(), 8 * 128, 0, ws.data_ptr(),
                    ws.numel(), c._stream())
    assert torch.equal(out, want.out) and c.status() == 0


def test_a_captured_long_write_with_other_slots_and_counts():
    """More tokens than a call without a workspace takes, captured once: replays follow slots, count and values."""
    T, H, d = 3000, 2, 64
    c = make(16 * 300, H, d, fill=0)
    k, v = rand((T, H, d), BF16, 1), rand((T, H, d), BF16, 2)
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    count = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.write(k, v, slots, count)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.write(k, v, slots, count)
    held = {}
    for step, n in enumerate((T, 17, 0, 2500)):
        s = torch.randint(-2, c.num_slots, (T,), generator=torch.Generator().manual_seed(step))
        k.copy_(rand((T, H, d), BF16, 10 + step))
        v.copy_(rand((T, H, d), BF16, 20 + step))
        slots.copy_(s)
        count.fill_(n)
        g.replay()
        kk, vv = K.cache_values(f64(k), 0), K.cache_values(f64(v), 0)
        for t in range(n):
            if s[t] >= 0:
                held[int(s[t])] = kk[t], vv[t]
        at = list(held)
        got = c.read(torch.tensor(at, device=DEV))
        for of in range(2):
            np.testing.assert_array_equal(f64(got[of]), np.stack([held[x][of] for x in at]))
    assert c.status() == 0


@pytest.mark.parametrize("Hq,H,d,lens,news", [
    (256, 256, 64, [70, 1, 0], [2, 1, 1]),             # as many kv heads as there may be
    (256, 1, 64, [70, 33], [1, 3]),                    # all q heads on one
    (8, 2, 64, [1500, 1024, 600], [1024, 1024, 1024]),  # as many new tokens as there may be: some rows see nothing
    (4, 2, 128, [2100], [1024]),
])
def test_the_largest_head_counts_and_prompt_chunks(Hq, H, d, lens, news):
    b = Batch(lens, Hq, H, d)
    check(b, news)
    check(b, news, window=50, sinks=3)


def test_thousands_of_requests():
    rng = np.random.default_rng(6)
    check(Batch(rng.integers(0, 25, 3000).tolist(), 2, 1, 64), [1] * 3000)
    check(Batch(rng.integers(0, 100, 700).tolist(), 4, 1, 256), [1] * 700, window=20, sinks=2)


def test_windows_first_tokens_and_pages_as_large_as_they_come():
    b = Batch([1000, 40, 3], 8, 2, 128)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 30, 2 ** 31 - 1), (2 ** 30 - 1, 1), (7, 2 ** 31 - 1)):
        check(b, [2, 1, 5], window=window, sinks=sinks)
    check(Batch([70000], 2, 1, 64, page=65536, spare=0), [3], window=66000, sinks=100)
    full = Batch([64, 32], 4, 2, 128, page=32)          # kv_len fills the table
    full.table = full.table[:, :2].contiguous()
    check(full, [1, 1])
