"""Accumulated attention weights and eviction on the GPU against the float64 oracle.

An eviction is whole numbers and moved bytes: lists, lengths, weights and cache contents equal the
oracle's.  Accumulated weights are compared with a tolerance derived from the arithmetic (`close`).
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


def f64(t):
    return t.cpu().double().numpy()


class Batch:
    """A cache with requests of `lens` entries in pages of their own."""

    def __init__(self, lens, H, d, page=16, dtype=BF16, seed=0, k_exp=0, v_exp=0, spare=3, more_pages=0, scale=1.0):
        from sparse_long_context_tail_gb300.kvcache import QuantKVCache
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.d, self.page, self.k_exp, self.v_exp = list(lens), H, d, page, k_exp, v_exp
        need = [-(-n // page) for n in lens]
        order = torch.randperm(sum(need) + spare, generator=g).int()
        self.free = order[sum(need):]
        width = max(max(need), 1) + more_pages
        table = torch.full((len(lens), width), -7, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = order[at:at + n]
            at += n
        self.table = table.to(DEV)
        self.cache = QuantKVCache(order.numel() * page, H, d, k_exp=k_exp, v_exp=v_exp)
        self.cache.storage.fill_(0xA5)
        self.slots = [self.slot_list(self.table[r], n) for r, n in enumerate(lens)]
        T = sum(lens)
        k = torch.randn(T, H, d, generator=g) * torch.exp(0.4 * torch.randn(H, d, generator=g)) * 2.0 ** k_exp * scale
        v = torch.randn(T, H, d, generator=g) * 2.0 ** v_exp
        self.k, self.v = k.to(dtype).to(DEV), v.to(dtype).to(DEV)
        if T:
            self.cache.write(self.k, self.v, torch.cat(self.slots))
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def slot_list(self, row, n):
        e = torch.arange(n, device=DEV)
        return row[e // self.page].long() * self.page + e % self.page

    def keys(self):
        """Float64 keys of each request as the cache holds them."""
        k = K.cache_values(f64(self.k), self.k_exp)
        return np.split(k, np.cumsum(self.lens)[:-1])

    def contents(self, slots):
        k, v = self.cache.read(slots)
        return k.view(torch.int16), v.view(torch.int16)


# ------------------------------------------------------------- accumulating --

def queries(news, Hq, d, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(news), Hq, d, generator=g) * torch.exp2(torch.randint(-2, 2, (sum(news), Hq, 1), generator=g).float())
    cu = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device=DEV)
    return (q * scale).to(dtype).to(DEV), cu


def close(got, old, decay, drawn, slack, d, rows):
    """weights = decay old + sum of `rows` terms exp(x - lse), within the arithmetic:

    a logit's product sums d terms in fp32 (2^-23 of their magnitudes each time, truncating) of a query rounded by
    2^-25 of the row's largest element; logit factor, difference, the part 2^-48 of lse and exp2 (2^-22 of its value,
    2^-24 |x| of its argument): under 2^-22 (|x| + 1) with |x| <= reach + |lse|; then the sum's own roundings."""
    want = decay * old + drawn
    bound = (slack["reach"] * (d + 8) * 2.0 ** -23 + slack["flat"] * 2.0 ** -25 + slack["far"] * 2.0 ** -22
             + slack["one"] * 2.0 ** -21 + (rows + 2) * 2.0 ** -24 * (np.abs(want) + np.abs(old)) + 2.0 ** -125 * rows)
    off = np.abs(got - want)
    assert (off <= bound).all(), ((off / bound).max(), int((off / bound).argmax()))


def check_accumulate(b, news, Hq, dtype=BF16, window=0, sinks=0, decay=1.0, scale=None, kv_of_q=None, plain=False, seed=5,
                     q_scale=1.0, rows=None):
    q, cu = queries(news, Hq, b.d, dtype, seed, q_scale * 2.0 ** -b.k_exp)
    if rows is not None:          # what each row is multiplied by
        q = q * rows.to(q)[:, :, None]
    cuq = None if plain else cu
    kw = dict(cu_q=cuq, max_q_len=max(max(news), 1), window=window, sinks=sinks, softmax_scale=scale, kv_of_q=kv_of_q)
    lse = b.cache.attend(q, b.table, b.kv_len, b.page, **kw).lse
    cols = b.table.shape[1] * b.page + 5
    g = torch.Generator().manual_seed(seed + 1)
    old = torch.rand(len(news), cols, generator=g).to(DEV)
    out = torch.full_like(old, 7.0)
    got = b.cache.accumulate(q, lse, b.table, b.kv_len, b.page, old, decay=decay, out=out, **kw)
    assert got is out
    drawn, slack = K.accumulate(f64(q), f64(lse), b.keys(), cu.tolist(), window, sinks, scale, kv_of_q)
    for r, n in enumerate(b.lens):
        if news[r] == 0:
            n = 0
        close(f64(out[r, :n]), decay * 0 + f64(old[r, :n]), decay, drawn[r][:n], {k: v[:n] for k, v in slack[r].items()}, b.d,
              news[r] * Hq)
        assert (out[r, n:] == 7.0).all()
    assert b.cache.status() == 0
    # in place, and from zero; the same bits every time
    mine = old.clone()
    b.cache.accumulate(q, lse, b.table, b.kv_len, b.page, mine, decay=decay, **kw)
    zero = torch.zeros_like(old)
    b.cache.accumulate(q, lse, b.table, b.kv_len, b.page, None, out=zero, **kw)
    from_zero = b.cache.accumulate(q, lse, b.table, b.kv_len, b.page, torch.zeros_like(old), **kw)
    for r, n in enumerate(b.lens):
        n = n if news[r] else 0
        assert torch.equal(mine[r, :n], out[r, :n]) and torch.equal(mine[r, n:], old[r, n:])
    assert torch.equal(zero, from_zero)
    return q, lse, zero


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,H,d", [(8, 2, 64), (5, 1, 64), (32, 8, 128), (4, 4, 128), (12, 1, 128), (16, 2, 256), (3, 3, 256)])
def test_one_new_token_each(Hq, H, d, dtype):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 200, 331]
    check_accumulate(Batch(lens, H, d, k_exp=1), [1] * len(lens), Hq, dtype, plain=True)


@pytest.mark.parametrize("Hq,H,d", [(8, 2, 64), (16, 2, 128), (28, 4, 128), (16, 8, 256)])
@pytest.mark.parametrize("news", [[3, 1, 0, 4, 2], [9, 17, 1, 8, 16], [33, 40, 2, 64, 31]])
def test_several_new_tokens(Hq, H, d, news):
    check_accumulate(Batch([70, 5, 40, 129, 2], H, d, page=32, seed=3), news, Hq, decay=0.75)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (20, 5), (100, 37), (1000, 4), (2 ** 30, 0), (2 ** 31 - 1, 0)])
@pytest.mark.parametrize("news", [[1, 1, 1], [7, 2, 30]])
def test_windows_and_first_entries(window, sinks, news):
    check_accumulate(Batch([150, 64, 33], 2, 64, seed=4), news, 6, window=window, sinks=sinks, decay=0.5)


def test_more_rows_than_entries_and_long_queries():
    check_accumulate(Batch([3, 1, 0, 300], 2, 128, seed=6), [5, 4, 2, 200], 8)
    check_accumulate(Batch([1100], 1, 64, seed=7), [1024], 2)


def test_head_maps_scales_and_exponents():
    check_accumulate(Batch([90, 31], 2, 128, k_exp=-7), [1, 3], 6, scale=0.31, kv_of_q=[1, 0, 0, 1, 1, 0])
    check_accumulate(Batch([90, 31], 2, 128, k_exp=13, dtype=BF16), [1, 3], 6, kv_of_q=[1, 0, 0, 1, 1, 0])
    check_accumulate(Batch([64], 256, 64, seed=8), [1], 256)


@pytest.mark.parametrize("page", [16, 64, 4096])
def test_page_sizes(page):
    check_accumulate(Batch([10, 5000, 333], 2, 64, page=page, seed=9, more_pages=2), [1, 2, 1], 4)


def test_many_requests():
    lens = [(7 * i) % 40 for i in range(700)]
    check_accumulate(Batch(lens, 1, 64, seed=10), [i % 3 for i in range(700)], 2)


@pytest.mark.parametrize("Hq,H,d", [(5, 5, 64), (7, 7, 128), (24, 24, 64), (25, 25, 64), (32, 32, 128), (64, 64, 64), (49, 7, 128),
                                    (24, 3, 256), (200, 100, 64), (256, 32, 64), (11, 11, 256)])
def test_few_rows_of_any_number_of_heads(Hq, H, d):
    check_accumulate(Batch([130, 1, 700, 16], H, d, seed=50), [1] * 4, Hq, window=300, sinks=20)


@pytest.mark.parametrize("Hq,H,d", [(9, 1, 64), (64, 1, 128), (128, 1, 256), (256, 1, 64), (256, 2, 128), (20, 2, 256), (45, 5, 64)])
def test_many_rows_of_one_new_token(Hq, H, d):
    check_accumulate(Batch([130, 1, 2500, 16, 0, 129], H, d, seed=51), [1] * 6, Hq, plain=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("low", [-14, -15, -40])
@pytest.mark.parametrize("news,Hq", [([3, 20, 1], 16), ([70, 5, 33], 8), ([1, 1, 1], 4)])
def test_rows_far_apart(news, Hq, low, d):
    """Largest elements of a request's rows 2^14 apart, just further, and much further; some rows of zeros."""
    g = torch.Generator().manual_seed(52)
    rows = torch.exp2(torch.randint(low, 1, (sum(news), Hq), generator=g).float())
    rows[torch.rand(rows.shape, generator=g) < 0.1] = 0.0
    check_accumulate(Batch([300, 40, 129], 2, d, seed=53), news, Hq, rows=rows)


@pytest.mark.parametrize("seed", range(16))
def test_drawn_batches(seed):
    g = np.random.default_rng(600 + seed)
    d, H = int(g.choice([64, 128, 256])), int(g.integers(1, 9))
    Hq = H * int(g.integers(1, 9))
    R = int(g.integers(1, 9))
    lens = [int(x) for x in np.floor(np.exp(g.uniform(0, np.log(3000), R)))]
    most = int(g.choice([1, 2, 6, 60]))
    news = [int(x) for x in g.integers(0, most + 1, R)]
    if sum(news) == 0:
        news[0] = 1
    window = int(g.choice([0, 0, 1, 17, 128, 500]))
    b = Batch(lens, H, d, page=int(g.choice([16, 32, 128])), dtype=BF16 if seed % 2 else F16, seed=seed, k_exp=int(g.integers(-2, 3)))
    check_accumulate(b, news, Hq, dtype=BF16 if seed % 2 else F16, window=window, sinks=int(g.integers(0, 40)),
                     decay=float(g.choice([0.0, 0.5, 1.0])), seed=seed)


def test_a_wait_of_an_accumulation_that_runs_out_is_reported():
    """With a limit of one cycle the kernel gives up and says so; the context stays usable."""
    b = Batch([3000, 200], 2, 128, seed=54)
    q, cu = queries([40, 9], 8, 128, BF16, 55)
    kw = dict(cu_q=cu, max_q_len=40)
    lse = b.cache.attend(q, b.table, b.kv_len, 16, **kw).lse
    assert b.cache.status() == 0
    B.upf_set_wait_limit(b.cache.ctx, 1)
    b.cache.accumulate(q, lse, b.table, b.kv_len, 16, torch.zeros(2, 3000, device=DEV), **kw)
    assert b.cache.status() == 6
    B.upf_set_wait_limit(b.cache.ctx, 0)
    check_accumulate(b, [40, 9], 8)


def test_weights_of_a_row_add_up_to_one():
    b = Batch([5000, 77], 4, 128, seed=11)
    q, lse, w = check_accumulate(b, [1, 1], 8)
    assert np.allclose(f64(w[:, :5000]).sum(1), 8, rtol=1e-5)


def test_rows_that_are_not_finite_add_nothing():
    b = Batch([40, 50, 60], 2, 64, seed=12)
    q, cu = queries([1, 2, 1], 4, 64, BF16, 13)
    kw = dict(cu_q=cu, max_q_len=2)
    lse = b.cache.attend(q, b.table, b.kv_len, 16, **kw).lse
    base = b.cache.accumulate(q, lse, b.table, b.kv_len, 16, torch.zeros(3, 64, device=DEV), **kw)
    assert b.cache.status() == 0
    for i, (where, what) in enumerate([("q", "nan"), ("q", "inf"), ("lse", "nan"), ("lse", "inf"), ("lse", "-inf")]):
        q2, l2 = q.clone(), lse.clone()
        if where == "q":
            q2[2, 1, 17] = float(what)
        else:
            l2[2, 1] = float(what)
        got = b.cache.accumulate(q2, l2, b.table, b.kv_len, 16, torch.zeros(3, 64, device=DEV), **kw)
        assert b.cache.status() == (0 if what == "-inf" else 5)
        assert torch.equal(got[0], base[0]) and torch.equal(got[2], base[2])
        l2 = lse.clone()
        l2[2, 1] = float("-inf")
        drawn, slack = K.accumulate(f64(q), f64(l2), b.keys(), cu.tolist())
        close(f64(got[1, :50]), 0 * drawn[1], 1.0, drawn[1], slack[1], 64, 8)


def test_a_key_with_a_nan_marks_its_entry_alone():
    b = Batch([40], 2, 64, seed=14)
    q, cu = queries([1], 4, 64, BF16, 15)
    lse = b.cache.attend(q, b.table, b.kv_len, 16).lse
    base = b.cache.accumulate(q, lse, b.table, b.kv_len, 16, torch.zeros(1, 64, device=DEV))
    k = b.k.clone()
    k[17, 1, 5] = float("nan")
    b.cache.write(k, b.v, b.slots[0])
    got = b.cache.accumulate(q, lse, b.table, b.kv_len, 16, torch.zeros(1, 64, device=DEV))
    assert torch.isnan(got[0, 17]) and torch.equal(got[0, :17], base[0, :17]) and torch.equal(got[0, 18:], base[0, 18:])


def test_tables_that_make_no_sense():
    b = Batch([40, 50, 60, 20], 2, 64, seed=16)
    q, cu = queries([1, 1, 1, 1], 4, 64, BF16, 17)
    lse = b.cache.attend(q, b.table, b.kv_len, 16).lse
    old = torch.rand(4, 64, device=DEV)
    base = b.cache.accumulate(q, lse, b.table, b.kv_len, 16, old, out=old.clone())
    for bad in (-1, 65, 2 ** 31 - 1, -2 ** 31):
        n = b.kv_len.clone()
        n[1] = bad
        got = b.cache.accumulate(q, lse, b.table, n, 16, old, out=old.clone())
        assert b.cache.status() == 1
        assert torch.equal(got[1], old[1]) and torch.equal(got[[0, 2, 3]], base[[0, 2, 3]])
    # more entries than weights
    n = b.kv_len.clone()
    got = b.cache.accumulate(q, lse, b.table, n, 16, old[:, :50].contiguous(), out=old[:, :50].contiguous())
    assert b.cache.status() == 1 and torch.equal(got[2], old[2, :50]) and torch.equal(got[1], base[1, :50])
    for page in (-1, b.cache.num_slots // 16, 2 ** 31 - 1, -2 ** 31):
        t = b.table.clone()
        t[2, 1] = page
        got = b.cache.accumulate(q, lse, t, b.kv_len, 16, old, out=old.clone())
        assert b.cache.status() == 1
        want = base.clone()
        want[2, 16:32] = old[2, 16:32]
        assert torch.equal(got, want)
    # bad pages that no row sees are not looked at
    t = b.table.clone()
    t[2, 1] = -1
    b.cache.accumulate(q, lse, t, b.kv_len, 16, old.clone(), window=20, sinks=2)
    assert b.cache.status() == 0
    for rows in ([0, 2, 1, 3, 4], [0, 1, 2, 3, 9], [-1, 1, 2, 3, 4], [0, 0, 3, 3, 4]):
        c = torch.tensor(rows, dtype=torch.int32, device=DEV)
        got = b.cache.accumulate(q, lse, b.table, b.kv_len, 16, old, out=old.clone(), cu_q=c, max_q_len=2)
        assert b.cache.status() == 1
        for r in range(4):
            if not 0 <= rows[r] <= rows[r + 1] <= 4 or rows[r + 1] - rows[r] > 2 or rows[r] == rows[r + 1]:
                assert torch.equal(got[r], old[r])
            elif rows[r] == r and rows[r + 1] == r + 1:
                assert torch.equal(got[r], base[r])


def test_weights_with_strides_and_accumulate_in_a_graph():
    b = Batch([40, 50], 2, 64, seed=18, more_pages=4)
    q, cu = queries([1, 1], 4, 64, BF16, 19)
    lse = b.cache.attend(q, b.table, b.kv_len, 16).lse
    wide = torch.rand(2, 200, device=DEV)
    old = wide.clone()
    part = wide[:, 30:130]
    b.cache.accumulate(q, lse, b.table, b.kv_len, 16, part)
    want = b.cache.accumulate(q, lse, b.table, b.kv_len, 16, old[:, 30:130].contiguous())
    assert torch.equal(part, want) and torch.equal(wide[:, :30], old[:, :30]) and torch.equal(wide[:, 130:], old[:, 130:])
    w = torch.zeros(2, 100, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.cache.accumulate(q, lse, b.table, b.kv_len, 16, w)
    for n in ([40, 50], [3, 17]):
        b.kv_len.copy_(torch.tensor(n, dtype=torch.int32))
        lse.copy_(b.cache.attend(q, b.table, b.kv_len, 16).lse)
        w.zero_()
        graph.replay()
        graph.replay()
        once = b.cache.accumulate(q, lse, b.table, b.kv_len, 16, torch.zeros(2, 100, device=DEV))
        assert torch.equal(w, 2 * once)


def test_two_graphs_of_many_rows_on_two_streams():
    b = Batch([700, 90], 2, 64, seed=56)
    graphs, want = [], []
    for i, news in enumerate(([20, 3], [2, 31])):
        q, cu = queries(news, 8, 64, BF16, 57 + i)
        kw = dict(cu_q=cu, max_q_len=31)
        lse = b.cache.attend(q, b.table, b.kv_len, 16, **kw).lse
        want.append(b.cache.accumulate(q, lse, b.table, b.kv_len, 16, torch.zeros(2, 704, device=DEV), **kw))
        w = torch.zeros(2, 704, device=DEV)
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            w.zero_()
            b.cache.accumulate(q, lse, b.table, b.kv_len, 16, w, **kw)
        graphs.append((graph, stream, w, (q, cu, lse)))
    for _ in range(20):
        for graph, stream, _, _ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(graphs, want):
            assert torch.equal(x[2], y)
            x[2].fill_(9.0)
    assert b.cache.status() == 0


def test_a_cache_and_weights_past_32_bits_of_bytes():
    """The same entries near the start and at the far end of a cache of 5 GB, weights 8 GiB apart."""
    from sparse_long_context_tail_gb300.kvcache import QuantKVCache
    H, d, n, page = 8, 128, 300, 16
    cache = QuantKVCache(1 << 22, H, d)
    assert cache.storage.numel() > 2 ** 32
    need, last = -(-n // page), (1 << 22) // page - 1
    near, far = torch.arange(need), last - torch.arange(need)
    table = torch.stack([near, far]).int().to(DEV)
    g = torch.Generator().manual_seed(58)
    k, v = torch.randn(n, H, d, generator=g).to(BF16).to(DEV), torch.randn(n, H, d, generator=g).to(BF16).to(DEV)
    e = torch.arange(n, device=DEV)
    slots = [table[r, e // page].long() * page + e % page for r in range(2)]
    for s in slots:
        cache.write(k, v, s)
    kv_len = torch.full((2,), n, dtype=torch.int32, device=DEV)
    room = torch.empty(2 ** 31 + 512, device=DEV)
    w = room.as_strided((2, 304), (2 ** 31, 1))
    for news in (1, 5):
        q, _ = queries([news], 32, d, BF16, 59)
        q = torch.cat([q, q])
        kw = dict(cu_q=torch.tensor([0, news, 2 * news], dtype=torch.int32, device=DEV), max_q_len=news)
        lse = cache.attend(q, table, kv_len, page, **kw).lse
        w.zero_()
        cache.accumulate(q, lse, table, kv_len, page, w, **kw)
        assert torch.equal(w[0], w[1]) and float(w[0, :n].sum()) > 31 * news and not w[:, n:].any()
    old = w.clone()
    kept = cache.evict(w, table, kv_len, page, 100, recent=10)
    assert cache.status() == 0 and torch.equal(kept[0], kept[1]) and kv_len.tolist() == [100, 100]
    want = K.evict(old[0, :n].tolist(), 100, 100, 0, 10)
    assert kept[0].tolist() == want and torch.equal(w[0], w[1])
    (k0, v0), (k1, v1) = (cache.read(s[:100]) for s in slots)
    assert torch.equal(k0, k1) and torch.equal(v0, v1)


# ------------------------------------------------------------------ eviction --

def weights_of(lens, cols, seed, kind="mixed"):
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(3 * torch.randn(len(lens), cols, generator=g) - 3)
    if kind == "mixed":            # many equal ones
        w = torch.where(w < 0.05, torch.zeros(()), w)
        w = torch.where(torch.rand(w.shape, generator=g) < 0.1, torch.tensor(0.25), w)
    elif kind == "equal":
        w.fill_(0.5)
    elif kind == "zero":
        w.fill_(0.0)
        w[:, ::3] = -0.0
    elif kind == "near":           # they differ in their last bits
        w = (torch.randint(0x3F800000, 0x3F800000 + 2 * cols, w.shape, generator=g).int()).view(torch.float32)
    elif kind == "rising":
        w = torch.arange(cols).float().expand(len(lens), cols).clone()
    elif kind == "falling":
        w = torch.arange(cols, 0, -1).float().expand(len(lens), cols).clone()
    elif kind == "tiny":
        w = torch.randint(0, 50, w.shape, generator=g).int().view(torch.float32)
    return w.to(DEV)


def check_evict(b, budget, trigger=None, sinks=0, recent=0, kind="mixed", elsewhere=False, seed=1, cols=None):
    trigger = budget if trigger is None else trigger
    R = len(b.lens)
    cols = max(b.lens + [1]) + 3 if cols is None else cols
    w = weights_of(b.lens, cols, seed, kind)
    old_w = w.clone()
    was = [b.contents(s) for s in b.slots]
    storage = b.cache.storage.clone()
    kw = dict(trigger=trigger, sinks=sinks, recent=recent)
    table_out = None
    if elsewhere:
        need = max(1, -(-max(min(n, trigger) for n in b.lens) // b.page))
        assert b.free.numel() >= R * need
        table_out = b.free[:R * need].view(R, need).to(DEV)
        w2, n2 = torch.full((R, cols), 9.0, device=DEV), torch.full((R,), -5, dtype=torch.int32, device=DEV)
        kept = b.cache.evict(w, b.table, b.kv_len, b.page, budget, page_table_out=table_out, weights_out=w2, kv_len_out=n2, **kw)
        assert torch.equal(w, old_w) and b.kv_len.tolist() == b.lens
    else:
        w2, n2 = w, b.kv_len
        kept = b.cache.evict(w, b.table, b.kv_len, b.page, budget, **kw)
    assert b.cache.status() == 0
    assert kept.shape == (R, budget) and kept.dtype == torch.int32
    mine = torch.zeros(b.cache.num_slots, dtype=torch.bool, device=DEV)
    for r, n in enumerate(b.lens):
        want = K.evict(old_w[r, :n].tolist(), budget, trigger, sinks, recent)
        left = len(want)
        assert int(n2[r]) == left
        assert kept[r].tolist() == (want + [-1] * budget)[:budget], r
        at = torch.tensor(want, dtype=torch.long, device=DEV)
        assert torch.equal(w2[r, :left], old_w[r, at])
        assert not w2[r, left:n].any()
        if n > 0:
            rest = w2[r, n:]
            assert torch.equal(rest, torch.full_like(rest, 9.0) if elsewhere else old_w[r, n:])
        slots = b.slot_list(table_out[r] if elsewhere else b.table[r], left)
        mine[slots] = True
        if not elsewhere:
            mine[b.slots[r]] = True
        if left:
            for x, y in zip(b.contents(slots), was[r]):
                assert torch.equal(x, y[at])
    others = (~mine).nonzero().flatten()
    now = b.contents(others)
    after = b.cache.storage.clone()
    b.cache.storage.copy_(storage)
    before = b.contents(others)
    b.cache.storage.copy_(after)
    assert all(torch.equal(x, y) for x, y in zip(now, before))


@pytest.mark.parametrize("elsewhere", [False, True])
@pytest.mark.parametrize("kind", ["mixed", "equal", "zero", "near", "rising", "falling", "tiny"])
@pytest.mark.parametrize("H,d", [(2, 64), (1, 128), (3, 256)])
def test_the_heaviest_stay(H, d, kind, elsewhere):
    lens = [300, 64, 65, 0, 1, 129, 200, 63, 1000]
    check_evict(Batch(lens, H, d, seed=20, spare=9 * 4), 64, sinks=3, recent=17, kind=kind, elsewhere=elsewhere)


@pytest.mark.parametrize("budget,trigger,sinks,recent", [(1, 1, 0, 0), (1, 1, 1, 0), (1, 1, 0, 1), (2, 2, 1, 1), (5, 40, 0, 0),
                                                         (16, 16, 16, 0), (16, 16, 0, 16), (17, 100, 4, 13), (100, 100, 0, 50),
                                                         (100, 101, 99, 0), (130, 131, 7, 3), (500, 500, 4, 32)])
@pytest.mark.parametrize("elsewhere", [False, True])
def test_budgets_triggers_and_kept_ends(budget, trigger, sinks, recent, elsewhere):
    lens = [101, 100, 131, 132, 499, 500, 501, 2, 1, 0, 17, 777]
    b = Batch(lens, 2, 64, seed=21, spare=12 * 32)
    check_evict(b, budget, trigger, sinks, recent, elsewhere=elsewhere)


@pytest.mark.parametrize("n,budget,H,d,page", [(20000, 4096, 2, 64, 16), (20000, 19000, 1, 128, 64), (70001, 30011, 1, 64, 128),
                                               (9000, 100, 2, 256, 16), (131072, 32768, 2, 64, 4096)])
@pytest.mark.parametrize("kind", ["mixed", "rising", "falling"])
def test_long_requests(n, budget, H, d, page, kind):
    """Clusters of every size, thousands of chunks that wait for one another."""
    check_evict(Batch([n, n // 3, 50], H, d, page=page, seed=22), budget, sinks=4, recent=64, kind=kind)


def test_many_requests_are_cut():
    lens = [(13 * i) % 90 for i in range(1500)]
    check_evict(Batch(lens, 1, 64, seed=23), 33, 40, 1, 5)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_evictions(seed):
    g = np.random.default_rng(700 + seed)
    d, H, R = int(g.choice([64, 128, 256])), int(g.integers(1, 9)), int(g.integers(1, 12))
    lens = [int(x) for x in np.floor(np.exp(g.uniform(0, np.log(9000), R)))]
    budget = int(np.exp(g.uniform(0, np.log(max(lens) + 1))))
    sinks = int(g.integers(0, budget + 1))
    recent = int(g.integers(0, budget - sinks + 1)) if seed % 3 else 0
    elsewhere = bool(seed % 2)
    trigger = budget + int(g.integers(0, 50))
    page = int(g.choice([16, 64]))
    b = Batch(lens, H, d, page=page, seed=seed, spare=R * -(-min(trigger, max(lens)) // page) + 3)
    check_evict(b, budget, trigger, sinks, recent, str(g.choice(["mixed", "near", "tiny", "zero"])), elsewhere, seed=seed)


def test_evicting_again_and_again():
    b = Batch([400, 350], 2, 128, seed=24)
    for i, budget in enumerate((300, 299, 170, 64, 1)):
        check_evict(b, budget, sinks=min(1, budget), seed=30 + i)
        b.lens = b.kv_len.tolist()
        b.slots = [b.slot_list(b.table[r], n) for r, n in enumerate(b.lens)]


def test_places_that_are_partly_the_same_pages():
    """The first pages stay in place, the others are new."""
    b = Batch([200], 2, 64, seed=25, spare=10)
    w = weights_of([200], 200, 26)
    old = w.clone()
    was = b.contents(b.slots[0])
    table_out = b.table.clone()
    table_out[0, 2:8] = b.free[:6].to(DEV)
    kept = b.cache.evict(w, b.table, b.kv_len, 16, 120, page_table_out=table_out)
    want = K.evict(old[0].tolist(), 120, 120, 0, 0)
    assert kept[0].tolist() == want and b.cache.status() == 0
    for x, y in zip(b.contents(b.slot_list(table_out[0], 120)), was):
        assert torch.equal(x, y[torch.tensor(want, device=DEV)])


def test_requests_that_cannot_be_cut_are_left_alone():
    b = Batch([100, 90, 80], 2, 64, seed=27, spare=30)
    w = weights_of(b.lens, 120, 28)
    storage = b.cache.storage.clone()
    ok = {}

    def run(w, table, n, status, skipped, **kw):
        b.cache.storage.copy_(storage)
        w, n = w.clone(), n.clone()
        before = w.clone()
        kept = b.cache.evict(w, table, n, 16, 50, recent=5, **kw)
        assert b.cache.status() == status
        for r in range(3):
            if r in skipped:
                assert (kept[r] == -1).all() and torch.equal(w[r].view(torch.int32), before[r].view(torch.int32))
            elif "page_table_out" not in kw and ok:
                assert kept[r].tolist() == ok["kept"][r] and torch.equal(w[r], ok["w"][r, :w.shape[1]]) and int(n[r]) == 50
        for r in () if "page_table_out" in kw else skipped:
            after = b.cache.storage.clone()
            now = b.contents(b.slots[r])
            b.cache.storage.copy_(storage)
            assert all(torch.equal(x, y) for x, y in zip(now, b.contents(b.slots[r])))
            b.cache.storage.copy_(after)
        return kept, w, n

    kept, w2, n2 = run(w, b.table, b.kv_len, 0, ())
    ok.update(kept=kept.tolist(), w=w2)
    for bad in (float("nan"), float("inf"), -1.0, -float("inf")):
        for at in (0, 50, 89):
            x = w.clone()
            x[1, at] = bad
            kept, w2, n2 = run(x, b.table, b.kv_len, 5, (1,))
            assert n2.tolist() == [50, 90, 50]
    x = w.clone()
    x[1, 90:] = float("nan")      # behind the request's entries
    kept = b.cache.evict(x, b.table, b.kv_len.clone(), 16, 50, recent=5)
    assert kept.tolist() == ok["kept"] and b.cache.status() == 0
    for bad in (-1, 113, 2 ** 31 - 1, -2 ** 31):
        n = b.kv_len.clone()
        n[1] = bad
        kept, w2, n2 = run(w, b.table, n, 1, (1,))
        assert n2.tolist() == [50, bad, 50]
    for page in (-1, b.cache.num_slots // 16, 2 ** 31 - 1, -2 ** 31):
        for at in (0, 5):
            t = b.table.clone()
            t[1, at] = page
            run(w, t, b.kv_len, 1, (1,))
    # weights that end before the entries do
    run(w[:, :95].contiguous(), b.table, b.kv_len, 1, (0,))
    # a bad page among the places, too few of them, too short a row of weights
    out = b.free[:12].view(3, 4).to(DEV)
    t = out.clone()
    t[1, 3] = -1
    len_out = torch.zeros(3, dtype=torch.int32, device=DEV)
    run(w, b.table, b.kv_len, 1, (1,), page_table_out=t, kv_len_out=len_out)
    assert len_out.tolist() == [50, 0, 50]
    run(w, b.table, b.kv_len, 1, (0, 1, 2), page_table_out=out[:, :3].contiguous(), kv_len_out=len_out)
    assert len_out.tolist() == [0, 0, 0]
    run(w, b.table, b.kv_len, 1, (0, 1, 2), weights_out=torch.zeros(3, 49, device=DEV), kv_len_out=len_out)
    assert len_out.tolist() == [100, 90, 80]


def test_a_cache_that_ends_inside_a_page():
    """48 slots and pages of 32: entries of page 1 are in the cache up to slot 48."""
    from sparse_long_context_tail_gb300.kvcache import QuantKVCache
    g = torch.Generator().manual_seed(62)
    for in_place in (True, False):
        for n, status in ((16, 0), (15, 0), (17, 1), (32, 1)):
            cache = QuantKVCache(48, 2, 64)
            k = torch.randn(32, 2, 64, generator=g).to(BF16).to(DEV)
            cache.write(k, k, torch.arange(32, device=DEV))
            table = torch.tensor([[1 if in_place else 0]], dtype=torch.int32, device=DEV)
            kw = {} if in_place else dict(page_table_out=torch.ones_like(table))
            kv_len = torch.tensor([n if in_place else 32], dtype=torch.int32, device=DEV)
            w = weights_of([32], 32, 63, "rising")
            storage = cache.storage.clone()
            cache.evict(w, table, kv_len, 32, 10 if in_place else n, **kw)
            assert cache.status() == status
            if status:
                assert torch.equal(cache.storage, storage)
            elif not in_place:
                want = cache.read(torch.arange(32 - n, 32, device=DEV))[0]
                assert torch.equal(cache.read(torch.arange(32, 32 + n, device=DEV))[0], want)


def test_captured_evictions():
    """One graph serves lengths below and above the trigger."""
    b = Batch([100, 70], 2, 64, seed=31)
    w = torch.zeros(2, 112, device=DEV)
    kept = torch.zeros(2, 48, dtype=torch.int32, device=DEV)
    storage = b.cache.storage.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.cache.evict(w, b.table, b.kv_len, 16, 48, trigger=64, sinks=2, recent=8, kept=kept)
    for i, lens in enumerate(([100, 60], [64, 65], [10, 100 - 36])):
        b.cache.storage.copy_(storage)
        b.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        w.copy_(weights_of(lens, 112, 40 + i))
        old = w.clone()
        graph.replay()
        torch.cuda.synchronize()
        for r, n in enumerate(lens):
            want = K.evict(old[r, :n].tolist(), 48, 64, 2, 8)
            assert int(b.kv_len[r]) == len(want) and kept[r].tolist() == (want + [-1] * 48)[:48]
            assert torch.equal(w[r, :len(want)], old[r, torch.tensor(want, device=DEV)])
    assert b.cache.status() == 0


def test_a_wait_that_runs_out_is_reported():
    """With a limit of one cycle a chunk that has to wait gives up; the context stays usable."""
    b = Batch([20000] * 8, 2, 64, seed=32)
    w = weights_of(b.lens, 20000, 33, "mixed")
    B.upf_set_wait_limit(b.cache.ctx, 1)
    b.cache.evict(w, b.table, b.kv_len, 16, 19000)
    assert b.cache.status() in (0, 6)
    B.upf_set_wait_limit(b.cache.ctx, 0)
    b = Batch([2000], 2, 64, seed=34)
    check_evict(b, 1500)


def test_what_the_front_end_refuses():
    b = Batch([40, 50], 2, 64, seed=35)
    room = torch.zeros(200, device=DEV)
    w = room[:128].view(2, 64)
    for kw, word in [(dict(budget=0), "budget"), (dict(trigger=9), "trigger"), (dict(sinks=-1), "sinks"),
                     (dict(sinks=5, recent=6), "sinks"), (dict(budget=2 ** 31), "32 bits"),
                     (dict(weights_out=room[1:129].view(2, 64)), "overlap"),
                     (dict(weights_out=torch.zeros(3, 64, device=DEV)), "weights_out"),
                     (dict(kept=torch.zeros(2, 11, dtype=torch.int32, device=DEV)), "kept"),
                     (dict(kv_len_out=torch.zeros(3, dtype=torch.int32, device=DEV)), "kv_len_out"),
                     (dict(page_table_out=torch.zeros(3, 4, dtype=torch.int32, device=DEV)), "page_table_out")]:
        a = dict(budget=10)
        a.update(kw)
        with pytest.raises((ValueError, B.UpfError), match=word):
            b.cache.evict(w, b.table, b.kv_len, 16, **a)
    for bad, word in [((w.double(), b.table, b.kv_len), "weights"), ((w[0], b.table, b.kv_len), "weights"),
                      ((w, b.table.long(), b.kv_len), "page_table"), ((w, b.table, b.kv_len.long()), "kv_len"),
                      ((w[:, ::2], b.table, b.kv_len), "weights")]:
        with pytest.raises(ValueError, match=word):
            b.cache.evict(*bad, 16, 10)
    with pytest.raises(B.UpfError, match="page_size"):
        b.cache.evict(w, b.table, b.kv_len, 24, 10)
    q, cu = queries([1, 1], 4, 64, BF16, 36)
    lse = torch.zeros(2, 4, device=DEV)
    for kw, word in [(dict(decay=-0.1), "decay"), (dict(decay=1.5), "decay"), (dict(decay=float("nan")), "decay"),
                     (dict(out=torch.zeros(2, 60, device=DEV)), "shape"), (dict(softmax_scale=0.0), "softmax_scale"),
                     (dict(out=room[1:129].view(2, 64)[:, :63]), "shape"), (dict(window=-1), "window")]:
        with pytest.raises((ValueError, B.UpfError), match=word):
            b.cache.accumulate(q, lse, b.table, b.kv_len, 16, w, **kw)
    with pytest.raises(ValueError, match="weights or out"):
        b.cache.accumulate(q, lse, b.table, b.kv_len, 16, None)
    with pytest.raises(ValueError, match="lse"):
        b.cache.accumulate(q, lse.half(), b.table, b.kv_len, 16, w)
    assert b.kv_len.tolist() == [40, 50]


# --------------------------------------------------------- all of it together --

def test_from_unrotated_rows_to_an_evicted_cache():
    """Rotate, select, write the kept tokens, decode with weights, evict, decode on."""
    from sparse_long_context_tail_gb300.rotary import RotaryEmbedding
    from sparse_long_context_tail_gb300.selector import TokenSelector
    torch.manual_seed(0)
    T, Hq, H, d, page = 1500, 8, 2, 64, 16
    rope = RotaryEmbedding(d, base=10000.0)
    sel = TokenSelector(0)
    rows = torch.randn(T, Hq + 2 * H, d, device=DEV).to(BF16)
    pos = torch.arange(T, device=DEV)
    table = torch.randperm(-(-T // page) + 4, device=DEV).int()[None]
    q, k = rope.apply(rows[:, :Hq], rows[:, Hq:Hq + H], pos)
    cu = np.array([0, T], np.int32)
    e = torch.arange(T, device=DEV)
    out = sel.select_tokens(q, k, cu, torch.from_numpy(cu).to(DEV), Hq, H, d, hidden=rows.reshape(T, -1), positions=pos,
                            params=B.make_params(32, 16, 32, 32, 0.6))
    n = int(out.total_kept)
    assert 64 <= n < T and sel.status() == 0
    # the kept tokens' rows, rotated at their positions, are the rows rotated before
    hidden = out.hidden_out.view(T, -1, d)
    k2 = rope.apply(None, hidden[:, Hq:Hq + H], out.pos_out, num_tokens=out.total_kept)[1]
    idx = out.kept_index[:n].long()
    assert torch.equal(k2[:n], k[idx])
    from sparse_long_context_tail_gb300.kvcache import QuantKVCache
    cache = QuantKVCache(table.numel() * page, H, d)
    slots = table[0, e // page].long() * page + e % page
    cache.write(k2, hidden[:, Hq + H:], slots, out.total_kept)
    kv_len = out.total_kept.clone()
    weights = torch.zeros(1, table.numel() * page, device=DEV)
    budget, total, keys, vals = 48, np.zeros(n), list(K.cache_values(f64(k2[:n]), 0)), list(
        K.cache_values(f64(hidden[:n, Hq + H:]), 0))
    for step in range(3):
        new = torch.randn(1, Hq + 2 * H, d, device=DEV).to(BF16)
        qn, kn = rope.apply(new[:, :Hq], new[:, Hq:Hq + H], pos[-1:] + 1 + step)
        at = kv_len.long()
        cache.write(kn, new[:, Hq + H:], table[0, at // page].long() * page + at % page)
        kv_len += 1
        keys.append(K.cache_values(f64(kn), 0)[0])
        vals.append(K.cache_values(f64(new[:, Hq + H:]), 0)[0])
        got = cache.attend(qn, table, kv_len, page)
        cache.accumulate(qn, got.lse, table, kv_len, page, weights)
        ref = K.attend(f64(qn), [np.stack(keys)], [np.stack(vals)], [0, 1])
        assert np.abs(f64(got.out) - ref[0]).max() < 0.02 * np.abs(ref[0]).max()
        drawn, slack = K.accumulate(f64(qn), f64(got.lse), [np.stack(keys)], [0, 1])
        total = np.append(total, 0) + drawn[0]
        now = f64(weights[0, :len(keys)])
        assert np.allclose(now, total, rtol=1e-4, atol=1e-9) and not weights[0, len(keys):].any()
        kept = cache.evict(weights, table, kv_len, page, budget, sinks=2, recent=8)[0].long()
        want = K.evict(now.tolist(), budget, budget, 2, 8)
        assert kept.tolist() == want and kv_len.tolist() == [budget]
        keys, vals, total = [keys[i] for i in want], [vals[i] for i in want], total[want]
        held = cache.read(table[0, e[:budget] // page].long() * page + e[:budget] % page)
        np.testing.assert_array_equal(f64(held[0]), np.stack(keys))
        np.testing.assert_array_equal(f64(held[1]), np.stack(vals))
    assert cache.status() == 0
