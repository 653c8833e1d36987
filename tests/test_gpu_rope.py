"""Rotary positions on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import rope_oracle as O
from sparse_long_context_tail_gb300 import _binding as B

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def rotation(*args, **kw):
    from sparse_long_context_tail_gb300.rotary import RotaryEmbedding
    return RotaryEmbedding(*args, **kw)


def rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-3, 4, shape[:-1] + (1,), generator=g).float())
    return x.to(dtype).to(DEV)


def check(got, x, rope, positions, interleaved=False, inverse=False):
    """`got` is `x` turned: dims past the rotary ones bit for bit, the others within the arithmetic.

    An output is m (a c - b s) with c and s off by 2^-22 at most (2 ulp of sincospif, and an angle rounded by pi 2^-25 and
    2 pi 2^-33), two fp32 roundings of the sum and one of each factor (m c, m s): under 2^-21 m (|a| + |b|) in all; then
    half a step of the output type (for values under its normal range, half its least step)."""
    n = rope.rotary_dim
    angle = O.angles(positions.tolist(), rope.turns.cpu().numpy().view(np.uint64))
    xs = x.cpu().double().numpy()
    want = O.rotate(xs, angle, n, interleaved, rope.magnitude, inverse)
    assert torch.equal(got[..., n:].contiguous().view(torch.int16), x[..., n:].contiguous().view(torch.int16))
    first, second = (np.arange(0, n, 2), np.arange(1, n, 2)) if interleaved else (np.arange(n // 2), np.arange(n // 2, n))
    size = np.zeros_like(xs)
    size[..., first] = size[..., second] = np.abs(xs[..., first]) + np.abs(xs[..., second])
    m = 1 / rope.magnitude if inverse else rope.magnitude
    info = torch.finfo(x.dtype)
    bound = 2.0 ** -21 * m * size
    bound = bound + info.eps / 2 * (np.abs(want) + bound) + info.smallest_normal * info.eps / 2
    off = np.abs(got.cpu().double().numpy() - want)[..., :n]
    assert (off <= bound[..., :n]).all(), (off / bound[..., :n]).max()


def places(T, seed=0, far=1 << 20):
    return torch.randint(0, far, (T,), generator=torch.Generator().manual_seed(seed)).to(DEV)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,n", [(64, 64), (64, 2), (128, 128), (128, 64), (128, 16), (128, 48), (128, 10), (128, 126),
                                 (256, 256), (256, 64), (256, 250)])
@pytest.mark.parametrize("T,hq,hk", [(1, 8, 2), (5, 5, 1), (67, 3, 3)])
def test_queries_and_keys_are_turned(T, hq, hk, d, n, interleaved, dtype):
    rope = rotation(d, n, 10000.0, interleaved=interleaved)
    q, k, pos = rand((T, hq, d), dtype, 1), rand((T, hk, d), dtype, 2), places(T)
    q2, k2 = rope.apply(q, k, pos)
    check(q2, q, rope, pos, interleaved)
    check(k2, k, rope, pos, interleaved)
    # one of them alone, and in place
    assert torch.equal(rope.apply(q, None, pos)[0], q2) and torch.equal(rope.apply(None, k, pos)[1], k2)
    a, b = q.clone(), k.clone()
    got = rope.apply(a, b, pos, out=(a, b))
    assert got[0] is a and torch.equal(a, q2) and torch.equal(b, k2)
    # q in place, k elsewhere
    a, b = q.clone(), torch.zeros_like(k)
    rope.apply(a, k, pos, out=(a, b))
    assert torch.equal(a, q2) and torch.equal(b, k2)


@pytest.mark.parametrize("kind", [dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                                  dict(scaling="yarn", factor=16.0, original_len=4096),
                                  dict(scaling="bands", factor=8.0, original_len=8192), dict(magnitude=0.7),
                                  dict(divisors=np.linspace(1, 30, 64))])
def test_frequencies_for_long_contexts(kind):
    rope = rotation(128, base=500000.0, **kind)
    x, pos = rand((40, 4, 128), BF16, 3), places(40, 4)
    check(rope.apply(x, None, pos)[0], x, rope, pos)
    y = rope.apply(x, None, pos, inverse=True)[0]
    check(y, x, rope, pos, inverse=True)


def test_any_position():
    """Angles are exact modulo a turn, at positions of every size and sign."""
    pos = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 7, 2 ** 63 - 1, -2 ** 63], device=DEV)
    for interleaved in (False, True):
        rope = rotation(64, interleaved=interleaved)
        x = rand((len(pos), 2, 64), F16, 5)
        got = rope.apply(x, None, pos)[0]
        check(got, x, rope, pos, interleaved)
        assert torch.equal(got[0], x[0])
    # positions p and -p turn to and fro
    there = rope.apply(x, None, pos[3:4].expand(len(pos)).contiguous())[0]
    back = rope.apply(there, None, -pos[3:4].expand(len(pos)).contiguous())[0]
    again = rope.apply(there, None, pos[3:4].expand(len(pos)).contiguous(), inverse=True)[0]
    assert torch.equal(back, again)


@pytest.mark.parametrize("n", [128, 20])
def test_rows_with_strides_and_a_device_count(n):
    T, hq, hk, d = 37, 6, 2, 128
    rope = rotation(d, n, scaling="yarn", factor=4.0, original_len=64)
    rows = rand((T, hq + 2 * hk, d), BF16, 6)
    pos = places(T, 7)
    q, k = rows[:, :hq], rows[:, hq:hq + hk]
    want = rope.apply(q.contiguous(), k.contiguous(), pos)
    got = rope.apply(q, k, pos)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for count, done in ((0, 0), (1, 1), (20, 20), (37, 37), (1000, 37), (-5, 0)):
        before = rand((T, hq + hk + 1, d), BF16, 8)
        out = before.clone()
        c = torch.tensor([count], dtype=torch.int32, device=DEV)
        rope.apply(q, k, pos, num_tokens=c, out=(out[:, :hq], out[:, hq:hq + hk]))
        assert torch.equal(out[:done, :hq], want[0][:done]) and torch.equal(out[:done, hq:hq + hk], want[1][:done])
        assert torch.equal(out[done:], before[done:]) and torch.equal(out[:, hq + hk:], before[:, hq + hk:])
    # in place inside the projection's rows: the values stay
    mine = rows.clone()
    rope.apply(mine[:, :hq], mine[:, hq:hq + hk], pos, out=(mine[:, :hq], mine[:, hq:hq + hk]))
    assert torch.equal(mine[:, :hq], want[0]) and torch.equal(mine[:, hq:hq + hk], want[1])
    assert torch.equal(mine[:, hq + hk:], rows[:, hq + hk:])


def test_nan_and_infinity_stay_in_their_pair():
    rope = rotation(64)
    x, pos = rand((4, 2, 64), BF16, 9), places(4, 10)
    y = x.clone()
    y[1, 0, 3], y[2, 1, 40] = float("nan"), float("inf")
    a, b = rope.apply(x, None, pos)[0], rope.apply(y, None, pos)[0]
    hit = torch.zeros(4, 2, 64, dtype=torch.bool, device=DEV)
    hit[1, 0, [3, 35]] = hit[2, 1, [8, 40]] = True
    assert torch.equal(a[~hit], b[~hit]) and not torch.isfinite(b[hit]).any()


def test_many_tokens_and_heads():
    """All heads by one thread, a part of them, and rows past 2^32 bytes."""
    rope = rotation(128, base=500000.0)
    g = torch.Generator(device=DEV).manual_seed(11)
    for T, hq, hk in ((60001, 5, 2), (30000, 32, 8), (3, 700, 300)):
        q = torch.randn(T, hq, 128, device=DEV, generator=g).to(BF16)
        k = torch.randn(T, hk, 128, device=DEV, generator=g).to(BF16)
        pos = torch.randint(0, 1 << 17, (T,), device=DEV, generator=g)
        q2, k2 = rope.apply(q, k, pos)
        at = torch.tensor([0, 1, T // 2, T - 2, T - 1], device=DEV).clamp(min=0)
        check(q2[at], q[at], rope, pos[at])
        check(k2[at], k[at], rope, pos[at])
    wide = torch.empty(9, 1 << 29, dtype=BF16, device=DEV)       # 1 GiB a row
    x = wide.as_strided((9, 2, 128), (1 << 29, 128, 1))
    x.copy_(rand((9, 2, 128), BF16, 12))
    pos = places(9, 13)
    want = rope.apply(x.contiguous(), None, pos)[0]
    rope.apply(x, None, pos, out=(x, None))
    assert torch.equal(x, want)


def test_no_tokens_and_no_heads():
    rope = rotation(64)
    q, k = rope.apply(torch.empty(0, 4, 64, dtype=BF16, device=DEV), torch.empty(0, 1, 64, dtype=BF16, device=DEV),
                      torch.empty(0, dtype=torch.int64, device=DEV))
    assert q.shape == (0, 4, 64) and k.shape == (0, 1, 64)
    x, pos = rand((3, 2, 64), BF16, 14), places(3)
    q, k = rope.apply(torch.empty(3, 0, 64, dtype=BF16, device=DEV), x, pos)
    assert q.shape == (3, 0, 64) and torch.equal(k, rope.apply(x, None, pos)[0])


def test_captured_and_on_another_stream():
    rope = rotation(128)
    q, k, pos = rand((50, 4, 128), BF16, 15), rand((50, 2, 128), BF16, 16), places(50, 17)
    count = torch.tensor([50], dtype=torch.int32, device=DEV)
    out = (torch.zeros_like(q), torch.zeros_like(k))
    want = [x.clone() for x in rope.apply(q, k, pos)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = rope.apply(q, k, pos)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.apply(q, k, pos, num_tokens=count, out=out)
    for n in (50, 13):                       # another count and other positions at the replay
        pos.copy_(places(50, n))
        count.fill_(n)
        for x in out:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(out[0][:n], q[:n], rope, pos[:n])
        check(out[1][:n], k[:n], rope, pos[:n])
        assert not out[0][n:].any() and not out[1][n:].any()


def test_what_the_front_end_refuses():
    rope = rotation(128)
    q, k, pos = rand((4, 2, 128), BF16, 18), rand((4, 1, 128), BF16, 19), places(4)
    for bad, word in [((None, None, pos), "q or k"), ((q.float(), k, pos), "bfloat16"), ((q, k.half(), pos), "k must be"),
                      ((q, k, pos.int()), "positions"), ((q, k, pos[:3]), "tokens"), ((q, k, pos[:, None]), "positions"),
                      ((q[0], k, pos), "shape"), ((q[..., :64], k, pos), "shape"), ((q.cpu(), k, pos), "cpu"),
                      ((q, k, pos.repeat(2)[::2]), "positions"), ((rand((4, 4, 128), BF16, 1)[:, ::2], k, pos), "contiguous")]:
        with pytest.raises(ValueError, match=word):
            rope.apply(*bad)
    for kw, word in [(dict(num_tokens=torch.tensor([4], device=DEV)), "num_tokens"), (dict(out=(q[:3], None)), "shape"),
                     (dict(out=(None, k.half())), "type"), (dict(num_tokens=torch.tensor([4], dtype=torch.int32)), "num_tokens")]:
        with pytest.raises(ValueError, match=word):
            rope.apply(q, k, pos, **kw)
    with pytest.raises(ValueError, match="k, which is None"):
        rope.apply(q, None, pos, out=(None, k))
    big = rand((6, 2, 128), BF16, 20)
    with pytest.raises(B.UpfError, match="overlaps"):
        rope.apply(big[:4], None, pos, out=(big[2:], None))
    for bad in (dict(magnitude=0.0), dict(magnitude=-1.0), dict(scaling="ntk")):
        with pytest.raises(ValueError):
            rotation(128, **bad)
    for bad in (dict(head_dim=96), dict(head_dim=128, rotary_dim=3), dict(head_dim=128, scaling="yarn", factor=2.0)):
        with pytest.raises(B.UpfError):
            rotation(**bad)


@pytest.mark.parametrize("seed", range(10))
def test_drawn_rotations(seed):
    g = np.random.default_rng(800 + seed)
    d = int(g.choice([64, 128, 256]))
    n = 2 * int(g.integers(1, d // 2 + 1)) if seed % 2 else 16 * int(g.integers(1, d // 16 + 1))
    T, heads = int(np.exp(g.uniform(0, np.log(3000)))), [int(x) for x in g.integers(0, 12, 2)]
    heads[0] += sum(heads) == 0
    interleaved, inverse = bool(g.integers(2)), bool(g.integers(2))
    rope = rotation(d, n, base=float(10 ** g.uniform(1, 7)), interleaved=interleaved,
                    magnitude=float(g.uniform(0.5, 2)))
    pos = places(T, seed, 2 ** 40)
    q, k = (rand((T, h, d), BF16 if seed % 3 else F16, seed) if h else None for h in heads)
    for x, y in zip((q, k), rope.apply(q, k, pos, inverse=inverse)):
        if x is not None:
            check(y, x, rope, pos, interleaved, inverse)


def test_rows_past_32_bits_of_bytes():
    """Rows 4 GiB apart."""
    rope = rotation(64)
    room = torch.empty(2 ** 32 + 256, dtype=BF16, device=DEV)
    x = room.as_strided((3, 2, 64), (2 ** 31, 64, 1))
    x.copy_(rand((3, 2, 64), BF16, 1))
    pos = torch.tensor([5, 2 ** 40, -3], device=DEV)
    want = rope.apply(x.contiguous(), None, pos)[0]
    assert rope.apply(x, None, pos, out=(x, None))[0] is x
    assert torch.equal(x, want)


def test_selection_of_rows_that_are_not_turned_yet():
    from sparse_long_context_tail_gb300.selector import TokenSelector
    T, Hq, H, d = 700, 8, 2, 128
    rope, sel = rotation(d, 64), TokenSelector(0)
    rows = rand((T, Hq + 2 * H, d), BF16, 3)
    q, k = rows[:, :Hq], rows[:, Hq:Hq + H]
    pos = places(T, 4)
    cu = np.array([0, 300, T], np.int32)
    cu_dev = torch.from_numpy(cu).to(DEV)
    kw = dict(hidden=rows.reshape(T, -1), positions=pos, params=B.make_params(32, 16, 32, 32, 0.6))
    q2, k2 = rope.apply(q, k, pos)
    want = sel.select_tokens(q2, k2, cu, cu_dev, Hq, H, d, **kw)
    got = sel.select_tokens(q, k, cu, cu_dev, Hq, H, d, rope=rope, **kw)
    assert want.q_out is None and torch.equal(got.q_out, q2) and torch.equal(got.k_out, k2)
    n = int(want.total_kept)
    assert 0 < n < T and torch.equal(got.scores, want.scores) and int(got.total_kept) == n
    assert torch.equal(got.kept_index[:n], want.kept_index[:n]) and torch.equal(got.pos_out[:n], want.pos_out[:n])
    assert torch.equal(got.hidden_out[:n], want.hidden_out[:n])
    # in place
    got.q_out, got.k_out = q, k
    again = sel.select_tokens(q, k, cu, cu_dev, Hq, H, d, rope=rope, out=got, **kw)
    assert again is got and again.q_out is q and torch.equal(q, q2) and torch.equal(k, k2) and int(got.total_kept) == n
    with pytest.raises(ValueError, match="positions"):
        sel.select_tokens(q, k, cu, cu_dev, Hq, H, d, rope=rope, params=kw["params"])
    assert sel.status() == 0
