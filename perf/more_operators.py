"""Cases of three operators around the 4-bit KV cache: rotary positions of queries and keys,
accumulating the attention weight of cache entries, and evicting entries by it.

The packed cache has records of 18*d bytes for 16 slots of one kv head; with
P = max(1, d/128) parts of D = d/P dims and C = D/16:

* K codes  [P][16 rows][D/2]                  low nibble = even dim
* V codes  [P][2 halves][8 chunks][4][2][C]   row = 8*half + 2*pair + bit
* K scales [16 rows][d/16]
* V scales [P][2 halves][D/16][4][2]          row as for the V codes

``run`` computes an operator in plain torch operations, or, where ``own`` is true, through
``RotaryEmbedding`` and ``QuantKVCache``.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases --

def _rope(name, tokens, q_heads, heads, dim, rotary=0, interleaved=False, dtype="bf16", scaling="none", factor=1.0,
          base=500000.0, far=131072, fused=False, counted=0):
    """``counted``: tokens that the device-side count leaves (0: all, no count)."""
    return dict(name=name, op="rope", tokens=tokens, q_heads=q_heads, heads=heads, dim=dim, rotary=rotary or dim,
                interleaved=interleaved, dtype=dtype, scaling=scaling, factor=factor, base=base, far=far, fused=fused,
                counted=counted)


def _weigh(name, reqs, lo, hi, q_heads, heads, dim, dtype="bf16", page=16, window=0, sinks=0, q_len=1, ragged_q=False,
           decay=1.0, k_exp=0, lens_seed=1):
    return dict(name=name, op="weigh", reqs=reqs, lo=lo, hi=hi, q_heads=q_heads, heads=heads, dim=dim, dtype=dtype,
                page=page, window=window, sinks=sinks, q_len=q_len, ragged_q=ragged_q, decay=decay, k_exp=k_exp,
                lens_seed=lens_seed)


def _evict(name, reqs, lo, hi, heads, dim, budget, trigger=0, sinks=4, recent=64, dtype="bf16", page=16, lens_seed=1):
    return dict(name=name, op="evict", reqs=reqs, lo=lo, hi=hi, heads=heads, dim=dim, budget=budget,
                trigger=trigger or budget, sinks=sinks, recent=recent, dtype=dtype, page=page, lens_seed=lens_seed)


def listed():
    return [
        # one new token of each of 8 decoding requests at a 32/8-head layer (the smallest call: latency)
        _rope("rope-8-tokens", 8, 32, 8, 128),
        # a 128K prompt at the same layer, q and k views of one projection's rows, frequencies scaled in bands
        _rope("rope-131072-tokens", 131072, 32, 8, 128, scaling="bands", factor=8.0, fused=True),
        # the kept tokens of a 32K chunk after a selection (count on the device), a quarter of a d = 256 head rotated
        _rope("rope-20011-kept-d256", 32768, 16, 2, 256, rotary=64, scaling="yarn", factor=4.0, base=1e7, far=262144,
              counted=20011),
        # interleaved pairs on a small fp16 layer, an odd number of tokens, positions interpolated
        _rope("rope-4097-interleaved-d64", 4097, 8, 2, 64, interleaved=True, dtype="fp16", scaling="linear", factor=2.0,
              base=10000.0, far=8192),
        # one decoding request of 4K entries on a small layer (latency)
        _weigh("weigh-1x4096-d64", 1, 4096, 4096, 8, 2, 64),
        # a decoding step of a continuous batch of 16, lengths log-uniform in [4096, 131072]
        _weigh("weigh-16-ragged", 16, 4096, 131072, 32, 8, 128, lens_seed=4),
        # the last 32 queries of a 128K prompt weigh its entries before the first eviction
        _weigh("weigh-1x131072-32-queries", 1, 131072, 131072, 32, 8, 128, q_len=32),
        # a step of 24 requests of an fp16 layer with d = 256, old weight fading
        _weigh("weigh-24-decay-d256", 24, 2048, 16384, 16, 8, 256, dtype="fp16", page=64, decay=0.98, k_exp=1,
               lens_seed=2),
        # eight requests 64 entries over their budget on a small layer (latency)
        _evict("evict-8x1088-d64", 8, 1088, 1088, 2, 64, 1024),
        # a 128K prompt cut to a quarter
        _evict("evict-1x131072", 1, 131072, 131072, 8, 128, 32768, recent=1024),
        # a ragged batch cut to 4096 entries each, shorter ones only moved
        _evict("evict-16-ragged", 16, 1500, 131072, 8, 128, 4096, trigger=4352, recent=256, lens_seed=4),
        # many requests, an odd budget, two heads of d = 256, fp16, larger pages
        _evict("evict-64-odd-d256", 64, 1000, 9000, 2, 256, 2011, sinks=3, recent=129, dtype="fp16", page=64,
               lens_seed=3),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "weigh", "evict"])
    dtype = rng.choice(["bf16", "fp16"])
    page = rng.choice([16, 32, 64, 128])
    seed = rng.randrange(1 << 20)
    if op == "rope":
        q_heads, heads, dim = rng.choice([(8, 2, 64), (5, 1, 64), (32, 8, 128), (28, 4, 128), (12, 1, 128), (16, 2, 256),
                                          (16, 8, 256)])
        tokens = _log_int(rng, 1, min(131072, 131072 * 40 * 128 // ((q_heads + heads) * dim)))
        scaling = rng.choice(["none", "linear", "base", "yarn", "bands"])
        c = _rope("", tokens, q_heads, heads, dim, rng.choice([dim, dim, dim // 2, dim // 4, 48, 10]), rng.random() < 0.4,
                  dtype, scaling, 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                  rng.choice([10000.0, 500000.0, 1e6, 1e7]), _log_int(rng, 4096, 1 << 20), rng.random() < 0.5,
                  rng.randint(0, tokens) if rng.random() < 0.3 else 0)
    elif op == "weigh":
        q_heads, heads, dim = rng.choice([(8, 2, 64), (5, 1, 64), (32, 8, 128), (28, 4, 128), (8, 8, 128), (16, 2, 256),
                                          (16, 8, 256), (12, 1, 128)])
        reqs = _log_int(rng, 1, 128)
        q_len = rng.choice([1, 1, 1, 2, 5, 16, 32])
        hi = _log_int(rng, 16, min(131072, (1 << 28) // (reqs * heads * dim), (1 << 27) // (reqs * q_heads * q_len)))
        window = rng.choice([0, 0, 0, 1, 100, 1024])
        c = _weigh("", reqs, max(1, hi // 32), hi, q_heads, heads, dim, dtype, page, window,
                   rng.choice([0, 1, 4, 37]) if window else 0, q_len, q_len > 1 and rng.random() < 0.5,
                   rng.choice([1.0, 1.0, 0.9, 0.999]), rng.randint(-4, 4), seed)
    else:
        heads, dim = rng.choice([(1, 64), (2, 64), (8, 64), (3, 128), (8, 128), (2, 256), (8, 256)])
        reqs = _log_int(rng, 1, 128)
        hi = _log_int(rng, 16, min(131072, (1 << 28) // (reqs * heads * dim)))
        budget = _log_int(rng, 1, hi)
        recent = rng.randint(0, budget)
        c = _evict("", reqs, max(1, hi // 32), hi, heads, dim, budget, budget + rng.choice([0, 0, 1, 16, 257]),
                   min(rng.choice([0, 1, 4, 33]), budget - recent), recent, dtype, page, seed)
    del c["name"]
    return c


def _lengths(case):
    """(entries of each request, new tokens of each request), from the case alone."""
    r = random.Random(case["lens_seed"])
    n = [_log_int(r, case["lo"], case["hi"]) for _ in range(case["reqs"])]
    most = case.get("q_len", 1)
    q = [r.randint(1, most) if case.get("ragged_q") else most for _ in n]
    return n, q


def work(case):
    if case["op"] == "rope":
        tokens = case["counted"] or case["tokens"]
        heads = case["q_heads"] + case["heads"]
        return dict(bytes=tokens * (heads * case["dim"] * 4 + 8), flops=3.0 * tokens * heads * case["rotary"])
    width = case["heads"] * case["dim"]
    lens, news = _lengths(case)
    if case["op"] == "evict":
        kept = sum(n if n <= case["trigger"] else case["budget"] for n in lens)
        # the weights, the kept entries' packed bytes in and out, the list, and the entries read back as values
        return dict(bytes=4 * sum(lens) + kept * (2 * width * 9 / 16 * 2 + 8 + 2 * width * 2), flops=0)
    w, s = case["window"], case["sinks"]
    entries = pairs = 0
    for n, q in zip(lens, news):
        seen = lambda p: 0 if p < 0 else (p + 1 if w == 0 else min(p + 1, min(s, max(0, p + 1 - w)) + w))  # noqa: E731
        pairs += sum(seen(n - q + i) for i in range(q))
        first = max(0, n - q)
        entries += n if w == 0 else min(n, min(s, max(0, first + 1 - w)) + n - max(0, first + 1 - w))
    rows = sum(news) * case["q_heads"]
    return dict(bytes=entries * width * 9 / 16 + 8 * sum(lens) + rows * (2 * case["dim"] + 4),
                flops=2.0 * pairs * case["q_heads"] * case["dim"])


# ------------------------------------------------------------------ inputs --

def _frequencies(case):
    """Radians per position of each pair, in 64 bits, and what the cosines are multiplied by."""
    n, base, factor, first_len = case["rotary"], case["base"], case["factor"], 8192
    i = torch.arange(0, n, 2, dtype=torch.float64)
    if case["scaling"] == "base" and n > 2:
        base = base * factor ** (n / (n - 2))
    f = base ** (-i / n)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "bands":                    # long wavelengths slowed down, short ones kept
        turns = first_len * f / (2 * math.pi)         # in the first length
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    if case["scaling"] == "yarn":
        at = lambda turns: n * math.log(first_len / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), n - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _values(gen, tokens, heads, dim, spread):
    """N(0, 1) times a magnitude per channel, as keys have them."""
    x = torch.randn(tokens, heads, dim, device=DEVICE, generator=gen)
    return x * torch.exp(spread * torch.randn(heads, dim, device=DEVICE, generator=gen))


def _storage(gen, slots, case):
    """A cache that already holds entries: packed bytes of `slots` slots."""
    heads, dim = case["heads"], case["dim"]
    cache = torch.zeros(slots // 16, heads, 18 * dim, dtype=torch.uint8, device=DEVICE)
    step = max(16, (1 << 27) // (heads * dim) // 16 * 16)
    for a in range(0, slots, step):            # in parts, to bound the temporaries
        n = min(step, slots - a)
        at = torch.arange(a, a + n, device=DEVICE)
        _put(cache, dim, at, _quantise(_values(gen, n, heads, dim, 0.4)), _quantise(_values(gen, n, heads, dim, 0.2)))
    return cache


def _prepare_rope(case, gen):
    T, hq, hk, d, dtype = case["tokens"], case["q_heads"], case["heads"], case["dim"], TYPES[case["dtype"]]
    rows = torch.cat([_values(gen, T, hq, d, 0.2), _values(gen, T, hk, d, 0.4)], 1).to(dtype)
    if case["fused"]:                          # views of one projection's rows: [q | k | v]
        rows = torch.cat([rows, _values(gen, T, hk, d, 0.2).to(dtype)], 1)
        q, k = rows[:, :hq], rows[:, hq:hq + hk]
    else:
        q, k = rows[:, :hq].contiguous(), rows[:, hq:].contiguous()
    if T <= 256:                               # decoding: requests at places of their own
        pos = torch.randint(0, case["far"], (T,), device=DEVICE, generator=gen)
    else:                                      # a chunk, or what a selection kept of it: ascending
        gap = torch.randint(1, max(2, 2 * case["far"] // T), (T,), device=DEVICE, generator=gen)
        pos = torch.cumsum(gap, 0) - gap[0]
    freqs, scale = _frequencies(case)
    state = dict(op="rope", q=q, k=k, pos=pos, freqs=freqs.to(DEVICE), scale=scale, rotary=case["rotary"],
                 interleaved=case["interleaved"], case=dict(case), count=None, out=None)
    if case["counted"]:
        state["count"] = torch.tensor([case["counted"]], dtype=torch.int32, device=DEVICE)
        state["out"] = (torch.zeros(T, hq, d, dtype=dtype, device=DEVICE),
                        torch.zeros(T, hk, d, dtype=dtype, device=DEVICE))
    return state


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    if case["op"] == "rope":
        return _prepare_rope(case, gen)
    dtype, heads, dim, page = TYPES[case["dtype"]], case["heads"], case["dim"], case["page"]
    lens, news = _lengths(case)
    evict = case["op"] == "evict"
    need = [-(-n // page) for n in lens]
    left = [n if n <= case["trigger"] else case["budget"] for n in lens] if evict else []
    more = [-(-n // page) for n in left]
    order = torch.randperm(sum(need) + sum(more) + 3, device=DEVICE, generator=gen).int()
    pad = lambda rows: torch.nn.utils.rnn.pad_sequence(rows, batch_first=True, padding_value=-1)  # noqa: E731
    table = pad(torch.split(order[:sum(need)], need))
    s = dict(op=case["op"], dim=dim, heads=heads, dtype=dtype, page=page, table=table, k_exp=case.get("k_exp", 0),
             cache=_storage(gen, order.numel() * page, case), max_kv=max(lens),
             kv_len=torch.tensor(lens, dtype=torch.int32, device=DEVICE))
    held = torch.arange(max(lens), device=DEVICE) < s["kv_len"][:, None]
    # weights of earlier steps: a few heavy entries, many light ones
    s["weights"] = torch.where(held, torch.exp(2 * torch.randn(held.shape, device=DEVICE, generator=gen) - 4), 0.0)
    if evict:
        # equal weights, as entries that few steps have seen have them
        s["weights"] = torch.where(s["weights"] < 0.004, 0.0, s["weights"])
        s["table_out"] = pad(torch.split(order[sum(need):sum(need) + sum(more)], more))
        cap = s["table_out"].shape[1] * page
        j = torch.arange(cap, device=DEVICE)
        slots = s["table_out"].long()[:, j // page] * page + j % page
        s["slots"] = slots[j < torch.tensor(left, device=DEVICE)[:, None]]
        s.update(budget=case["budget"], trigger=case["trigger"], sinks=case["sinks"], recent=case["recent"],
                 weights_out=torch.zeros(len(lens), max(lens), device=DEVICE),
                 len_out=torch.zeros(len(lens), dtype=torch.int32, device=DEVICE), max_out=max(left))
        return s
    q = torch.randn(sum(news), case["q_heads"], dim, device=DEVICE, generator=gen)
    s.update(q=(q * 1.3 * 2.0 ** -case["k_exp"]).to(dtype), max_q=case["q_len"], single=case["q_len"] == 1,
             window=case["window"], sinks=case["sinks"], decay=case["decay"],
             cu_q=torch.tensor([sum(news[:i]) for i in range(len(news) + 1)], dtype=torch.int32, device=DEVICE),
             out=torch.zeros_like(s["weights"]))
    lse = torch.logsumexp(_logits(s)[0], -1)                         # [R, Hq, Q], what the attention gave
    at, real = _rows(s)
    s["lse"] = lse.transpose(1, 2)[real].contiguous()
    return s


# ------------------------------------------------------------- plain forms --

def _quantise(x):
    """Codes [T, H, d/2] and scale bytes [T, H, d/16] of values [T, H, d]."""
    T, H, d = x.shape
    g = x.float().view(T, H, d // 16, 16)
    s = (g.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    t = g.abs() / s.float()[..., None]
    code = ((t > 0.25).byte() + (t >= 0.75).byte() + (t > 1.25).byte() + (t >= 1.75).byte() + (t > 2.5).byte()
            + (t >= 3.5).byte() + (t > 5).byte() + 8 * (g < 0).byte())
    code = torch.where((s.float() > 0)[..., None], code, 0).view(T, H, d)
    return code[..., 0::2] | code[..., 1::2] << 4, s.view(torch.uint8)


def _parts(cache, dim):
    """Views of the packed bytes: K codes, V codes, K scales, V scales (layout above)."""
    n, H, _ = cache.shape
    P = max(1, dim // 128)
    D = dim // P
    return (cache[..., :8 * dim].view(n, H, P, 16, D // 2),
            cache[..., 8 * dim:16 * dim].view(n, H, P, 2, 8, 4, 2, D // 16),
            cache[..., 16 * dim:17 * dim].view(n, H, 16, dim // 16),
            cache[..., 17 * dim:].view(n, H, P, 2, D // 16, 4, 2))


def _put(cache, dim, slots, k, v):
    kc, vc, ks, vs = _parts(cache, dim)
    T, H = k[0].shape[:2]
    P = kc.shape[2]
    b, r = slots // 16, slots % 16
    half, pair, bit = r // 8, r % 8 // 2, r % 2
    kc[b, :, :, r] = k[0].view(T, H, P, -1)
    ks[b, :, r] = k[1].view(T, H, -1)
    vc[b, :, :, half, :, pair, bit] = v[0].view(T, H, P, 8, -1)
    vs[b, :, :, half, :, pair, bit] = v[1].view(T, H, P, -1)


def _packed(cache, dim, slots, of_values):
    """Codes [T, H, d/2] and scale bytes [T, H, d/16] of K (or V) at `slots`."""
    kc, vc, ks, vs = _parts(cache, dim)
    T, H = slots.numel(), cache.shape[1]
    b, r = slots // 16, slots % 16
    half, pair, bit = r // 8, r % 8 // 2, r % 2
    code = (vc[b, :, :, half, :, pair, bit] if of_values else kc[b, :, :, r]).reshape(T, H, dim // 2)
    return code, (vs[b, :, :, half, :, pair, bit] if of_values else ks[b, :, r]).reshape(T, H, dim // 16)


def _get(cache, dim, slots, of_values):
    """K (or V) at `slots`, as the values that the bytes stand for: float32 [T, H, d]."""
    code, scale = _packed(cache, dim, slots, of_values)
    T, H = code.shape[:2]
    code = torch.stack([code & 15, code >> 4], -1).view(T, H, dim)
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=cache.device)
    x = table[code.int()].view(T, H, dim // 16, 16)
    return x.mul_(scale.view(torch.float8_e4m3fn).float()[..., None]).view(T, H, dim)


def _plain_rope(s):
    half = s["rotary"] // 2
    angle = s["pos"].double()[:, None] * s["freqs"]                  # far positions: 64 bits
    cos, sin = (x.mul_(s["scale"]).float()[:, None] for x in (torch.cos(angle), torch.sin(angle)))
    outs = []
    for i, x in enumerate((s["q"], s["k"])):
        r = x[..., :s["rotary"]].float()
        a, b = (r[..., 0::2], r[..., 1::2]) if s["interleaved"] else (r[..., :half], r[..., half:])
        y = (a * cos - b * sin, b * cos + a * sin)
        y = torch.stack(y, -1).flatten(-2) if s["interleaved"] else torch.cat(y, -1)
        y = torch.cat([y.to(x.dtype), x[..., s["rotary"]:]], -1)
        if s["count"] is None:
            outs.append(y)
        else:
            done = torch.arange(x.shape[0], device=x.device) < s["count"]
            s["out"][i].copy_(torch.where(done[:, None, None], y, s["out"][i]))
            outs.append(s["out"][i])
    return tuple(outs)


def _rows(s):
    """Row of q of each (request, query), and which of them there are: [R, Q]."""
    first = s["cu_q"][:-1].long()
    real = torch.arange(s["max_q"], device=first.device) < (s["cu_q"][1:].long() - first)[:, None]
    return torch.where(real, first[:, None] + torch.arange(s["max_q"], device=first.device), 0), real


def _slots(table, page, n, L):
    """Slots [R, L] of the entries, 0 past a request's n [R]."""
    e = torch.arange(L, device=table.device).expand(table.shape[0], L)
    held = e < n[:, None]
    return torch.where(held, table.long().gather(1, torch.where(held, e // page, 0)) * page + e % page, 0)


def _logits(s):
    """Logits [R, Hq, Q, L] of every new token over every entry, -inf where it is not seen."""
    d, H, L, Q = s["dim"], s["heads"], s["max_kv"], s["max_q"]
    R, dev = s["kv_len"].numel(), s["q"].device
    n = s["kv_len"].long()
    at, real = _rows(s)
    q = s["q"].float()[at]                                           # [R, Q, Hq, d]
    G = q.shape[2] // H
    q = q.view(R, Q, H, G, d).permute(0, 2, 3, 1, 4).reshape(R, H, G * Q, d)
    k = _get(s["cache"], d, _slots(s["table"], s["page"], n, L).view(-1), False).view(R, L, H, d).permute(0, 2, 3, 1)
    x = torch.matmul(q, k).mul_(2.0 ** s["k_exp"] / math.sqrt(d)).view(R, H * G, Q, L)
    p = (n - real.sum(1))[:, None, None] + torch.arange(Q, device=dev)[:, None]   # [R, Q, 1] position
    e = torch.arange(L, device=dev)
    seen = (e <= p) & real[..., None] & (e < n[:, None, None])
    if s["window"]:
        seen &= (p - e < s["window"]) | (e < s["sinks"])
    return x.masked_fill_(~seen[:, None], -math.inf), real


def _plain_weigh(s):
    x, real = _logits(s)
    at, _ = _rows(s)
    lse = s["lse"][at].transpose(1, 2)[..., None]                    # [R, Hq, Q, 1]
    w = torch.exp_(x.sub_(torch.where(torch.isinf(lse), 0.0, lse))).sum((1, 2))
    held = torch.arange(s["max_kv"], device=w.device) < s["kv_len"][:, None]
    s["out"].copy_(torch.where(held, s["decay"] * s["weights"] + w, s["out"]))
    return s["out"]


def _plain_evict(s):
    n, B = s["kv_len"].long()[:, None], s["budget"]
    e = torch.arange(s["max_kv"], device=n.device)
    # the first and the last ones before all, those that do not exist behind all
    rank = torch.where((e < s["sinks"]) | (e >= n - s["recent"]), math.inf, s["weights"])
    rank = torch.where(e < n, rank, -1.0)
    cut = n > s["trigger"]
    top = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :B]   # of equal ones the lower entry
    top = torch.sort(top, 1)[0]
    left = torch.where(cut, min(B, s["max_kv"]), n)
    j = torch.arange(s["max_out"], device=n.device)
    old = torch.where(cut, torch.nn.functional.pad(top, (0, max(0, s["max_out"] - top.shape[1])))[:, :s["max_out"]], j)
    there = j < left
    old = torch.where(there, old, 0)
    slots = torch.where(there, s["table"].long().gather(1, old // s["page"]) * s["page"] + old % s["page"], 0)[there]
    k, v = (_packed(s["cache"], s["dim"], slots, of) for of in (False, True))
    _put(s["cache"], s["dim"], s["slots"], k, v)
    w = torch.where(there, s["weights"].gather(1, old), 0.0)
    s["weights_out"][:, :w.shape[1]] = w
    s["weights_out"][:, w.shape[1]:] = 0.0
    s["len_out"].copy_(left[:, 0])
    kept = torch.where(there, old, -1)[:, :B].int()
    if kept.shape[1] < B:
        kept = torch.nn.functional.pad(kept, (0, B - kept.shape[1]), value=-1)
    return (kept, s["len_out"], s["weights_out"],
            _get(s["cache"], s["dim"], s["slots"], False).to(s["dtype"]),
            _get(s["cache"], s["dim"], s["slots"], True).to(s["dtype"]))


def _handle(s):
    """What a program makes once beside its layer: the rotation's table, the cache's handle."""
    if "handle" not in s:
        if s["op"] == "rope":
            from sparse_long_context_tail_gb300.rotary import RotaryEmbedding
            c = s["case"]
            s["handle"] = RotaryEmbedding(c["dim"], c["rotary"], c["base"], interleaved=c["interleaved"],
                                          scaling=c["scaling"], factor=c["factor"], original_len=8192)
        else:
            from sparse_long_context_tail_gb300.kvcache import QuantKVCache
            s["handle"] = QuantKVCache(s["cache"].shape[0] * 16, s["heads"], s["dim"], k_exp=s["k_exp"],
                                       storage=s["cache"])
    return s["handle"]


def run(state):
    s = state
    if not own:
        return {"rope": _plain_rope, "weigh": _plain_weigh, "evict": _plain_evict}[s["op"]](s)
    if s["op"] == "rope":
        return _handle(s).apply(s["q"], s["k"], s["pos"], num_tokens=s["count"], out=s["out"])
    cache = _handle(s)
    if s["op"] == "weigh":
        return cache.accumulate(s["q"], s["lse"], s["table"], s["kv_len"], s["page"], s["weights"],
                                cu_q=None if s["single"] else s["cu_q"], max_q_len=s["max_q"], window=s["window"],
                                sinks=s["sinks"], decay=s["decay"], out=s["out"])
    kept = cache.evict(s["weights"], s["table"], s["kv_len"], s["page"], s["budget"], trigger=s["trigger"],
                       sinks=s["sinks"], recent=s["recent"], page_table_out=s["table_out"],
                       weights_out=s["weights_out"], kv_len_out=s["len_out"])
    return (kept, s["len_out"], s["weights_out"], *cache.read(s["slots"], dtype=s["dtype"]))


# ---------------------------------------------------------- 64-bit results --

def _exact_entries(cache, dim, slots, of_values):
    """64-bit values of the given slots' K or V by byte addresses, without the exponent."""
    H = cache.shape[1]
    P = max(1, dim // 128)
    D = dim // P
    j = torch.arange(dim, device=cache.device)
    r = (slots % 16)[:, None]
    p, jj = j // D, j % D
    if of_values:
        c = D // 16
        code = 8 * dim + p * 8 * D + r // 8 * 4 * D + jj // (D // 8) * 8 * c + r % 8 * c + jj % (D // 8) // 2
        scale = 17 * dim + p * D + r // 8 * (D // 2) + jj // 16 * 8 + r % 8
    else:
        code = p * 8 * D + r * (D // 2) + jj // 2
        scale = 16 * dim + r * (dim // 16) + j // 16
    block = cache[slots // 16]                                        # [T, H, 18 d]
    take = lambda at: torch.gather(block, 2, at[:, None].expand(-1, H, -1)).long()  # noqa: E731
    nib = take(code) >> 4 * (j % 2) & 15
    e, m = nib % 8 // 2, nib % 2
    x = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + m / 2), m / 2) * (1 - 2 * (nib // 8))
    byte = take(scale)
    e, m = byte // 8, byte % 8
    return x * torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + m / 8), m / 8 * 2.0 ** -6)


def _exact_rope(s):
    """Rotation as the product with a complex number, in chunks."""
    n, outs = s["rotary"], []
    last = s["pos"].numel() if s["count"] is None else int(s["count"])
    for x in (s["q"], s["k"]):
        y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        for a in range(0, last, 16384):
            part = x[a:min(last, a + 16384)].double()
            turn = torch.polar(torch.full((1, n // 2), float(s["scale"]), dtype=torch.float64, device=x.device),
                               s["pos"][a:a + part.shape[0], None] * s["freqs"])[:, None]
            i = torch.arange(n // 2, device=x.device)
            first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + n // 2)
            z = torch.complex(part[..., first], part[..., second]) * turn
            part[..., first], part[..., second] = z.real, z.imag
            y[a:a + part.shape[0]] = part
        outs.append(y)
    return tuple(outs)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rope":
        return _exact_rope(s)
    lens, news = _lengths(case)
    if s["op"] == "evict":
        w, kept = s["weights"].tolist(), []
        weights = torch.zeros(s["weights_out"].shape, dtype=torch.float64, device=DEVICE)
        slots = []
        for r, n in enumerate(lens):
            mine = list(range(n))
            if n > s["trigger"]:
                middle = range(s["sinks"], n - s["recent"])
                heavy = sorted(middle, key=lambda e: (-w[r][e], e))[:s["budget"] - s["sinks"] - s["recent"]]
                mine = list(range(s["sinks"])) + sorted(heavy) + list(range(n - s["recent"], n))
            mine = torch.tensor(mine, dtype=torch.long, device=DEVICE)
            weights[r, :mine.numel()] = s["weights"][r, mine].double()
            slots.append(s["table"][r, mine // s["page"]].long() * s["page"] + mine % s["page"])
        parts = torch.split(torch.cat(slots), 8192)
        return (None, None, weights, *(torch.cat([_exact_entries(s["cache"], s["dim"], p, of) for p in parts])
                                       for of in (False, True)))
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEVICE)
    H, group, row = s["heads"], s["q"].shape[1] // s["heads"], 0
    for r, (n, new) in enumerate(zip(lens, news)):
        e = torch.arange(n, device=DEVICE)
        slots = s["table"][r, e // s["page"]].long() * s["page"] + e % s["page"]
        k = torch.cat([_exact_entries(s["cache"], s["dim"], p, False) for p in torch.split(slots, 8192)])
        k *= 2.0 ** s["k_exp"]
        out[r, :n] = s["decay"] * s["weights"][r, :n].double()
        for i in range(new):
            p = n - new + i
            see = e <= p
            if s["window"]:
                see &= (e > p - s["window"]) | (e < s["sinks"])
            at = e[see]
            if at.numel():
                q = s["q"][row].double().view(H, group, -1)
                x = torch.einsum("hgd,ehd->hge", q, k[at]) / math.sqrt(s["dim"])
                out[r, at] += torch.exp(x - s["lse"][row].double().view(H, group, 1)).sum((0, 1))
            row += 1
    return out
