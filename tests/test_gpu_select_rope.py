"""Selection with a rotary embedding: calls that are refused, and outputs that serve several calls."""
import numpy as np
import pytest
import torch

from sparse_long_context_tail_gb300 import _binding as B
from test_gpu_rope import BF16, DEV, F16, places, rand, rotation

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def inputs(T=700, Hq=8, H=2, d=128, dtype=BF16):
    from sparse_long_context_tail_gb300.selector import TokenSelector
    rows = rand((T, Hq + 2 * H, d), dtype, 3)
    cu = np.array([0, 300, T], np.int32)
    return TokenSelector(0), rotation(d, 64), rows, rows[:, :Hq], rows[:, Hq:Hq + H], places(T, 4), cu, torch.from_numpy(cu).to(DEV)


def test_a_refused_selection_leaves_queries_and_keys_as_they_were():
    """In place: a call that is refused for any of its arguments has turned nothing, so that it can be made again."""
    sel, rope, rows, q, k, pos, cu, cu_dev = inputs()
    params = B.make_params(32, 16, 32, 32, 0.6)
    hidden, slots = rows.reshape(700, -1), torch.arange(700, device=DEV)
    history = torch.zeros(2, 800, dtype=torch.int32, device=DEV)

    def out():
        x = sel.alloc_outputs(cu, params.block, hidden, pos, slots)
        x.q_out, x.k_out = q, k
        return x

    good = dict(hidden=hidden, positions=pos, slots=slots, params=params, rope=rope)
    was = rows.clone()
    for bad, word in [(dict(params=B.make_params(32, 16, 32, 32, 0.0)), "top_p"), (dict(hidden=None), "hidden_in"),
                      (dict(slots=None), "slot_in"), (dict(hidden=torch.zeros(700, 12, dtype=torch.uint8, device=DEV)), "row_bytes"), (dict(history=history), "history"),
                      (dict(kv_of_q=[0] * 8), "kv_of_q"), (dict(heads=(7, 2, 128)), "H_q"), (dict(heads=(4, 2, 128)), "q has shape"),
                      (dict(heads=(8, 4, 128)), "k has shape"), (dict(heads=(8, 2, 64)), "shape"), (dict(cu=cu - 1), "cu_seqlens"),
                      (dict(cu=cu + np.int32([0, 0, 1])), "q has shape"), (dict(positions=None), "positions"), (dict(positions=pos.int()), "positions"),
                      (dict(positions=pos[:600]), "tokens")]:
        a = dict(good, out=out())
        a.update(bad)
        heads, host = a.pop("heads", (8, 2, 128)), a.pop("cu", cu)
        with pytest.raises((ValueError, B.UpfError), match=word):
            sel.select_tokens(q, k, host, cu_dev, *heads, **a)
        assert torch.equal(rows, was), word
    q2, k2 = rope.apply(q, k, pos)
    want = sel.select_tokens(q2, k2, cu, cu_dev, 8, 2, 128, hidden=hidden, positions=pos, slots=slots, params=params)
    n = int(want.total_kept)
    keep = want.hidden_out[:n].clone()
    got = sel.select_tokens(q, k, cu, cu_dev, 8, 2, 128, out=out(), **good)
    assert got.q_out is q and torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(got.scores, want.scores)
    # hidden_in are the projection's rows themselves, turned by then
    assert int(got.total_kept) == n and torch.equal(got.hidden_out[:n, 10 * 128:], keep[:, 10 * 128:]) and sel.status() == 0


def test_queries_of_another_type_are_refused_with_a_rotary_embedding():
    """The selection scores bf16; the rotation alone takes fp16 too."""
    sel, rope, rows, q, k, pos, cu, cu_dev = inputs(dtype=F16)
    with pytest.raises(ValueError, match="bfloat16"):
        sel.select_tokens(q, k, cu, cu_dev, 8, 2, 128, positions=pos, rope=rope)
    assert torch.isfinite(rope.apply(q, k, pos)[0]).all()


def test_outputs_that_serve_calls_of_several_lengths():
    """Outputs that were made for 700 tokens, given to a call of 450 and again to one of 700."""
    sel, rope, rows, q, k, pos, cu, cu_dev = inputs()
    params = B.make_params(32, 16, 32, 32, 0.6)
    out = None
    for T in (700, 450, 700, 1):
        host = np.array([0, min(300, T), T], np.int32)
        dev = torch.from_numpy(host).to(DEV)
        a = (q[:T], k[:T], host, dev, 8, 2, 128)
        got = sel.select_tokens(*a, positions=pos[:T], params=params, rope=rope, out=out)
        assert out is None or got is out
        out = got
        want = rope.apply(q[:T], k[:T], pos[:T])
        assert torch.equal(out.q_out[:T], want[0]) and torch.equal(out.k_out[:T], want[1])
        plain = sel.select_tokens(want[0], want[1], host, dev, 8, 2, 128, positions=pos[:T], params=params)
        n = int(plain.total_kept)
        assert int(out.total_kept) == n and torch.equal(out.scores[:T], plain.scores)
        assert torch.equal(out.pos_out[:n], plain.pos_out[:n])
    assert out.q_out.shape[0] == 700
    # too few rows
    small = sel.alloc_outputs(cu, params.block, None, pos)
    small.q_out, small.k_out = torch.empty_like(q[:600]), torch.empty_like(k)
    with pytest.raises(ValueError, match="q"):
        sel.select_tokens(q, k, cu, cu_dev, 8, 2, 128, positions=pos, params=params, rope=rope, out=small)
    assert sel.status() == 0
