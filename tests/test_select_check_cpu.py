"""upf_select_tokens_check refuses what upf_select_tokens refuses, with the same words."""
import numpy as np
import pytest

from sparse_long_context_tail_gb300 import _binding as B
from sparse_long_context_tail_gb300 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return B.load()


def test_without_a_context():
    b, keep = B.make_batch(0x1000, np.asarray([0, 1000], np.int32), 32, 8, 128, None)
    io = B.make_compact_io(cu_seqlens_out=16, total_kept=16)
    words = []
    for call in (lambda: B.upf_select_tokens(None, b, B.make_params(), 16, 4096, 16, 1024, 0, 0, 16, 16, io, 256, 1 << 20),
                 lambda: B.upf_select_tokens_check(None, b, B.make_params(), 16, 4096, 16, 1024, 16, 16, io, 256, 1 << 20)):
        with pytest.raises(B.UpfError) as e:
            call()
        words.append((e.value.status, e.value.message))
    assert words[0] == words[1] and "context" in words[0][1]


def test_a_check_of_nothing():
    assert B.load().upf_select_tokens_check(None, None, None, None, 0, None, 0, None, None, None, None, 0) == 1
    assert "NULL" in B.upf_last_error()
