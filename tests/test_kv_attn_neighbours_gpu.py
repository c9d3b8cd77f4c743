"""tl_kv_attn where blocks to an SM serve several sequences: no sequence's result depends on its neighbours."""
import numpy as np
import pytest

from tests.kv_cases import Batch, f64
from tests.kv_rows import check_rows, expected_rows
from tests.test_kv_attn_gpu import Call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


# More tiles than blocks, so that a block goes from one sequence to the next.  Every other sequence has value blocks 2^40
# (2^100) larger; those between end in the first half of a chunk of 32 tokens.
@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("above", [40, 100])
@pytest.mark.parametrize("D", [64, 128])
def test_a_neighbours_value_scale_does_not_enter(B, q_len, above, D):
    seqs = 600
    lens = [70 if s % 2 == 0 else (5, 37, 69, 48)[s // 2 % 4] for s in range(seqs)]

    def edit(c):
        c.vs[:] = 121
        for s in range(0, seqs, 2):
            c.vs[c.b.table[s][c.b.table[s] >= 0]] = 121 + above
    b = Batch([q_len] * seqs, lens, H=8, Hkv=2, D=D, ps=16, seed=31)
    c = Call(B, b, edit=edit, max_q_len=q_len).run()
    assert B.tl_query_status(c.sig)[0] == 0
    check_rows(f64(c.out), f64(c.lse), *expected_rows(b, f64(c.q), c.kc, c.ks, c.vc, c.vs, True, D ** -0.5))


# The same between the kv heads of one sequence.
@pytest.mark.parametrize("q_len", [1, 4])
def test_a_heads_value_scale_does_not_enter_the_next(B, q_len):
    seqs, heads = 90, 8

    def edit(c):
        c.vs[:, 0::2], c.vs[:, 1::2] = 121, 171
    b = Batch([q_len] * seqs, [(37, 5, 48)[s % 3] for s in range(seqs)], H=heads, Hkv=heads, D=64, ps=16, seed=32)
    c = Call(B, b, edit=edit, max_q_len=q_len).run()
    assert B.tl_query_status(c.sig)[0] == 0
    check_rows(f64(c.out), f64(c.lse), *expected_rows(b, f64(c.q), c.kc, c.ks, c.vc, c.vs, True, 0.125))
