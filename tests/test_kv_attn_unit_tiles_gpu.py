"""tl_kv_attn and tl_kv_tree_attn, many rows: units of two query tiles among units of one, whose second tile is left out."""
import numpy as np
import pytest
import torch

from tests.kv_cases import Batch, check_attention, expected_attention, f64
from tests.test_kv_attn_gpu import Call
from tests.test_kv_tree_attn_gpu import TreeCall

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


# A unit to a sequence and some eight units to a run, so that what a run keeps of four units is used again: 132 rows, then
# `between` units of 36.  NaN values lie among the new tokens of every unit, in dims of its own, and scales differ from one
# sequence to the next by up to 2^24.
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("between", [1, 3, 4, 7])
def test_a_units_nan_and_scales_are_its_own(B, between, D, tree):
    seqs = 1200
    q = [33 if s % (between + 1) == 0 else 9 for s in range(seqs)]

    def edit(c):
        b = c.b
        for s in range(seqs):
            pages = b.table[s][b.table[s] >= 0]
            c.ks[pages], c.vs[pages] = 118 + s % 5, 108 + 6 * (s % 5)
            pos = b.lens[s] - 1 - s % 4
            c.vc[b.table[s, pos // b.ps], :, pos % b.ps, s * 13 % D] = 127
    b = Batch(q, [n + s % 3 for s, n in enumerate(q)], H=4, Hkv=1, D=D, ps=64, seed=61)
    c = (TreeCall if tree else Call)(B, b, edit=edit, max_q_len=33).run()
    if tree:
        want = c.expected()
    else:
        want = expected_attention(b, f64(c.q), c.kc, c.ks, c.vc, c.vs, True, D ** -0.5)
    for _ in range(5):
        assert B.tl_query_status(c.sig)[0] == 0
        got = f64(c.out)
        assert np.array_equal(np.isnan(got), np.isnan(want[0])) and np.isnan(got).any()
        check_attention(got, f64(c.lse), *want)
        torch.cuda.synchronize()
        c.run()
