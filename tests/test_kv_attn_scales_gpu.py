"""tl_kv_attn for few query rows where the block scales of one sequence differ by far more than fp16 spans."""
import numpy as np
import pytest

from tests.kv_cases import Batch, f64
from tests.kv_rows import check_rows, expected_rows
from tests.test_kv_attn_gpu import Call

pytestmark = pytest.mark.gpu
A, C, E = dict(H=4, Hkv=2, D=128, ps=16), dict(H=3, Hkv=3, D=64, ps=48), dict(H=16, Hkv=2, D=64, ps=16)
DRAFTS = [(A, 2), (A, 4), (A, 30), (C, 2), (C, 4), (C, 60), (E, 2), (E, 4)]  # up to 64 query rows of a kv head
SOME = [(A, 1), (A, 3), (A, 30), (C, 1), (C, 3), (C, 60), (E, 1), (E, 3)]


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


def check(B, b, edit, causal=True, scale=0.0):
    c = Call(B, b, edit=edit, causal=causal, scale=scale, spread=1).run()
    assert B.tl_query_status(c.sig)[0] == 0
    check_rows(f64(c.out), f64(c.lse),
               *expected_rows(b, f64(c.q), c.kc, c.ks, c.vc, c.vs, causal, scale or b.D ** -0.5))
    return c


@pytest.mark.parametrize("layout,q_len", DRAFTS)
@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("above", [12, 28, 100])
def test_a_page_that_only_the_last_rows_see(B, layout, which, above, q_len):
    """The last new tokens begin a page of their own, of far larger keys or values: earlier rows do not feel it."""
    ps = layout["ps"]
    lens = [ps * (-(-(q_len + 20) // ps)) + 1, ps * (-(-(q_len + 200) // ps)) + 2]

    def edit(c):
        for s in range(2):
            last = c.b.table[s, c.b.lens[s] // ps]
            if which != "v":
                c.ks[last] = 121 + above
            if which != "k":
                c.vs[last] = 121 + above
    check(B, Batch([q_len] * 2, lens, seed=41, **layout), edit)


@pytest.mark.parametrize("layout,q_len", SOME)
@pytest.mark.parametrize("above", [24, 40, 90])
@pytest.mark.parametrize("at", [0, 3, -1])
def test_large_keys_that_a_query_does_not_meet(B, layout, q_len, above, at):
    """One page's keys are far larger, in a dim where every query is 0: all other keys' scores count as they are."""
    def edit(c):
        c.q[..., 5] = 0
        page = c.b.table[0, at % (-(-c.b.lens[0] // c.b.ps))]
        c.ks[page] = 121 + above
        c.kc[page] = 0
        c.kc[page, :, :, 5] = 0x70
    check(B, Batch([q_len], [400 + q_len], seed=42, **layout), edit)


@pytest.mark.parametrize("layout,q_len", SOME)
@pytest.mark.parametrize("above", [24, 40, 90])
@pytest.mark.parametrize("at", [0, 3, -1])
def test_large_values_of_little_weight(B, layout, q_len, above, at):
    """One page's values are 2^above larger and their weights about as much smaller: they and the rest both count."""
    def edit(c):
        c.q[..., 5] = 1.0
        c.kc[:, :, :, 5] = 0
        page = c.b.table[0, at % (-(-c.b.lens[0] // c.b.ps))]
        c.vs[page] = 121 + above
        c.kc[page], c.ks[page] = 0, 127
        c.kc[page, :, :, 5] = ora_code(-above * 0.6931 * c.b.D ** 0.5)
    check(B, Batch([q_len], [400 + q_len], seed=43, **layout), edit, causal=False)


def ora_code(x):
    from oracle import kv_cache as ora
    return ora.encode(np.clip(x, -448, 448))


@pytest.mark.parametrize("layout,q_len", SOME)
@pytest.mark.parametrize("causal", [True, False])
def test_every_page_of_another_scale(B, layout, q_len, causal):
    """Scales of keys and values from 2^-60 to 2^20 in any order, all-zero blocks of byte 0 among them."""
    def edit(c):
        rng = np.random.default_rng(44)
        c.ks[:] = rng.integers(67, 127, c.ks.shape)
        c.vs[:] = rng.integers(67, 147, c.vs.shape)
        for s, j in ((0, 1), (1, 4)):
            page = c.b.table[s, j]
            c.ks[page], c.kc[page], c.vs[page], c.vc[page] = 0, 0, 0, 0
    check(B, Batch([q_len, q_len + 1], [300 + q_len, 700], seed=44, **layout), edit, causal)


@pytest.mark.parametrize("q_len", [1, 3, 16])
def test_a_long_context_of_mixed_scales(B, q_len):
    """Shared by many blocks, whose partial results have references of their own."""
    def edit(c):
        rng = np.random.default_rng(45)
        c.vs[:] = rng.choice([101, 121, 161], c.vs.shape, p=[0.1, 0.8, 0.1])
        c.ks[:] = rng.choice([91, 121], c.ks.shape, p=[0.1, 0.9])
    check(B, Batch([q_len], [4000], H=4, Hkv=1, D=128, ps=64, seed=45), edit)


@pytest.mark.parametrize("q_len", [4, 30])
def test_nan_blocks_beside_large_ones(B, q_len):
    """A page of byte 255 is NaN for the rows that see it; a large page beside it changes nothing for the others."""
    ps = 16
    n = ps * (-(-(q_len + 60) // ps)) + 1

    def edit(c):
        last = c.b.table[0, n // ps]
        c.vs[last], c.ks[last] = 255, 161
    b = Batch([q_len, 2], [n, 50], H=4, Hkv=2, D=128, ps=ps, seed=46)
    c = Call(B, b, edit=edit, spread=1).run()
    out, lse = f64(c.out), f64(c.lse)
    assert np.isnan(out[q_len - 1]).all()
    c.vs[c.vs == 255] = 121
    want = expected_rows(b, f64(c.q), c.kc, c.ks, c.vc, c.vs, True, b.D ** -0.5)
    keep = np.r_[0:q_len - 1, q_len:q_len + 2]
    check_rows(out[keep], lse[:, keep], want[0][keep], want[1][:, keep], want[2][keep], want[3][:, keep])


def falling_weights(c, step):
    """Every page's values are 2^step larger than the page's before and its weights about as much smaller (step 0: the second
    half of the pages 2^28 larger): all pages count alike."""
    c.q[..., 5] = 1.0
    c.rng = np.random.default_rng(48)
    for s in range(len(c.b.q)):
        pages = -(-c.b.lens[s] // c.b.ps)
        for j in range(pages):
            up = step * j if step else 28 * (2 * j >= pages)
            page = c.b.table[s, j]
            c.vs[page] = 115 + up
            c.ks[page] = 127
            c.kc[page] = 0
            c.kc[page, :, :, 5] = ora_code(-up * 0.6931 * c.b.D ** 0.5)
            c.kc[page, :, :, 6] = c.kc[page, :, :, 7] = ora_code(c.rng.standard_normal(c.kc[page, :, :, 6].shape) * 4)


# Enough tiles that a warp goes through many chunks of one tile.
@pytest.mark.parametrize("layout,q_len", [(dict(H=8, Hkv=8, D=128, ps=64), 1), (dict(H=16, Hkv=4, D=64, ps=64), 4),
                                          (dict(H=16, Hkv=4, D=128, ps=32), 4)])
@pytest.mark.parametrize("step", [0, 1, 2, 4])
def test_scales_that_rise_as_weights_fall(B, layout, q_len, step):
    seqs = 160
    rng = np.random.default_rng(47)
    lens = [int(x) for x in rng.integers(200, 400, seqs)]
    check(B, Batch([q_len] * seqs, lens, seed=47, **layout), lambda c: falling_weights(c, step))


@pytest.mark.parametrize("q_len,n,seqs", [(1, 37, 1), (1, 37, 40), (3, 60, 300), (16, 700, 2), (1, 3000, 3)])
@pytest.mark.parametrize("score", [20.0, 96.0, 400.0])
def test_large_values_of_no_weight(B, q_len, n, seqs, score):
    """One key has all the weight and values of 2^-80; the last page's values are 2^134 larger and have none."""
    def edit(c):
        c.q[:] = 0
        c.q[..., 5] = 1.0
        c.kc[:, :, :, 5] = 0
        c.ks[:], c.vs[:] = 127, 120
        for s in range(seqs):
            c.vs[c.b.table[s, 0]], c.vs[c.b.table[s, n // 16]] = 47, 181
            c.kc[c.b.table[s, 0], :, 3, 5] = ora_code(score)
    check(B, Batch([q_len] * seqs, [n] * seqs, H=2, Hkv=1, D=64, ps=16, seed=51), edit, causal=False, scale=1.0)
