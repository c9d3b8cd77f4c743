"""tl_kv_attn for many query rows: the cases of test_kv_attn_scales_gpu.py with chunks of prompts."""
import pytest

from tests import test_kv_attn_scales_gpu as few
from tests.test_kv_attn_scales_gpu import A, B, C, E  # noqa: F401

pytestmark = pytest.mark.gpu
CHUNKS = [(A, 40), (A, 150), (C, 150), (E, 40), (E, 150)]  # above 64 query rows of a kv head


@pytest.mark.parametrize("layout,q_len", CHUNKS)
@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("above", [12, 28, 100])
def test_a_page_that_only_the_last_rows_see(B, layout, which, above, q_len):  # noqa: F811
    few.test_a_page_that_only_the_last_rows_see(B, layout, which, above, q_len)


@pytest.mark.parametrize("layout,q_len", CHUNKS)
@pytest.mark.parametrize("above", [24, 40, 90])
@pytest.mark.parametrize("at", [0, 3, -1])
def test_large_keys_that_a_query_does_not_meet(B, layout, q_len, above, at):  # noqa: F811
    few.test_large_keys_that_a_query_does_not_meet(B, layout, q_len, above, at)


@pytest.mark.parametrize("layout,q_len", CHUNKS)
@pytest.mark.parametrize("above", [24, 40, 90])
@pytest.mark.parametrize("at", [0, 3, -1])
def test_large_values_of_little_weight(B, layout, q_len, above, at):  # noqa: F811
    few.test_large_values_of_little_weight(B, layout, q_len, above, at)


@pytest.mark.parametrize("layout,q_len", CHUNKS)
@pytest.mark.parametrize("causal", [True, False])
def test_every_page_of_another_scale(B, layout, q_len, causal):  # noqa: F811
    few.test_every_page_of_another_scale(B, layout, q_len, causal)


@pytest.mark.parametrize("q_len", [20, 100])
def test_a_long_context_of_mixed_scales(B, q_len):  # noqa: F811
    few.test_a_long_context_of_mixed_scales(B, q_len)


@pytest.mark.parametrize("q_len", [60, 150])
def test_nan_blocks_beside_large_ones(B, q_len):  # noqa: F811
    few.test_nan_blocks_beside_large_ones(B, q_len)


@pytest.mark.parametrize("layout,q_len", [(dict(H=8, Hkv=2, D=128, ps=64), 60), (dict(H=2, Hkv=1, D=64, ps=64), 200)])
@pytest.mark.parametrize("step", [0, 1, 2, 4])
def test_scales_that_rise_as_weights_fall(B, layout, q_len, step):  # noqa: F811
    few.check(B, few.Batch([q_len] * 3, [520, 300, 390], seed=49, **layout), lambda c: few.falling_weights(c, step))


def test_a_tail_of_small_weights_and_larger_values(B):  # noqa: F811
    """One key of weight nearly 1 and small values; 4000 keys of weight 2^-32 each whose values are 2^14 larger than its
    block's: together a fiftieth of the result."""
    n = 4096

    def edit(c):
        c.kc[:], c.vc[:] = 0, 0x38          # zeros; 1
        c.ks[:], c.vs[:] = 127, 127
        c.q[:] = 0
        c.q[..., 0] = 1.0
        first = c.b.table[0, 0]
        c.vs[first] = 113
        c.kc[first, :, 1:, 0] = few.ora_code(-448.0)
        c.kc[first, :, 0, 0] = few.ora_code(22.0)    # e^22 = 2^31.7 times the others' weights
    b = few.Batch([80], [n], H=1, Hkv=1, D=64, ps=64, seed=50)
    c = few.check(B, b, edit, causal=False, scale=1.0)
    tail = (n - 64) * 2.718281828459045 ** -22
    want = (2.0 ** -14 + tail) / (1 + tail)
    assert (abs(few.f64(c.out) - want) <= 2.0 ** -8 * want).all()


@pytest.mark.parametrize("q_len,n,seqs", [(60, 70, 1), (40, 700, 3), (150, 3000, 2)])
@pytest.mark.parametrize("score", [20.0, 96.0, 400.0])
def test_large_values_of_no_weight(B, q_len, n, seqs, score):  # noqa: F811
    few.test_large_values_of_no_weight(B, q_len, n, seqs, score)
