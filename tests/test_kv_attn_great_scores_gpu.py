"""tl_kv_attn with scores so great that fp32 steps of theirs are far more than a softmax spans: the largest key has it all."""
import numpy as np
import pytest

from oracle import kv_cache as ora
from tests.kv_cases import Batch, f64
from tests.test_kv_attn_gpu import Call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


@pytest.mark.parametrize("q_len", [1, 20, 150])
@pytest.mark.parametrize("exponent", [5, 10, 14, 18, 20, 24, 60, 100])
@pytest.mark.parametrize("at", [0, 170, 1499])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_key_has_it_all(B, q_len, exponent, at, sign):
    """Scores are 2^exponent times a code, and the largest is 2^9 or more above the next: it is taken alone.  A query's one element and the codes are exact, so a score is off by its own rounding to fp32, less than
    2^-20 of it, and the next key is 2^-5 of it and more away."""
    other, best = (224.0, 240.0) if sign > 0 else (448.0, 416.0)

    def edit(c):
        c.ks[:], c.vs[:] = 127, 121
        c.q[:] = 0
        c.q[..., 9] = sign * 2.0 ** exponent
        c.kc[:, :, :, 9] = ora.encode(np.array(other))
        c.kc[c.b.table[0, at // 64], :, at % 64, 9] = ora.encode(np.array(best))
    b = Batch([q_len], [1500], H=4, Hkv=1, D=128, ps=64, seed=71)
    c = Call(B, b, edit=edit, scale=1.0, causal=False, max_q_len=q_len).run()
    assert B.tl_query_status(c.sig)[0] == 0
    want = ora.values(c.vc, c.vs, b.table[0], 1500)[at, 0]
    out, lse = f64(c.out), f64(c.lse)
    assert (np.abs(out - want) <= 2.0 ** -8 * np.abs(want)).all()
    score = sign * best * 2.0 ** exponent
    # (2^7 is the reference's own offset, which a great score's fp32 steps may swallow)
    assert (np.abs(lse - score) <= 2.0 ** -20 * abs(score) + 10.0).all()


@pytest.mark.parametrize("q_len", [1, 20, 150])
@pytest.mark.parametrize("exponent", [20, 60])
def test_equal_great_scores_share_it(B, q_len, exponent):
    def edit(c):
        c.ks[:], c.vs[:] = 127, 121
        c.q[:] = 0
        c.q[..., 9] = 2.0 ** exponent
        c.kc[:, :, :, 9] = ora.encode(np.array(-240.0))
        c.vc[:] = 0x38   # 1
        for at in (3, 700, 701, 1400):
            c.kc[c.b.table[0, at // 64], :, at % 64, 9] = ora.encode(np.array(240.0))
            c.vc[c.b.table[0, at // 64], :, at % 64] = ora.encode(np.array(float(at % 5 + 2)))
    b = Batch([q_len], [1500], H=4, Hkv=1, D=128, ps=64, seed=72)
    c = Call(B, b, edit=edit, scale=1.0, causal=False, max_q_len=q_len).run()
    want = np.mean([at % 5 + 2.0 for at in (3, 700, 701, 1400)]) * 2.0 ** -6
    # equal scores have equal weights: the mean, rounded to bf16 once (sums of eight terms in fp32)
    assert (np.abs(f64(c.out) - want) <= (2.0 ** -8 + 2.0 ** -18) * want).all()
