"""tl_moe_decode's selection where logits are zeros of both signs: they are equal, and the lower index goes first."""
import numpy as np
import pytest

from tests.test_moe_decode_gpu import B, Call  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 7, 40])
@pytest.mark.parametrize("E,topk", [(2, 1), (8, 3), (64, 8), (100, 16)])
@pytest.mark.parametrize("normalize", [True, False])
def test_zeros_of_both_signs_are_equal(B, T, E, topk, normalize):  # noqa: F811
    rng = np.random.default_rng(T + E)
    logits = np.where(rng.random((T, E)) < 0.5, 0.0, -0.0).astype(np.float32)
    logits[:, E - 1] = np.where(rng.random(T) < 0.3, 1.0, logits[:, E - 1])
    logits[T // 2, 0] = -1.0
    c = Call(B, T, 64, 24, 40, E, topk, normalize=normalize, logits=logits, seed=E).run().check()
    if T == 1:
        return
    plain = next(t for t in range(T) if t != T // 2 and logits[t, E - 1] == 0)
    assert c.ids[plain].tolist() == list(range(topk))


def test_rounded_logits(B):  # noqa: F811
    logits = np.round(np.random.default_rng(9).standard_normal((60, 33))).astype(np.float32)
    assert np.signbit(logits[logits == 0]).any() and not np.signbit(logits[logits == 0]).all()
    Call(B, 60, 64, 24, 40, 33, 6, logits=logits, seed=9).run().check()
