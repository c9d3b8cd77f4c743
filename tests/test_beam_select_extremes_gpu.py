"""tl_beam_select with scores and sums at the ends of fp32: the same beams offer something whichever way the best are found."""
import numpy as np
import pytest
import torch

from tests.test_beam_select_gpu import Case, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


# Plateaus of more values than the list holds are taken value by value, a few tokens above the rest from the list.
@pytest.mark.parametrize("plateau", [False, True])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_a_score_less_lse_that_leaves_fp32_offers_nothing(B, plateau, sign):
    x = normal(3, 1, 3, 20000)
    if plateau:
        x[0, 0] = 0.0
    x[0, 1] = sign * 3e38
    c = Case(B, x, np.array([[0.0, -sign * 3e38, -50.0 if plateau else -1.0]]), 30).run()
    assert set(c.parents[0].tolist()) <= {0, 2} and torch.isfinite(c.out).all()
    assert abs(float(c.lse[0, 1]) - sign * 3e38) <= 2.0 ** -20 * 3e38
