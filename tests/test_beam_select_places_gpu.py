"""tl_beam_select: where a row of logits begins does not enter its result, so beams of the same logits stay in their order."""
import numpy as np
import pytest
import torch

from tests.test_beam_select_gpu import Case, normal, some_scores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("scale", [2.5, 1e5])
@pytest.mark.parametrize("V", [3, 101, 1003, 8191, 16387, 50001, 70006])
def test_equal_beams_stay_in_order(B, V, scale, half):
    users, K, N = 3, 8, 40
    x = normal(V, users, 1, V, scale=scale, half=half).expand(users, K, V).contiguous()
    c = Case(B, x, np.full((users, K), -2.0), N).run()
    assert (c.lse == c.lse[:, :1]).all()
    n = min(N, K * V)
    for b in range(users):
        row = x[b, 0].double().numpy()
        beam, token = (a.ravel() for a in np.meshgrid(np.arange(K), np.arange(V), indexing="ij"))
        best = np.lexsort((token, beam, -row[token]))[:n]
        assert c.parents[b, :n].tolist() == (b * K + beam[best]).tolist() and c.tokens[b, :n].tolist() == token[best].tolist()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("scale", [2.5, 1e5])
@pytest.mark.parametrize("V", [5, 1000, 9001, 65544, 150001])
def test_the_same_bits_wherever_rows_begin(B, V, scale, half):
    users, K, N = 2, 4, 16
    x, scores = normal(V + 1, users, K, V, scale=scale, half=half), some_scores(5, users, K)
    first = None
    for offset in range(9):
        for gap in (0, 1, 2, 7, 8):
            rows = users * K
            store = torch.full((rows * (V + gap) + 16,), float("nan"), dtype=x.dtype, device="cuda")
            place = store[offset:offset + rows * (V + gap)].view(rows, V + gap)[:, :V]
            c = Case(B, x, scores, N, place=place).run()
            if first is None:
                first = c.check()
            for a, b in ((c.parents, first.parents), (c.tokens, first.tokens), (c.out, first.out), (c.lse, first.lse)):
                assert torch.equal(a, b), (offset, gap)
