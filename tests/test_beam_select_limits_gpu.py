"""tl_beam_select on the largest vocabulary."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


def test_the_largest_vocabulary(B):
    V, N = 1 << 30, 8
    x = torch.empty(V + 8, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(3))
    row = x[3:3 + V][None]
    x[:3], x[3 + V:] = 100.0, float("nan")
    places = [V - 1, 0, V - 2, 5, V // 2 + 1, V - 8191, 16383, V - 65537]
    for i, t in enumerate(places):
        row[0, t] = 20.0 - 0.5 * i
    ws = torch.zeros(B.tl_beam_select_workspace_size(1, 1, N, V), dtype=torch.uint8, device="cuda")
    parents, tokens = (torch.full((1, N), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    out, lse = torch.full((1, N), 9.0, device="cuda"), torch.full((1, 1), 9.0, device="cuda")
    B.tl_beam_select(row, torch.tensor([[-3.0]], device="cuda"), parents, tokens, out, ws, lse=lse)
    want = math.log(sum(float(c.double().exp().sum()) for c in row[0].split(1 << 26)))
    assert parents.tolist() == [[0] * N] and tokens.tolist() == [places]
    # Logits lie up to 28 below the maximum: 3 (28 + 2) steps of 2^-24 in the exponent, 4 of 2^-22 for the exponentials, 12 of
    # 2^-24 for the sums; and the rounding of the result.
    tol = (3 * 30 + 16 + 12) * 2.0 ** -24 + 2.0 ** -24 * want
    assert abs(float(lse) - want) <= tol
    for i in range(N):
        score = -3.0 + (20.0 - 0.5 * i) - want
        assert abs(float(out[0, i]) - score) <= tol + 2.0 ** -24 * abs(score)
