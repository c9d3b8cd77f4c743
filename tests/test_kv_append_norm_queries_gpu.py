"""tl_kv_append_norm's queries to the bound that follows from their present summation."""
import numpy as np
import pytest
import torch

from tests.kv_cases import Batch, f64
from tests.test_kv_append_norm_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


# A thread adds up 16 squares (exact in fp32) in four chains, 3 roundings, and joins them, 2; the row's threads' sums are log2(D /
# 16) more, at most 3; the mean and eps 1: 9 of 2^-24, halved by the root, and one and a half for the corrected root.  An
# element's two products with the tables, their sum and the product with the factor are 3: 9 in all, relative to the
# products' magnitudes, at most sqrt(2) of the row's largest normed element: below 2^-20 of it.  Then 2^-8 for bf16.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", ["all", 32, 0])
def test_queries_to_the_derived_bound(B, rot, interleaved, D):
    b = Batch([700, 1, 40], [700, 300, 2000], H=6, Hkv=1, D=D, ps=64, seed=71)
    c = Case(B, b, rot=D if rot == "all" else rot, interleaved=interleaved)
    c.call()
    assert B.tl_query_status(c.sig)[0] == 0
    q, _ = c.expected()
    assert (np.abs(f64(c.q_out) - q) <= 2.0 ** -8 * np.abs(q) + 2.0 ** -20 * c.q_large).all()
    assert torch.isfinite(c.q_out).all()
