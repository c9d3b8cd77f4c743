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
