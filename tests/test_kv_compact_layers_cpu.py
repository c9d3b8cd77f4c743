"""tl_kv_compact moves tokens in place: a layer's cache that is given twice is refused."""
import ctypes

import pytest

from tests.test_drafts_beams_cpu import B  # noqa: F401
from tests.test_serving_cpu import cache


@pytest.mark.parametrize("n", [2, 3, 65, 4096])
@pytest.mark.parametrize("side", ["k", "v"])
def test_a_cache_twice_is_refused(B, side, n):  # noqa: F811
    def call(*addresses):
        caches = (B.tl_kv_cache * n)(*[cache(B, k=a, v=b) for a, b in addresses])
        a = B.tl_kv_compact_args(n_layers=n, B=3, max_pages=4, max_kept=5, caches=ctypes.addressof(caches), kept=4, n_kept=4, cu_seqlens=4,
                                 seq_lens=4096, page_table=4, seq_lens_out=8192, signals=64)
        assert B.lib.tl_kv_compact(ctypes.byref(a), None) == B.TL_ERR_INVALID
        return B.tl_last_error()
    apart = [((n - i) << 20, (n + 1 + i) << 20) for i in range(n)]
    twice = list(apart)
    twice[-1] = (apart[0][0], apart[-1][1]) if side == "k" else (apart[-1][0], apart[0][1])
    assert "twice" in call(*twice)
