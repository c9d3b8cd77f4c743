"""The largest vocabulary of tl_beam_select: places in a row are counted in 32 bits."""
import ctypes

import pytest

from tests.test_drafts_beams_cpu import B, beam_args  # noqa: F401


@pytest.mark.parametrize("K,V", [(1, (1 << 30) + 1), (1, (1 << 31) - 1), (1, (1 << 31) - 16), (2, (1 << 29) + 1), (64, 1 << 25)])
def test_more_logits_are_refused(B, K, V):  # noqa: F811
    assert B.tl_beam_select_workspace_size(1, K, 4, V) == 0
    a = beam_args(B, B=1, K=K, V=V, row_stride=V, workspace_bytes=1 << 40)
    assert B.lib.tl_beam_select(ctypes.byref(a), None) == B.TL_ERR_UNSUPPORTED
    assert "2^30" in B.tl_last_error()


@pytest.mark.parametrize("K,V", [(1, 1 << 30), (2, 1 << 29), (64, 1 << 24)])
def test_as_many_are_not(B, K, V):  # noqa: F811
    assert B.tl_beam_select_workspace_size(1, K, 4, V) > 0
    a = beam_args(B, B=1, K=K, V=V, row_stride=V, workspace_bytes=0)  # refused for the workspace, not for the size
    assert B.lib.tl_beam_select(ctypes.byref(a), None) == B.TL_ERR_INVALID
