"""tl_kv_append refuses to rotate queries in place: checks that need no device."""
import ctypes

import pytest

from tests.test_serving_cpu import B, append_args  # noqa: F401

Q = 1 << 20
ROW = 4 * 128 * 2  # bytes of a token's four heads of 128


def refused(B, **kw):  # noqa: F811
    code = B.lib.tl_kv_append(ctypes.byref(append_args(B, **kw)), None)
    overlap = "overlap" in B.tl_last_error()
    assert code != 0 and (not overlap or code == B.TL_ERR_INVALID)  # without a device no call gets further
    return overlap


# three tokens of four heads of 128 in each
@pytest.mark.parametrize("strides,offset,overlap", [
    ((512, 128), 0, True), ((512, 128), 16, True), ((512, 128), -16, True), ((512, 128), 3 * ROW - 16, True),
    ((512, 128), -3 * ROW + 16, True), ((512, 128), 3 * ROW, False), ((512, 128), -3 * ROW, False),
    ((1024, 128), ROW, True),               # a fused projection's rows: the gap after a token holds one row, not three
    ((4096, 128), ROW, False),              # between a token and the next: room for all three
    ((4096, 128), 8192 - 3 * ROW, False), ((4096, 128), 8192 - 3 * ROW + 16, True), ((4096, 128), ROW - 16, True),
    ((4096, 128), 2 * 8192 + ROW, False), ((4096, 128), 2 * 8192 + ROW - 16, True), ((4096, 128), 2 * 8192 - 16, True),
    ((0, 128), 0, True), ((0, 128), ROW, False), ((0, 128), -3 * ROW, False), ((0, 128), -16, True),
    ((512, 1024), 3 * 2048, True)])         # heads far apart: from a token's first to its last
def test_overlap(B, strides, offset, overlap):  # noqa: F811
    assert refused(B, q=Q, q_out=Q + offset, q_token_stride=strides[0], q_head_stride=strides[1]) == overlap


def test_every_place_of_the_output(B):  # noqa: F811
    """Against rows written out one by one."""
    for stride in (0, 512, 520, 1024, 2048, 2056):
        for offset in range(-4 * ROW, 13 * ROW, 112):
            rows = [(t * stride * 2, t * stride * 2 + ROW) for t in range(3)]
            want = any(a < offset + 3 * ROW and b > offset for a, b in rows)
            assert refused(B, q=Q, q_out=Q + offset, q_token_stride=stride) == want, (stride, offset)
