"""tl_kv_resize and tl_kv_fork with sequences of wrong lengths, behind whose pages the rows still name live pages of others."""
import numpy as np
import pytest
import torch

from tests.test_kv_pages_gpu import Tables, fork, i32
from oracle import kv_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


def stale(lens, wrong, *, spare=30, seed=11):
    """Tables whose row `wrong` names pages of the other sequences behind its own."""
    t = Tables(lens, 16, seed=seed, spare=spare, columns=8)
    held = -(-lens[wrong] // 16)
    others = np.concatenate([row[:-(-n // 16)] for s, (row, n) in enumerate(zip(t.table, lens)) if s != wrong])
    t.table[wrong, held:] = np.resize(others, t.table.shape[1] - held)
    return t


# One block for everything, and two launches.
@pytest.mark.parametrize("rows", [5, 700])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("length", [-1, 10 ** 7, "one above"])
@pytest.mark.parametrize("new", [0, 5, 90, "full"])
def test_resize_of_a_wrong_current_length(B, rows, in_place, length, new):
    lens = [40 + s % 37 for s in range(rows)]
    wrong = rows // 2
    t = stale(lens, wrong, spare=2 * rows + 30)
    room = t.table.shape[1] * 16
    now = t.lens.copy()
    now[wrong] = room + 1 if length == "one above" else length
    to = np.array([(0, 100, 41, 20)[s % 4] for s in range(rows)], np.int32)
    to[wrong] = room if new == "full" else new
    refs = i32(t.refs)
    out = refs if in_place else i32(np.full(t.pages, -9))
    ws, sig = torch.zeros(B.tl_kv_resize_workspace_size(rows), dtype=torch.uint8, device="cuda"), B.Signals(1)
    d = i32(t.table)
    B.tl_kv_resize(d, i32(now), i32(to), refs, out, ws, sig, page_size=16)
    assert B.tl_query_status(sig) == (B.TL_ERR_INVALID, wrong)
    to[wrong] = lens[wrong]  # the others' changes alone
    table, want = kv_pages.resize(t.table, t.lens, to, t.refs, 16)
    assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(d.cpu().numpy(), table)


@pytest.mark.parametrize("rows", [5, 700])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("length", [-1, 10 ** 7, "one above"])
@pytest.mark.parametrize("children", [0, 1, 3])
def test_fork_of_a_wrong_length(B, rows, in_place, length, children):
    lens = [40 + s % 37 for s in range(rows)]
    wrong = rows // 2
    t = stale(lens, wrong, spare=rows + 30)
    true = t.lens.copy()
    t.lens[wrong] = t.table.shape[1] * 16 + 1 if length == "one above" else length
    parents = np.random.default_rng(12).integers(-1, rows, rows)
    parents[parents == wrong] = -1
    parents[1:1 + children] = wrong
    got, status, before = fork(B, t, parents, in_place=in_place)
    assert status == (B.TL_ERR_INVALID, wrong)
    true[wrong] = 0  # it gives nothing on and nothing back
    table, out, refs, copies = kv_pages.fork(t.table, true, t.refs, parents, t.ps, before)
    assert np.array_equal(got[0], table) and np.array_equal(got[1], out) and np.array_equal(got[2], refs)
    assert got[4][0] == len(copies) and [tuple(c) for c in got[3].T[:len(copies)]] == copies
