"""tl_kv_fork, tl_kv_resize, tl_kv_copy_pages and tl_kv_compact against the oracle: every entry and every code."""
import numpy as np
import pytest
import torch

from tests.kv_cases import Batch
from oracle import kv_cache as ora
from oracle import kv_pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Tables:
    """Sequences with their pages in a pool; some full pages shared by neighbours, part-filled ones by nobody."""

    def __init__(self, lens, ps, *, seed, spare=20, share=0.5, columns=2):
        r = self.rng = np.random.default_rng(seed)
        self.lens, self.ps = np.array(lens, np.int32), ps
        need = [-(-n // ps) for n in lens]
        self.pages = sum(need) + spare
        deal, at = list(r.permutation(self.pages)), 0
        self.table = np.full((len(lens), max(need + [1]) + columns), -7, np.int32)
        for s, k in enumerate(need):
            full = lens[s] // ps
            common = min(full, lens[s - 1] // ps, int(r.integers(0, full + 1))) if s and r.random() < share else 0
            self.table[s, :common] = self.table[s - 1, :common]
            self.table[s, common:k] = deal[at:at + k - common]
            at += k - common
        self.refs = np.zeros(self.pages, np.int32)
        for row, k in zip(self.table, need):
            np.add.at(self.refs, row[:k], 1)
        assert (self.refs == 0).sum() >= spare


def fork(B, t, parents, *, in_place=False, times=1):
    """The call's results as arrays, and its status."""
    n, pages = len(parents), t.pages
    table_out, lens_out = np.full((n, t.table.shape[1]), -9, np.int32), np.full(n, -9, np.int32)
    refs = i32(t.refs)
    refs_out = refs if in_place else i32(np.full(pages, -9))
    d = [i32(t.table), i32(t.lens), refs, i32(parents), i32(table_out), i32(lens_out), refs_out,
         i32(np.full((3, n), -9)), i32([-9])]
    ws = torch.full((B.tl_kv_fork_workspace_size(len(t.lens), n),), 171, dtype=torch.uint8, device="cuda")
    sig = B.Signals(1)
    for _ in range(times):
        B.tl_kv_fork(*d, ws, sig, page_size=t.ps)
    status = B.tl_query_status(sig)
    return [x.cpu().numpy() for x in d[4:]], status, table_out


def check_fork(B, t, parents, **kw):
    got, status, before = fork(B, t, parents, **kw)
    table, lens, refs, copies = kv_pages.fork(t.table, t.lens, t.refs, parents, t.ps, before)
    assert status[0] == 0
    assert np.array_equal(got[0], table) and np.array_equal(got[1], lens) and np.array_equal(got[2], refs)
    assert got[4][0] == len(copies) and [tuple(c) for c in got[3].T[:len(copies)]] == copies
    return copies


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ps", [16, 64, 256])
@pytest.mark.parametrize("rows", [1, 5, 64])
def test_fork(B, ps, rows, in_place):
    r = np.random.default_rng(rows)
    lens = [int(r.integers(0, 700)) for _ in range(rows)]
    lens[0] = 3 * ps  # a sequence that ends with a page
    t = Tables(lens, ps, seed=rows + ps, spare=2 * rows + 3)
    check_fork(B, t, r.integers(-1, rows, rows), in_place=in_place)
    check_fork(B, t, r.integers(-1, rows, 2 * rows + 1), in_place=in_place)
    check_fork(B, t, np.zeros(rows, int), in_place=in_place)       # one goes on in all
    check_fork(B, t, np.arange(rows), in_place=in_place)           # nothing changes
    check_fork(B, t, np.full(3, -1), in_place=in_place)            # nothing is left


def test_fork_of_more_rows_than_threads(B):
    r = np.random.default_rng(3)
    t = Tables([int(x) for x in r.integers(0, 100, 1500)], 16, seed=3, spare=40000)
    check_fork(B, t, r.integers(-1, 1500, 2500))


def test_fork_takes_the_lowest_free_pages_of_a_large_pool(B):
    t = Tables([100, 37, 64, 5], 16, seed=4, spare=70003, share=0.0)
    free = np.flatnonzero(t.refs == 0)
    t.refs[free[:-4]] = 1  # held by others: the four free ones are scattered at the end
    assert len(check_fork(B, t, np.array([0, 0, 1, 3, 1, 3]))) == 3


def test_fork_copies_a_page_that_others_hold(B):
    t = Tables([40, 20], 16, seed=5, share=0.0)
    t.refs[t.table[0, 2]] += 1
    assert check_fork(B, t, np.array([0, 1])) == [(t.table[0, 2], int(np.flatnonzero(t.refs == 0)[0]), 8)]


@pytest.mark.parametrize("in_place", [False, True])
def test_fork_without_pages_changes_nothing(B, in_place):
    t = Tables([40, 20, 8], 16, seed=6, spare=1)
    t.refs[t.refs == 0] = 1
    t.refs[3] = t.refs[3] if (t.table == 3).any() else 0
    free = int((t.refs == 0).sum())
    got, status, before = fork(B, t, np.array([0, 0, 1, 1, 2, 2]), in_place=in_place)
    assert status == (B.TL_ERR_INVALID, 3 - free)
    assert np.array_equal(got[0], before) and (got[1] == -9).all() and np.array_equal(got[2], t.refs) and got[4][0] == 0


def test_fork_reports_wrong_data_and_stays_inside(B):
    def other_rows(t, got, parents, bad):
        for o, b in enumerate(parents):
            if 0 <= b < len(t.lens) and b != bad:
                n = -(-t.lens[b] // t.ps)
                assert np.array_equal(got[0][o, :t.lens[b] // t.ps], t.table[b, :t.lens[b] // t.ps]) and got[1][o] == t.lens[b] and n >= 0
    parents = np.array([0, 1, 2, 2, 0])
    t = Tables([70, 33, 90], 16, seed=7)
    bad = parents.copy()
    bad[1] = 3
    got, status, _ = fork(B, t, bad)
    assert status == (B.TL_ERR_INVALID, 1) and got[1][1] == 0
    other_rows(t, got, bad, None)
    for what in ("page", "length", "negative length"):
        t = Tables([70, 33, 90], 16, seed=7)
        if what == "page":
            t.table[1, :] = t.pages
        else:
            t.lens = t.lens.copy()
            t.lens[1] = 10 ** 6 if what == "length" else -4
        got, status, _ = fork(B, t, parents)
        assert status == (B.TL_ERR_INVALID, 1), what
        other_rows(t, got, parents, 1)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ps,rows", [(16, 1), (64, 9), (32, 1300)])
def test_resize(B, ps, rows, in_place):
    r = np.random.default_rng(rows)
    lens = [int(x) for x in r.integers(0, 300, rows)]
    t = Tables(lens, ps, seed=rows, spare=rows * (-(-300 // ps) + 1), columns=12)
    new = np.where(r.random(rows) < 0.3, 0, r.integers(0, 300, rows)).astype(np.int32)
    new[0] = lens[0] + 1
    refs = i32(t.refs)
    refs_out = refs if in_place else i32(np.full(t.pages, -9))
    d, ws, sig = i32(t.table), torch.full((B.tl_kv_resize_workspace_size(rows),), 99, dtype=torch.uint8, device="cuda"), B.Signals(1)
    B.tl_kv_resize(d, i32(t.lens), i32(new), refs, refs_out, ws, sig, page_size=ps)
    assert B.tl_query_status(sig)[0] == 0
    table, want = kv_pages.resize(t.table, t.lens, new, t.refs, ps)
    assert np.array_equal(d.cpu().numpy(), table) and np.array_equal(refs_out.cpu().numpy(), want)


def test_resize_without_pages_and_with_wrong_lengths(B):
    t = Tables([40, 20, 8], 16, seed=8, spare=2, columns=8)
    ws, sig = torch.zeros(B.tl_kv_resize_workspace_size(3), dtype=torch.uint8, device="cuda"), B.Signals(1)
    d, out = i32(t.table), i32(np.full(t.pages, -9))
    free = int((t.refs == 0).sum())
    B.tl_kv_resize(d, i32(t.lens), i32([160, 20, 100]), i32(t.refs), out, ws, sig, page_size=16)
    assert B.tl_query_status(sig) == (B.TL_ERR_INVALID, 7 + 6 - free)
    assert np.array_equal(out.cpu().numpy(), t.refs)
    held = [-(-n // 16) for n in t.lens]
    assert all(np.array_equal(a[:k], b[:k]) for a, b, k in zip(d.cpu().numpy(), t.table, held))
    for wrong in (-1, 10 ** 7):
        B.tl_kv_resize(d, i32(t.lens), i32([0, wrong, 8]), i32(t.refs), out, ws, sig, page_size=16)
        assert B.tl_query_status(sig) == (B.TL_ERR_INVALID, 1)
        assert np.array_equal(out.cpu().numpy(), kv_pages.resize(t.table, t.lens, [0, 20, 8], t.refs, 16)[1])


class Pools:
    """Layers' caches on both sides."""

    def __init__(self, B, pages, Hkv, ps, D, layers, *, seed, order="hnd", spread=6):
        r = self.rng = np.random.default_rng(seed)
        shape = (layers, 2, pages, Hkv, ps, D)
        self.codes = r.integers(0, 256, shape).astype(np.uint8)
        self.codes[(self.codes & 127) == 127] = 3
        self.scales = r.integers(127 - spread, 128 + spread, shape[:4]).astype(np.uint8)
        t = torch.from_numpy(self.codes)
        if order == "nhd":
            t = t.transpose(3, 4).contiguous().cuda().transpose(3, 4)
        elif order == "kv":  # keys and values of a page next to one another
            t = t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        self.d, self.ds = t.cuda(), torch.from_numpy(self.scales).cuda()
        self.B = B
        self.layers = B.KvLayers([B.KvCache(self.d[l, 0], self.d[l, 1], self.ds[l, 0], self.ds[l, 1]) for l in range(layers)])

    def check(self, f):
        """f(codes, scales) for each layer's keys and values; codes by the values they stand for."""
        got, scales = self.d.cpu().numpy(), self.ds.cpu().numpy()
        for l in range(len(got)):
            for x in range(2):
                c, s = f(self.codes[l, x], self.scales[l, x])[:2]
                assert np.array_equal(scales[l, x], s), (l, x)
                assert np.array_equal(ora.TABLE[got[l, x]], ora.TABLE[c], equal_nan=True), (l, x)


@pytest.mark.parametrize("order", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("Hkv,ps,D,layers", [(2, 16, 64, 1), (8, 64, 128, 3), (1, 256, 128, 2), (3, 48, 64, 70)])
def test_copy_pages(B, Hkv, ps, D, layers, order):
    p = Pools(B, 12, Hkv, ps, D, layers, seed=9, order=order)
    src, dst, slots = [0, 5, 5, 7, 3, 9], [1, 2, 4, 7, 11, 10], [ps, 1, 0, 3, ps - 1, 7]
    sig = B.Signals(1)
    B.tl_kv_copy_pages(p.layers, i32(src), i32(dst), sig, slots=i32(slots), count=i32([5]))
    assert B.tl_query_status(sig)[0] == 0
    p.check(lambda c, s: kv_pages.copy_pages(c, s, list(zip(src, dst, slots))[:5]))
    p = Pools(B, 12, Hkv, ps, D, layers, seed=10, order=order)
    B.tl_kv_copy_pages(p.layers, i32(src), i32(dst), sig)
    p.check(lambda c, s: kv_pages.copy_pages(c, s, [(a, b, ps) for a, b in zip(src, dst)]))
    assert B.tl_query_status(sig)[0] == 0


def test_copy_pages_leaves_wrong_copies_out(B):
    p = Pools(B, 6, 2, 16, 64, 2, seed=11)
    sig = B.Signals(1)
    for i, (src, dst, slots) in enumerate([(6, 1, 3), (0, -1, 3), (0, 1, 17), (0, 1, -1)]):
        B.tl_kv_copy_pages(p.layers, i32([2, src]), i32([3, dst]), sig, slots=i32([16, slots]))
        assert B.tl_query_status(sig) == (B.TL_ERR_INVALID, 1), i
    p.check(lambda c, s: kv_pages.copy_pages(c, s, [(2, 3, 16)]))
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    B.tl_kv_copy_pages(p.layers, empty, empty, sig)
    B.tl_kv_copy_pages(p.layers, i32([0]), i32([5]), sig, count=i32([0]))
    B.tl_kv_copy_pages(p.layers, i32([0]), i32([5]), sig, count=i32([-3]))
    p.check(lambda c, s: kv_pages.copy_pages(c, s, [(2, 3, 16)]))


def compact_case(B, b, kept, layers, *, seed, order="hnd", spread=6, edit=None):
    p = Pools(B, b.pages, b.Hkv, b.ps, b.D, layers, seed=seed, order=order, spread=spread)
    if edit:
        edit(p)
        p.d.copy_(torch.from_numpy(p.codes))
        p.ds.copy_(torch.from_numpy(p.scales))
    rows = np.zeros((len(kept), max(map(len, kept)) + 2), np.int32)
    for s, path in enumerate(kept):
        rows[s, :len(path)] = path
    cu, lens, table = b.device()
    out, sig = i32(np.full(len(kept), -9)), B.Signals(1)
    call = lambda: B.tl_kv_compact(p.layers, i32(rows), i32([len(x) for x in kept]), cu, lens, table, out, sig)
    return p, call, out, sig


@pytest.mark.parametrize("order", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("Hkv,ps,D,layers", [(2, 16, 64, 1), (8, 64, 128, 2), (1, 48, 128, 3), (5, 16, 128, 66)])
def test_compact(B, Hkv, ps, D, layers, order):
    r = np.random.default_rng(12)
    q = [1, 0, 26, 64, 7, 100, 40, 33, 5]
    lens = [n + int(r.integers(0, 90)) for n in q]
    lens[2] = q[2] + 2 * ps  # new tokens begin a page
    b = Batch(q, lens, H=Hkv, Hkv=Hkv, D=D, ps=ps, seed=13)
    kept = [sorted(r.choice(n, int(r.integers(0, n + 1)), replace=False).tolist()) for n in q]
    kept[5], kept[6], kept[7] = list(range(100)), list(range(3, 40)), [32]  # all, all but the first, the last alone
    p, call, out, sig = compact_case(B, b, kept, layers, seed=14, order=order)
    call()
    assert B.tl_query_status(sig)[0] == 0
    want = lambda c, s: kv_pages.compact(c, s, kept, b.cu, b.lens, b.table)
    p.check(want)
    assert np.array_equal(out.cpu().numpy(), want(p.codes[0, 0], p.scales[0, 0])[2])


def test_compact_of_scales_far_apart_and_nan(B):
    def edit(p):
        p.scales[..., ::3] = 60
        p.scales[..., 1::5] = 200
        p.scales[0, 1, b.table[1, 3]] = 255
        p.codes[:, :, b.table[0, 1], 0, 3, 5] = 127
    b = Batch([40, 50], [60, 90], H=3, Hkv=3, D=64, ps=16, seed=15)
    kept = [[0, 3, 7, 8, 20, 39], [1, 2, 5, 22, 30, 31, 32, 49]]
    p, call, out, sig = compact_case(B, b, kept, 2, seed=16, edit=edit)
    call()
    assert B.tl_query_status(sig)[0] == 0
    p.check(lambda c, s: kv_pages.compact(c, s, kept, b.cu, b.lens, b.table))


@pytest.mark.parametrize("what", [[3, 3], [5, 2], [-1, 4], [0, 40], "many", "few columns", "negative"])
def test_compact_leaves_a_sequence_of_wrong_drafts_as_it_is(B, what):
    b = Batch([30, 40, 20], [60, 90, 20], H=2, Hkv=2, D=64, ps=16, seed=17)
    kept = [[2, 5, 9], [1, 7], [0, 19]]
    p, _, out, sig = compact_case(B, b, kept, 2, seed=18)
    rows = np.zeros((3, 3), np.int32)
    for s, path in enumerate(kept):
        rows[s, :len(path)] = path
    n = np.array([3, 2, 2], np.int32)
    if what == "many":
        rows = np.tile(np.arange(60, dtype=np.int32), (3, 1))
        n = np.array([30, 41, 2], np.int32)
        kept = [list(range(30)), [], [0, 1]]
    elif what == "few columns":
        n[1] = 4
    elif what == "negative":
        n[1] = -1
    else:
        rows[1, :2] = what
    cu, lens, table = b.device()
    B.tl_kv_compact(p.layers, i32(rows), i32(n), cu, lens, table, out, sig)
    assert B.tl_query_status(sig) == (B.TL_ERR_INVALID, 1)
    others = [kept[0], list(range(40)), kept[2]]  # all of its own: as it is
    want = lambda c, s: kv_pages.compact(c, s, others, b.cu, b.lens, b.table)
    def as_it_is(c, s):
        w = want(c, s)
        return w
    got, scales = p.d.cpu().numpy(), p.ds.cpu().numpy()
    mine = b.table[1, :-(-b.lens[1] // b.ps)]
    assert np.array_equal(got[:, :, mine], p.codes[:, :, mine]) and np.array_equal(scales[:, :, mine], p.scales[:, :, mine])
    for l in range(2):
        for x in range(2):
            c, s, n_out = as_it_is(p.codes[l, x], p.scales[l, x])
            rest = np.setdiff1d(np.arange(b.pages), mine)
            assert np.array_equal(scales[l, x][rest], s[rest]) and np.array_equal(ora.TABLE[got[l, x][rest]], ora.TABLE[c[rest]])
    assert np.array_equal(out.cpu().numpy(), n_out)


def test_compact_bad_batches_stay_inside(B):
    b = Batch([30, 40, 20], [60, 90, 20], H=2, Hkv=2, D=64, ps=16, seed=19)
    kept = [[2, 5, 9], [1, 7], [0, 19]]
    for what in ("page", "length", "cu"):
        p, _, out, sig = compact_case(B, b, kept, 1, seed=20)
        cu, lens, table = b.device()
        if what == "page":
            table[1, 3:] = b.pages
        elif what == "length":
            lens[1] = 10
        else:
            cu[2] = -5
        rows = np.array([[2, 5, 9], [1, 7, 0], [0, 19, 0]], np.int32)
        B.tl_kv_compact(p.layers, i32(rows), i32([3, 2, 2]), cu, lens, table, out, sig)
        code, where = B.tl_query_status(sig)
        assert code == B.TL_ERR_INVALID and where in (1, 2)
        c, s, n = kv_pages.compact(p.codes[0, 0], p.scales[0, 0], kept, b.cu, b.lens, b.table)
        mine = b.table[0, :4]
        assert np.array_equal(ora.TABLE[p.d.cpu().numpy()[0, 0][mine]], ora.TABLE[c[mine]]) and out[0].item() == n[0]


def test_a_captured_step_of_beams(B):
    """Grow, fork in place of tables in turn, copy, shrink: captured once, replayed, the same as call by call."""
    ps, rows, layers = 16, 6, 2
    t = Tables([20, 33, 16, 47, 5, 64], ps, seed=21, spare=60, columns=10)
    r = np.random.default_rng(22)
    parents = [r.integers(-1, rows, rows) for _ in range(4)]
    p = Pools(B, t.pages, 2, ps, 64, layers, seed=23)
    table, lens, refs = i32(t.table), i32(t.lens), i32(t.refs)
    table2, lens2 = i32(np.full(t.table.shape, -7)), i32(np.zeros(rows))
    more, chosen, copies, count = i32(np.zeros(rows)), i32(parents[0]), i32(np.zeros((3, rows))), i32([0])
    ws = torch.zeros(B.tl_kv_fork_workspace_size(rows, rows), dtype=torch.uint8, device="cuda")
    sig = B.Signals(1)

    def step():
        torch.add(lens, 3, out=more)
        B.tl_kv_resize(table, lens, more, refs, refs, ws, sig, page_size=ps)
        B.tl_kv_fork(table, more, refs, chosen, table2, lens2, refs, copies, count, ws, sig, page_size=ps)
        B.tl_kv_copy_pages(p.layers, copies[0], copies[1], sig, slots=copies[2], count=count)
        table.copy_(table2)
        lens.copy_(lens2)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    w_table, w_lens, w_refs, pools = t.table, t.lens, t.refs, (p.codes, p.scales)
    for chosen_now in parents:
        chosen.copy_(i32(chosen_now))
        graph.replay()
        grown = w_lens + 3
        w_table, w_refs = kv_pages.resize(w_table, w_lens, grown, w_refs, ps)
        out = kv_pages.fork(w_table, grown, w_refs, chosen_now, ps, np.zeros_like(w_table))
        w_lens, w_refs, done = out[1], out[2], out[3]
        torch.cuda.synchronize()
        got = table.cpu().numpy()
        for s, n in enumerate(w_lens):
            assert np.array_equal(got[s, :-(-n // ps)], out[0][s, :-(-n // ps)])
        w_table = got.copy()
        assert np.array_equal(lens.cpu().numpy(), w_lens) and np.array_equal(refs.cpu().numpy(), w_refs)
        codes, scales = pools
        codes, scales = codes.copy(), scales.copy()
        for l in range(layers):
            for x in range(2):
                codes[l, x], scales[l, x] = kv_pages.copy_pages(codes[l, x], scales[l, x], done)
        pools = codes, scales
    assert B.tl_query_status(sig)[0] == 0
    assert np.array_equal(p.d.cpu().numpy(), pools[0]) and np.array_equal(p.ds.cpu().numpy(), pools[1])


def test_offsets_past_32_bits(B):
    """A pool of more than 4 GiB: pages at its far end."""
    D, ps = 128, 256
    pages = (1 << 32) // (D * ps) + 8
    k = torch.zeros(pages, 1, ps, D, dtype=torch.uint8, device="cuda")
    v, ks = torch.zeros_like(k), torch.zeros(2, pages, 1, dtype=torch.uint8, device="cuda")
    layers, sig = B.KvLayers([B.KvCache(k, v, ks[0], ks[1])]), B.Signals(1)
    x = torch.randint(0, 120, (ps, D), dtype=torch.uint8, device="cuda")
    k[pages - 2, 0], v[pages - 2, 0], ks[:, pages - 2] = x, x.flip(0), 120
    B.tl_kv_copy_pages(layers, i32([pages - 2]), i32([pages - 1]), sig)
    assert torch.equal(k[pages - 1, 0], x) and torch.equal(v[pages - 1, 0], x.flip(0)) and (ks[:, pages - 1] == 120).all()
    out = i32([0])
    B.tl_kv_compact(layers, i32([[3, 200]]), i32([2]), i32([0, 250]), i32([256]), i32([[pages - 1]]), out, sig)
    assert out.item() == 8 and torch.equal(k[pages - 1, 0, 6], x[9]) and torch.equal(v[pages - 1, 0, 7], x.flip(0)[206])
    assert B.tl_query_status(sig)[0] == 0


def test_binding_refuses(B):
    p = Pools(B, 4, 2, 16, 64, 2, seed=24)
    sig = B.Signals(1)
    one = i32([0])
    for bad in (dict(src=one.long()), dict(dst=one.cpu()), dict(dst=i32([0, 1])), dict(slots=i32([0, 1])), dict(count=i32([1, 2]))):
        kw = {**dict(src=one, dst=one), **bad}
        with pytest.raises(ValueError):
            B.tl_kv_copy_pages(p.layers, kw.pop("src"), kw.pop("dst"), sig, **kw)
    other = Pools(B, 5, 2, 16, 64, 1, seed=25)
    with pytest.raises(ValueError):
        B.KvLayers([p.layers.caches[0], other.layers.caches[0]])
    with pytest.raises(ValueError):
        B.KvLayers([])
    t = Tables([20, 33], 16, seed=26)
    table, lens, refs, parents = i32(t.table), i32(t.lens), i32(t.refs), i32([0, 1])
    ws = torch.zeros(B.tl_kv_fork_workspace_size(2, 2), dtype=torch.uint8, device="cuda")
    good = dict(page_table=table, seq_lens=lens, refs=refs, parents=parents, page_table_out=torch.empty_like(table),
                seq_lens_out=torch.empty_like(lens), refs_out=torch.empty_like(refs), copies=i32(np.zeros((3, 2))), n_copies=one,
                workspace=ws, signals=sig, page_size=16)
    B.tl_kv_fork(**good)
    for bad in (dict(seq_lens=lens[:1]), dict(refs_out=refs[:4]), dict(copies=i32(np.zeros((2, 2)))), dict(parents=parents.long()),
                dict(page_table_out=torch.empty_like(table)[:, :2])):
        with pytest.raises(ValueError):
            B.tl_kv_fork(**{**good, **bad})
    for bad in (dict(page_table_out=table), dict(seq_lens_out=lens), dict(workspace=ws[:64]), dict(page_size=24)):
        with pytest.raises(B.TLError):
            B.tl_kv_fork(**{**good, **bad})
    with pytest.raises(ValueError):
        B.tl_kv_resize(table, lens, lens[:1], refs, refs, ws, sig, page_size=16)
    with pytest.raises(B.TLError):
        B.tl_kv_resize(table, lens, lens, refs, refs, ws[:16], sig, page_size=16)
    assert B.tl_query_status(sig)[0] == 0
