"""tl_kv_tree_attn against the float64 oracle."""
import numpy as np
import pytest
import torch

from tests.kv_cases import Batch, check_attention, f64
from tests.test_kv_attn_gpu import LAYOUTS, Call
from oracle import kv_cache as ora

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


def tree_of(rng, n):
    """Each token's path in a random tree, itself included."""
    sees = np.zeros((n, n), bool)
    for i in range(n):
        parent = rng.integers(max(-1, i - 6), i) if i else -1
        if parent >= 0:
            sees[i] = sees[parent]
        sees[i, i] = True
    return sees


class TreeCall(Call):
    """sees: one matrix [n_s, n_s] for each sequence (None: random trees); words: of a token's mask (None: as needed)."""

    def __init__(self, B, b, *, sees=None, words=None, noise=True, **kw):
        super().__init__(B, b, **kw)
        self.sees = sees or [tree_of(b.rng, n) for n in b.q]
        self.words = words or max(1, -(-max(b.q) // 32))
        bits = np.zeros((b.n, self.words * 32), bool)
        for s, m in enumerate(self.sees):
            n = min(b.q[s], self.words * 32)
            bits[b.cu[s]:b.cu[s + 1], :n] = m[:, :n]
            if noise:  # bits of tokens that do not exist are not looked at
                bits[b.cu[s]:b.cu[s + 1], n:] = b.rng.random((b.q[s], self.words * 32 - n)) < 0.5
        self.tree = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).cuda()

    def run(self, stream=None):
        b = self.b
        self.out = torch.full((b.n, b.H, b.D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((b.H, b.n), 7.0, dtype=torch.float32, device="cuda")
        self.B.tl_kv_tree_attn(self.dq, self.cache, self.out, *self.args, self.tree, self.ws, self.sig, scale=self.scale,
                               max_q_len=self.max_q_len, lse=self.lse, stream=stream)
        return self

    def expected(self):
        b, scale = self.b, self.scale or self.b.D ** -0.5
        out, lse = np.zeros((b.n, b.H, b.D)), np.full((b.H, b.n), -np.inf)
        vmax, smax = np.zeros((b.n, b.H, 1)), np.zeros((b.n, b.H, 1))
        q = f64(self.q)
        for s, sees in enumerate(self.sees):
            if b.q[s] == 0:
                continue
            rows = slice(b.cu[s], b.cu[s + 1])
            k, v = ora.values(self.kc, self.ks, b.table[s], b.lens[s]), ora.values(self.vc, self.vs, b.table[s], b.lens[s])
            sees = sees & (np.arange(b.q[s]) < 32 * self.words)
            out[rows], lse[:, rows] = ora.tree_attention(q[rows], k, v, sees, scale)
            kk, vv = (np.abs(np.nan_to_num(x)).repeat(b.H // b.Hkv, 1) for x in (k, v))
            vmax[rows] = vv.max((0, 2))[None, :, None]
            smax[rows] = scale * np.einsum("thd,jhd->thj", np.abs(q[rows]), kk).max(2)[:, :, None]
        return out, lse, vmax, smax

    def check(self):
        assert self.B.tl_query_status(self.sig)[0] == 0
        check_attention(f64(self.out), f64(self.lse), *self.expected())
        return self


# Few rows of a kv head and many: 32 rows in batches of eight sequences or more, 64 in smaller ones, lie between two kernels.
@pytest.mark.parametrize("layout", LAYOUTS)
def test_ragged_trees(B, layout):
    b = Batch([4, 0, 1, 9, 33, 64, 0, 3], [100, 50, 1, 9, 47, 64, 0, 700], seed=31, **layout)
    TreeCall(B, b).run().check()
    b = Batch([26, 7, 3], [300, 70, 3], seed=32, **layout)
    TreeCall(B, b).run().check()


@pytest.mark.parametrize("q_len", [1, 5, 31, 32, 33, 65, 130])
@pytest.mark.parametrize("D,group", [(128, 4), (64, 1), (64, 8)])
def test_windows_of_bits_meet_tiles_anywhere(B, q_len, D, group):
    """The first new token at every place of a 64-token tile's two windows."""
    lens = [q_len + c for c in (0, 1, 15, 31, 32, 33, 47, 63, 64, 65, 100)]
    b = Batch([q_len] * len(lens), lens, H=2 * group, Hkv=2, D=D, ps=16, seed=33)
    TreeCall(B, b, max_q_len=q_len).run().check()


@pytest.mark.parametrize("q_len", [6, 80])
def test_any_masks(B, q_len):
    """Not a tree: tokens that see later ones, not themselves, nothing new, and (with no context) nothing at all."""
    rng = np.random.default_rng(34)
    b = Batch([q_len] * 4, [q_len, q_len + 50, q_len, 200], seed=34, **LAYOUTS[0])
    sees = [rng.random((q_len, q_len)) < 0.4 for _ in range(4)]
    sees[0][[1, q_len - 1]] = False
    sees[1][2] = False
    sees[2][:] = False
    c = TreeCall(B, b, sees=sees).run().check()
    empty = [1, q_len - 1] + list(range(2 * q_len, 3 * q_len))
    assert (c.out[empty] == 0).all() and torch.isneginf(c.lse[:, empty]).all()


@pytest.mark.parametrize("words,q_len", [(1, 50), (2, 64), (5, 20), (256, 40)])
def test_more_and_fewer_words_than_tokens(B, words, q_len):
    b = Batch([q_len, 3], [q_len + 70, 30], seed=35, **LAYOUTS[0])
    TreeCall(B, b, words=words).run().check()


@pytest.mark.parametrize("q", [[5, 3, 1], [40, 70, 2]])
def test_a_chain_is_the_causal_call(B, q):
    """Masks of a chain are the causal limits: the plain call's result, to its own bounds."""
    b = Batch(q, [n + 80 for n in q], seed=36, **LAYOUTS[0])
    c = TreeCall(B, b, sees=[np.tri(n, dtype=bool) for n in q]).run().check()
    tree_out, tree_lse = c.out.clone(), c.lse.clone()
    Call.run(c)
    check_attention(f64(tree_out), f64(tree_lse), *c.expected())
    Call.check(c)


@pytest.mark.parametrize("order", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("q", [[3, 2, 4], [60, 1, 33]])
def test_orders_and_strides(B, order, q):
    b = Batch(q, [99, 300, 64], seed=37, order=order, extra_columns=3, **LAYOUTS[0])
    TreeCall(B, b, strided=True, scale=0.2).run().check()


@pytest.mark.parametrize("q_len", [4, 24, 150])
@pytest.mark.parametrize("layout", LAYOUTS[:2])
def test_nan_reaches_those_that_see_it_and_no_others(B, q_len, layout):
    def edit(c):
        b = c.b
        for s, i, d in ((0, 1, 3), (0, 3, 60), (1, 2, 3), (2, 0, 5)):  # values of new tokens
            pos = b.lens[s] - q_len + i
            c.vc[b.table[s, pos // b.ps], :, pos % b.ps, d] = 127
        pos = b.lens[1] - q_len + 1  # a key of one
        c.kc[b.table[1, pos // b.ps], 0, pos % b.ps, 7] = 255
        pos = b.lens[3] - q_len - 1  # a value of the last token before: all see it
        c.vc[b.table[3, pos // b.ps], :, pos % b.ps, 9] = 255
        for s, n in enumerate(b.lens):  # slots past the end
            if n % b.ps:
                c.vc[b.table[s, n // b.ps], :, n % b.ps:] = 127
    b = Batch([q_len] * 4, [q_len + 40, q_len + 21, q_len, q_len + 2], seed=38, **layout)
    c = TreeCall(B, b, edit=edit, noise=False).run()
    assert B.tl_query_status(c.sig)[0] == 0
    want, lse, vmax, smax = c.expected()
    # the oracle's sum lets a NaN of one dim reach that dim only
    got = f64(c.out)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.isnan(got).any() and not np.isnan(got).all()
    check_attention(got, f64(c.lse), want, lse, vmax, smax)


@pytest.mark.parametrize("q_len", [3, 60])
def test_scale_byte_255_behind_the_context(B, q_len):
    """A page of NaN that holds the last new tokens alone: rows that see none of them keep their result."""
    def edit(c):
        b = c.b
        c.vs[b.table[0, (b.lens[0] - 1) // b.ps]] = 255
    ps = 16
    b = Batch([q_len, 1], [ps * 6 + 1, 9], H=4, Hkv=2, D=128, ps=ps, seed=39)  # the last token has a page of its own
    sees = [np.tri(q_len, dtype=bool), np.ones((1, 1), bool)]
    c = TreeCall(B, b, edit=edit, sees=sees).run()
    got = f64(c.out)
    assert np.isnan(got[q_len - 1]).all() and not np.isnan(got[:q_len - 1]).any() and not np.isnan(got[q_len]).any()
    want, lse, vmax, smax = c.expected()
    check_attention(got, f64(c.lse), want, lse, vmax, smax)


@pytest.mark.parametrize("q_len", [5, 60])
def test_scales_far_apart(B, q_len):
    def edit(c):
        c.ks[:] = c.b.rng.integers(95, 125, c.ks.shape)
        c.vs[:] = c.b.rng.integers(90, 150, c.vs.shape)
    b = Batch([q_len] * 3, [300, 140, q_len], seed=40, **LAYOUTS[0])
    c = TreeCall(B, b, edit=edit).run()
    assert B.tl_query_status(c.sig)[0] == 0
    # values of any magnitude: the bound's vmax is that of all a sequence's values, which the largest scale sets
    check_attention(f64(c.out), f64(c.lse), *c.expected())


@pytest.mark.parametrize("q_len", [5, 60])
def test_scores_of_great_spread(B, q_len):
    TreeCall(B, Batch([q_len] * 2, [900, 300], seed=41, **LAYOUTS[0]), q_scale=200.0).run().check()


@pytest.mark.parametrize("q", [[2, 5, 1, 3], [7, 40, 26, 130]])
def test_same_bits_again_on_a_stream_and_in_a_graph(B, q):
    c = TreeCall(B, Batch(q, [500, 70, 1300, 131], seed=42, **LAYOUTS[0])).run().check()
    first = c.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    side.synchronize()
    assert torch.equal(c.out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(3):
        c.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first)


def test_one_workspace_for_both_calls(B):
    calls = [TreeCall(B, Batch(q, n, seed=43, **LAYOUTS[i])) for i, q, n in
             ((0, [1, 4], [900, 30]), (1, [200, 3], [500, 400]), (0, [60], [1500]), (4, [2] * 9, [77] * 9))]
    ws = max((c.ws for c in calls), key=lambda w: w.numel()).clone()
    for c in calls + calls[::-1]:
        c.ws = ws
        c.run().check()
        Call.run(c)
        Call.check(c)


@pytest.mark.parametrize("q_len", [2, 100])
@pytest.mark.parametrize("what", ["page", "length", "cu"])
def test_bad_batches_are_reported_and_stay_inside(B, what, q_len):
    b = Batch([q_len] * 3, [130, 140, 190], seed=44, **LAYOUTS[0])
    c = TreeCall(B, b)
    cu, lens, table = c.args
    if what == "page":
        table[1, 1] = b.pages
    elif what == "length":
        lens[1] = 1  # below the new tokens
    else:
        cu[2] = 100000
    c.run()
    code, where = B.tl_query_status(c.sig)
    assert code == B.TL_ERR_INVALID and where in (1, 2)
    want, lse, vmax, smax = c.expected()
    rows = slice(0, q_len)
    check_attention(f64(c.out)[rows], f64(c.lse)[:, rows], want[rows], lse[:, rows], vmax[rows], smax[rows])
    c.args = b.device()
    c.run().check()


def test_binding_refuses_wrong_trees(B):
    b = Batch([2, 1], [30, 5], seed=45, **LAYOUTS[0])
    c = TreeCall(B, b)
    good = c.tree
    for bad in (good.long(), good.cpu(), good[:2], good.repeat(1, 2)[:, ::2]):
        c.tree = bad
        with pytest.raises(ValueError):
            c.run()
    c.tree = torch.zeros(b.n, 257, dtype=torch.int32, device="cuda")
    with pytest.raises(B.TLError):
        c.run()
    c.tree = good
    c.run().check()


# ------------------------------------------------------------------ the kernel for many rows
def by_many(b):
    """The rule by which the call's kernels share the sequences, on 152 SMs: whether those of many rows go to the one for many."""
    least = 32 if len(b.q) >= 8 else 64
    units = tiles = few = 0
    for q, n in zip(b.q, b.lens):
        rows = q * (b.H // b.Hkv)
        if rows > least:
            u = -(-rows // 256) * b.Hkv
            units, tiles = units + u, tiles + u * max(1, -(-n // 64))
            few += -(-rows // 16) * b.Hkv * (-(-n // 32) + 24)
    if not units:
        return False
    runs = min(152, max(units, tiles // 8))
    join = 0 if runs == units else 8000 + 2200 * runs // units
    return (950 * tiles + 8000 * units) // 152 + join + 20000 < 210 * few // 152 + 8000


MANY = dict(H=32, Hkv=8, D=128, ps=64)


@pytest.mark.parametrize("q,lens,layout", [
    ([64] * 8, [64, 65, 127, 128, 129, 400, 500, 300], MANY),                      # two tiles of rows
    ([64, 3, 40, 1, 0, 64, 33, 64, 64, 50], [164, 70, 300, 90, 10, 64, 200, 401, 90, 51], MANY),   # few and many, one tile and two
    ([31, 30, 64, 20] * 3, [131, 95, 164, 200] * 3, dict(H=24, Hkv=8, D=64, ps=16)),
    ([100] * 4, [900, 350, 100, 612], dict(H=40, Hkv=8, D=128, ps=128)),           # three units to a sequence, the last part-filled
    ([128], [9000], MANY)])
def test_ragged_trees_of_many_rows(B, q, lens, layout):
    b = Batch(q, lens, seed=51, extra_columns=600, **layout)
    assert by_many(b)
    TreeCall(B, b).run().check()


def test_any_masks_of_many_rows(B):
    rng = np.random.default_rng(52)
    b = Batch([64] * 8, [64, 100, 64, 300, 64, 65, 190, 400], seed=52, extra_columns=100, **MANY)
    assert by_many(b)
    sees = [rng.random((64, 64)) < 0.4 for _ in range(8)]
    sees[0][[1, 63]] = False
    sees[1][2] = False
    sees[2][:] = False
    c = TreeCall(B, b, sees=sees, words=3).run().check()
    empty = [1, 63] + list(range(128, 192))
    assert (c.out[empty] == 0).all() and torch.isneginf(c.lse[:, empty]).all()


@pytest.mark.parametrize("D,group", [(128, 4), (64, 8)])
def test_nan_in_trees_of_many_rows(B, D, group):
    n = 64
    def edit(c):
        b = c.b
        for s, i, d in ((0, 1, 3), (0, 3, 60), (1, 2, 3), (2, 0, 5), (3, 63, 50)):
            pos = b.lens[s] - n + i
            c.vc[b.table[s, pos // b.ps], :, pos % b.ps, d] = 127
        pos = b.lens[1] - n + 1
        c.kc[b.table[1, pos // b.ps], 0, pos % b.ps, 7] = 255
        pos = b.lens[4] - n - 1
        c.vc[b.table[4, pos // b.ps], :, pos % b.ps, 9] = 255
        c.vs[b.table[5, (b.lens[5] - 1) // b.ps], 2] = 255  # one head's last page, which holds its last new token alone
        for s, m in enumerate(b.lens):
            if m % b.ps:
                c.vc[b.table[s, m // b.ps], :, m % b.ps:] = 127
    b = Batch([n] * 8, [n + 40, n + 21, n, n + 70, n + 2, 16 * 9 + 1, n + 200, n + 90], H=8 * group, Hkv=8, D=D, ps=16, seed=53,
              extra_columns=100)
    assert by_many(b)
    c = TreeCall(B, b, edit=edit, noise=False).run()
    assert B.tl_query_status(c.sig)[0] == 0
    want, lse, vmax, smax = c.expected()
    got = f64(c.out)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got).any() and not np.isnan(got).all()
    check_attention(got, f64(c.lse), want, lse, vmax, smax)


@pytest.mark.parametrize("spread", [8, 25])
def test_scales_far_apart_in_trees_of_many_rows(B, spread):
    def edit(c):
        c.ks[:] = c.b.rng.integers(110 - spread // 2, 110 + spread // 2, c.ks.shape)
        c.vs[:] = c.b.rng.integers(120 - spread, 120 + spread, c.vs.shape)
    b = Batch([64, 30] * 4, [300, 140, 64, 95] * 2, seed=54, extra_columns=100, **MANY)
    assert by_many(b)
    c = TreeCall(B, b, edit=edit).run()
    assert B.tl_query_status(c.sig)[0] == 0
    check_attention(f64(c.out), f64(c.lse), *c.expected())


def test_great_scores_in_trees_of_many_rows(B):
    b = Batch([64] * 8, [300] * 8, seed=55, extra_columns=100, **MANY)
    assert by_many(b)
    TreeCall(B, b, q_scale=200.0).run().check()


def test_trees_of_many_rows_again_and_captured(B):
    b = Batch([64, 40, 64, 64, 7, 64, 64, 33, 64], [500, 70, 1300, 131, 90, 64, 300, 200, 400], seed=56, extra_columns=50, **MANY)
    assert by_many(b)
    c = TreeCall(B, b).run().check()
    first = c.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(3):
        c.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first)
    b2 = Batch([2, 64], [60, 80], seed=57, **LAYOUTS[0])
    d = TreeCall(B, b2)
    d.ws = c.ws if c.ws.numel() >= d.ws.numel() else d.ws
    d.run().check()
    c.run()
    assert torch.equal(c.out, first)
