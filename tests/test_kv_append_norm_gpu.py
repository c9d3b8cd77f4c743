"""tl_kv_append_norm against the float64 oracle: the values that codes and scale bytes stand for exactly, queries to one rounding."""
import numpy as np
import pytest
import torch

from tests.kv_cases import Batch, f64, tables
from oracle import kv_cache as ora

pytestmark = pytest.mark.gpu

EPS = 1e-6
LAYOUTS = [dict(H=4, Hkv=2, D=128, ps=64), dict(H=3, Hkv=3, D=64, ps=16), dict(H=8, Hkv=1, D=128, ps=16),
           dict(H=1, Hkv=1, D=64, ps=256), dict(H=6, Hkv=2, D=128, ps=48)]


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


class Case:
    """A batch with its cache on both sides; `expected` and `check` after the calls."""

    def __init__(self, B, b, *, rot, interleaved=False, norm="qk", positions=None, eps=EPS, scale=1.0, edit=None, weights=None,
                 fused=True, max_pos=None):
        self.B, self.b, self.rot, self.interleaved, self.norm, self.eps = B, b, rot, interleaved, norm, eps
        self.kc, self.ks = b.random_codes()
        self.vc, self.vs = b.random_codes()
        rows = b.bf16(b.n, b.H + 2 * b.Hkv, b.D, scale=scale)
        if edit:
            edit(rows)
        self.rows = rows
        self.wq, self.wk = weights or (b.bf16(b.D), b.bf16(b.D))
        self.pos = np.concatenate([np.arange(n - m, n) for m, n in zip(b.q, b.lens)]).astype(np.int32)
        self.positions = None if positions is None else positions(self.pos)
        at = self.pos if self.positions is None else self.positions
        self.cos, self.sin = tables(max_pos or int(at.max(initial=0)) + 1, rot) if rot else (None, None)
        self.dk, self.dv = b.both(self.kc, self.vc)
        self.dks, self.dvs = torch.from_numpy(self.ks).cuda(), torch.from_numpy(self.vs).cuda()
        d = rows.cuda()
        q, k, v = d[:, :b.H], d[:, b.H:b.H + b.Hkv], d[:, b.H + b.Hkv:]
        self.q, self.k, self.v = (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())
        self.q_out = torch.full((b.n, b.H, b.D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.cache, self.sig, self.batch = B.KvCache(self.dk, self.dv, self.dks, self.dvs), B.Signals(1), b.device()
        up = lambda x: None if x is None else torch.from_numpy(x).cuda()
        self.kw = dict(q=self.q, q_out=self.q_out, q_weight=self.wq.cuda() if "q" in norm else None,
                       k_weight=self.wk.cuda() if "k" in norm else None, eps=eps, cos=up(self.cos), sin=up(self.sin),
                       positions=up(self.positions), interleaved=interleaved)

    def call(self, **kw):
        self.B.tl_kv_append_norm(self.cache, self.k, self.v, *self.batch, self.sig, **{**self.kw, **kw})

    def expected(self):
        b, x = self.b, f64(self.rows)
        q, k, v = x[:, :b.H], x[:, b.H:b.H + b.Hkv], x[:, b.H + b.Hkv:]
        if "q" in self.norm:
            q = ora.normed(q, f64(self.wq), self.eps)
        if "k" in self.norm:
            k = ora.normed(k, f64(self.wk), self.eps)
        self.q_large = np.abs(np.nan_to_num(q, posinf=0, neginf=0)).max(2, keepdims=True, initial=0.0)
        if self.rot:
            at = self.pos if self.positions is None else self.positions
            with np.errstate(invalid="ignore"):
                qk = [ora.rotate(np.concatenate([q[t], k[t]]), p, self.cos, self.sin, self.interleaved) for t, p in enumerate(at)]
            q, k = np.stack(qk)[:, :b.H], np.stack(qk)[:, b.H:]
        return q, ora.append(self.kc, self.ks, k, b.cu, b.lens, b.table) + ora.append(self.vc, self.vs, v, b.cu, b.lens, b.table)

    def check(self):
        assert self.B.tl_query_status(self.sig)[0] == 0
        q, want = self.expected()
        got = (self.dk.cpu().numpy(), self.dks.cpu().numpy(), self.dv.cpu().numpy(), self.dvs.cpu().numpy())
        for name, g, w in zip(("k", "k scale", "v", "v scale"), got, want):
            same = np.array_equal(g, w) if "scale" in name else np.array_equal(ora.TABLE[g], ora.TABLE[w], equal_nan=True)
            assert same, (name, int((g != w).sum()), np.argwhere(g != w)[:4].tolist())
        # one rounding to bf16, 2^-8; the row's factor in fp32: a sum of D squares in chains of 8 and log2(D/8) at most 12
        # roundings of 2^-24 (half of them after the root), the root's 2^-22, and three roundings in products and their
        # sum, of terms up to the row's largest: below 2^-20 of it
        g = f64(self.q_out)
        nan = np.isnan(q)
        assert np.array_equal(nan, np.isnan(g))
        assert (np.abs(g - q)[~nan] <= (2.0 ** -8 * np.abs(q) + 2.0 ** -19 * self.q_large)[~nan]).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rot,interleaved,norm", [("all", False, "qk"), ("all", True, "qk"), (32, False, "k"), (16, True, "q"),
                                                  (0, False, "qk"), ("all", False, "")])
def test_ragged_batch(B, layout, rot, interleaved, norm):
    b = Batch([1, 0, 70, 5, 1, 33, 300], [1, 9, 70, 37, 256, 97, 411], seed=1, **layout)
    c = Case(B, b, rot=layout["D"] if rot == "all" else rot, interleaved=interleaved, norm=norm)
    c.call()
    c.check()


@pytest.mark.parametrize("layout", LAYOUTS[:3])
@pytest.mark.parametrize("order", ["hnd", "nhd", "kv"])
def test_positions_of_their_own(B, layout, order):
    b = Batch([1, 7, 26, 64, 3], [1, 64, 90, 200, 65], seed=2, order=order, **layout)
    c = Case(B, b, rot=layout["D"], positions=lambda p: np.random.default_rng(3).permutation(p) + 5, fused=order != "kv")
    c.call(max_q_len=64)
    c.check()


@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** 62, 2.0 ** -30, 2.0 ** -100])
def test_rows_of_any_magnitude(B, scale):
    """Squares of large elements leave fp32, those of small ones vanish beside eps."""
    b = Batch([40, 3], [40, 20], seed=4, H=4, Hkv=2, D=128, ps=16)
    c = Case(B, b, rot=128, scale=scale)
    c.call()
    c.check()


@pytest.mark.parametrize("weight", [2.0 ** -70, 2.0 ** 62, 2.0 ** -30])
def test_weights_of_any_magnitude(B, weight):
    """Scale bytes next to both ends."""
    b = Batch([40, 3], [40, 20], seed=13, H=4, Hkv=2, D=128, ps=16)
    w = (b.bf16(128).float() * weight).to(torch.bfloat16)
    c = Case(B, b, rot=128, weights=(w, w))
    c.call()
    c.check()


@pytest.mark.parametrize("rot,interleaved", [(128, False), (96, True), (48, False)])
def test_many_heads_and_rows_to_a_page(B, rot, interleaved):
    """More heads than a block takes at a time, and more rows of a page than its threads hold."""
    def edit(rows):
        rows[100, -3:, 5] = float("inf")
        rows[300, -2:, 77] = float("nan")
        rows[400, -1:, 8:16] = -float("inf")
    b = Batch([512, 1, 90], [700, 130, 90], seed=14, H=40, Hkv=8, D=128, ps=256)
    c = Case(B, b, rot=rot, interleaved=interleaved, edit=edit)
    c.call()
    c.check()


def test_rows_of_zeros_infinities_and_nan(B):
    def edit(rows):
        rows[2] = 0.0
        rows[5, :, 3] = float("inf")
        rows[6, :, 100] = -float("inf")
        rows[7, :, 9] = float("nan")
        rows[8, :, 1:] = 0.0
    b = Batch([12, 3], [12, 20], seed=5, H=4, Hkv=2, D=128, ps=16)
    c = Case(B, b, rot=64, edit=edit)
    c.call()
    c.check()


def test_a_largest_element_next_to_a_scale_border(B):
    """Rows of equal magnitudes are normed to just below the weight; 1.75 is the border of a scale byte (448 = 1.75 * 2^8)."""
    def edit(rows):
        rows.copy_(torch.sign(rows) * 0.5)
    b = Batch([30, 5], [30, 20], seed=6, H=2, Hkv=2, D=64, ps=16)
    w = torch.full((64,), 1.75, dtype=torch.bfloat16)
    for eps in (1e-12, 1e-9, 1e-6):
        c = Case(B, b, rot=0, edit=edit, weights=(w, w), eps=eps)
        c.call()
        c.check()


def test_again_and_captured(B):
    """The same call twice, the second from a graph, gives the same cache; on a stream of its own."""
    b = Batch([9, 1, 40], [30, 1, 70], seed=7, H=4, Hkv=2, D=128, ps=32)
    c = Case(B, b, rot=128, positions=lambda p: p // 2)
    c.call()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        c.call()
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_no_queries(B):
    b = Batch([9, 1], [30, 1], seed=8, H=4, Hkv=2, D=128, ps=32)
    c = Case(B, b, rot=128)
    c.call(q=None, q_out=None, q_weight=None)
    torch.cuda.synchronize()
    assert (c.q_out == 7.0).all()
    c.call()
    c.check()


def test_a_wrong_position_is_reported_and_the_others_come_out_right(B):
    b = Batch([4, 6, 5], [20, 16, 40], seed=9, H=2, Hkv=1, D=64, ps=16)
    def at(p):
        p = p.copy()
        p[6] = 1000
        return p
    c = Case(B, b, rot=64, positions=at, max_pos=2000)
    c.kw["cos"], c.kw["sin"] = c.kw["cos"][:50].contiguous(), c.kw["sin"][:50].contiguous()
    c.call()
    code, where = B.tl_query_status(c.sig)
    assert code == B.TL_ERR_INVALID and where == 1
    q, want = c.expected()
    mine = [0, 2]  # sequences that are right
    for s in mine:
        for p in b.table[s, :-(-b.lens[s] // b.ps)]:
            assert np.array_equal(c.dk.cpu().numpy()[p], want[0][p]) and np.array_equal(c.dks.cpu().numpy()[p], want[1][p])


def test_the_same_as_the_plain_call_without_norms_and_positions(B):
    b = Batch([9, 1, 40], [30, 1, 70], seed=10, H=4, Hkv=2, D=128, ps=32)
    c, d = (Case(B, Batch([9, 1, 40], [30, 1, 70], seed=10, H=4, Hkv=2, D=128, ps=32), rot=128, norm="") for _ in range(2))
    c.call()
    B.tl_kv_append(d.cache, d.k, d.v, *d.batch, d.sig, q=d.q, q_out=d.q_out, cos=d.kw["cos"], sin=d.kw["sin"])
    for x, y in ((c.dk, d.dk), (c.dks, d.dks), (c.dv, d.dv), (c.q_out, d.q_out)):
        assert torch.equal(x, y)


def test_binding_refuses(B):
    b = Batch([2], [20], seed=11, H=2, Hkv=1, D=64, ps=16)
    c = Case(B, b, rot=64)
    bad = [dict(q_weight=c.kw["q_weight"].float()), dict(k_weight=c.kw["k_weight"][:32]), dict(k_weight=c.wk),
           dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(positions=torch.zeros(2, dtype=torch.int64, device="cuda"))]
    for kw in bad:
        with pytest.raises(ValueError):
            c.call(**kw)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(B.TLError):
            c.call(eps=eps)
