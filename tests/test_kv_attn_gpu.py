"""tl_kv_attn against the float64 oracle."""
import numpy as np
import pytest
import torch

from tests.kv_cases import Batch, check_attention, expected_attention, f64
from oracle import kv_cache as ora

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


class Call:
    """One batch's device side; run() may be called again."""

    def __init__(self, B, b, *, causal=True, scale=0.0, q_scale=1.5, spread=3, edit=None, max_q_len=0, strided=False):
        self.B, self.b, self.causal, self.scale, self.max_q_len = B, b, causal, scale, max_q_len
        self.kc, self.ks = b.random_codes(spread)
        self.vc, self.vs = b.random_codes(spread)
        self.q = b.bf16(b.n, b.H, b.D, scale=q_scale)
        if edit:
            edit(self)
        k, v = b.both(self.kc, self.vc)
        self.cache = B.KvCache(k, v, torch.from_numpy(self.ks).cuda(), torch.from_numpy(self.vs).cuda())
        self.sig = B.Signals(1)
        self.args = b.device()
        self.dq = self.q.cuda()
        if strided:
            wide = torch.zeros(b.n, b.H + 3, b.D + 8, dtype=torch.bfloat16, device="cuda")
            wide[:, 1:b.H + 1, :b.D] = self.dq
            self.dq = wide[:, 1:b.H + 1, :b.D]
            assert self.dq.data_ptr() % 16 == 0
        self.ws = torch.zeros(B.tl_kv_attn_workspace_size(b.n, len(b.q), b.H, b.Hkv, b.D), dtype=torch.uint8,
                              device="cuda")

    def run(self, stream=None):
        b = self.b
        self.out = torch.full((b.n, b.H, b.D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((b.H, b.n), 7.0, dtype=torch.float32, device="cuda")
        self.B.tl_kv_attn(self.dq, self.cache, self.out, *self.args, self.ws, self.sig, causal=self.causal,
                          scale=self.scale, max_q_len=self.max_q_len, lse=self.lse, stream=stream)
        return self

    def check(self):
        assert self.B.tl_query_status(self.sig)[0] == 0
        b = self.b
        scale = self.scale or b.D ** -0.5
        want, lse, vmax, smax = expected_attention(b, f64(self.q), self.kc, self.ks, self.vc, self.vs, self.causal, scale)
        check_attention(f64(self.out), f64(self.lse), want, lse, vmax, smax)
        return self


LAYOUTS = [dict(H=4, Hkv=2, D=128, ps=64), dict(H=3, Hkv=3, D=64, ps=16), dict(H=16, Hkv=1, D=128, ps=16),
           dict(H=40, Hkv=2, D=64, ps=256), dict(H=7, Hkv=1, D=128, ps=48)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("causal", [True, False])
def test_single_tokens_of_ragged_lengths(B, layout, causal):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 129, 300, 1000, 1]
    Call(B, Batch([1] * len(lens), lens, seed=1, **layout), causal=causal).run().check()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("causal", [True, False])
def test_drafts_and_chunks(B, layout, causal):
    b = Batch([4, 0, 1, 9, 33, 64, 0, 3], [100, 50, 1, 9, 47, 64, 0, 700], seed=2, **layout)
    Call(B, b, causal=causal).run().check()


@pytest.mark.parametrize("D,group", [(128, 4), (64, 1), (128, 5), (64, 16)])
def test_prompt_chunks(B, D, group):
    b = Batch([130, 257, 64], [130, 300, 500], H=2 * group, Hkv=2, D=D, ps=32, seed=3)
    Call(B, b).run().check()


@pytest.mark.parametrize("order", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("layout", LAYOUTS[:2])
def test_orders_and_strides(B, order, layout):
    b = Batch([1, 3, 40], [77, 200, 90], seed=4, order=order, extra_columns=2, **layout)
    Call(B, b, strided=True).run().check()


def test_a_long_context_is_shared_by_many(B):
    Call(B, Batch([1], [5003], H=4, Hkv=1, D=128, ps=64, seed=5)).run().check()
    Call(B, Batch([2, 1, 1], [3000, 1, 17], H=2, Hkv=1, D=64, ps=16, seed=6)).run().check()


def test_many_short_sequences(B):
    rng = np.random.default_rng(7)
    lens = rng.integers(0, 60, 600).tolist()
    q = [0 if n == 0 or i % 7 == 0 else 1 for i, n in enumerate(lens)]
    Call(B, Batch(q, lens, H=2, Hkv=2, D=64, ps=16, seed=7)).run().check()


# Enough tiles for two and for four blocks to an SM, single tokens and tiles of 16 rows, some of them cut.
@pytest.mark.parametrize("seqs", [30, 70])
@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("D,longest", [(128, 700), (64, 40), (128, 1100)])
def test_several_blocks_of_an_sm(B, seqs, q_len, D, longest):
    rng = np.random.default_rng(seqs + longest)
    q = [q_len] * (seqs - 2) + [0, 1]
    lens = [int(x) for x in rng.integers(1, longest, seqs - 3)] + [longest, 0, 1]
    lens = [max(a, c) for a, c in zip(lens, q)]
    b = Batch(q, lens, H=32, Hkv=8, D=D, ps=32, seed=seqs)
    call = Call(B, b, max_q_len=q_len).run().check()
    first = call.out.clone(), call.lse.clone()
    call.run()
    torch.cuda.synchronize()
    assert torch.equal(first[0], call.out) and torch.equal(first[1], call.lse)


@pytest.mark.parametrize("q_len", [1, 40])
def test_rows_that_see_nothing(B, q_len):
    # sequence 0 has a new token and no length with it: an error by the batch's own count, rows empty all the same
    b = Batch([q_len, 2], [0, 5], seed=8, **LAYOUTS[0])
    c = Call(B, b, causal=True).run()
    assert B.tl_query_status(c.sig) == (B.TL_ERR_INVALID, 0)
    assert (c.out[:q_len] == 0).all() and torch.isneginf(c.lse[:, :q_len]).all()
    c.check()


@pytest.mark.parametrize("max_q_len", [0, 1, 3, 500])
def test_the_hint_changes_nothing_that_matters(B, max_q_len):
    Call(B, Batch([3, 1, 70], [80, 65, 200], seed=9, **LAYOUTS[0]), max_q_len=max_q_len).run().check()


@pytest.mark.parametrize("q_len", [1, 5, 160])
def test_nan_where_nothing_is_seen_stays_there(B, q_len):
    def edit(c):
        b = c.b
        for codes in (c.kc, c.vc):
            for s in range(len(b.q)):   # slots past the end, and pages of nobody
                n = b.lens[s]
                if n % b.ps:
                    codes[b.table[s, n // b.ps], :, n % b.ps:] = 127
        used = set(b.table[b.table >= 0].ravel().tolist())
        for p in set(range(b.pages)) - used:
            c.kc[p], c.vc[p], c.ks[p], c.vs[p] = 255, 127, 255, 255
    lens = [q_len, q_len + 3, 170, 191]
    Call(B, Batch([q_len] * 4, lens, seed=10, spare=3, **LAYOUTS[0]), edit=edit).run().check()
    Call(B, Batch([q_len] * 4, lens, seed=11, spare=3, **LAYOUTS[1]), edit=edit, causal=False).run().check()


@pytest.mark.parametrize("q_len", [4, 24, 150])
@pytest.mark.parametrize("layout", LAYOUTS[:2])
def test_nan_that_only_later_rows_see(B, q_len, layout):
    """A new token's own NaN value or key reaches the rows from it on and no earlier one."""
    def edit(c):
        b = c.b
        pos = b.lens[0] - 2   # the last but one token: seen by the last two rows
        c.vc[b.table[0, pos // b.ps], :, pos % b.ps, 3] = 127
        c.vc[b.table[0, pos // b.ps], 0, pos % b.ps, 60] = 255
        pos = b.lens[1] - 1
        c.kc[b.table[1, pos // b.ps], :, pos % b.ps, 7] = 127
    b = Batch([q_len, q_len], [q_len + 40, q_len + 21], seed=12, **layout)
    c = Call(B, b, edit=edit).run()
    out, lse = f64(c.out), f64(c.lse)
    assert not np.isnan(out[:q_len - 2]).any() and not np.isnan(out[q_len:2 * q_len - 1]).any()
    assert np.isnan(out[q_len - 2:q_len, :, 3]).all() and not np.isnan(out[q_len - 2:q_len, :, 5]).any()
    assert np.isnan(out[2 * q_len - 1]).all() and np.isnan(lse[:, 2 * q_len - 1]).all()
    # with the NaN replaced by zeros the rows before it have the same result
    c.vc[np.isin(c.vc, (127, 255))] = 0
    c.kc[np.isin(c.kc, (127, 255))] = 0
    want, wl, vmax, smax = expected_attention(b, f64(c.q), c.kc, c.ks, c.vc, c.vs, True, b.D ** -0.5)
    keep = np.r_[0:q_len - 2, q_len:2 * q_len - 1]
    check_attention(out[keep], lse[:, keep], want[keep], wl[:, keep], vmax[keep], smax[keep])


@pytest.mark.parametrize("q_len", [1, 60])
def test_scores_of_great_spread(B, q_len):
    """Large queries: the maximum jumps, most weights vanish, sums are rescaled."""
    Call(B, Batch([q_len, q_len], [400, 900], seed=13, **LAYOUTS[0]), q_scale=30.0).run().check()


@pytest.mark.parametrize("q_len", [1, 60])
def test_small_and_large_numbers(B, q_len):
    for q_scale, scale in [(1e-30, 1e29), (1e30, 1e-31), (1e-3, 100.0)]:
        Call(B, Batch([q_len, 1], [100, 50], seed=14, **LAYOUTS[0]), q_scale=q_scale, scale=scale).run().check()


@pytest.mark.parametrize("q_len", [1, 60])
def test_value_scales_of_great_spread(B, q_len):
    """Blocks whose scales differ by 2^20, the largest first, in the middle or last; all-zero blocks of scale byte 0."""
    def edit(c):
        b = c.b
        for s in range(len(b.q)):
            k = -(-b.lens[s] // b.ps)
            for j in range(k):
                c.vs[b.table[s, j]] = (140, 120, 131)[(j + s) % 3]
            zero = b.table[s, k // 2]
            c.vs[zero], c.vc[zero] = 0, 0
            c.ks[zero], c.kc[zero] = 0, 0
    Call(B, Batch([q_len] * 3, [300, 500, 260], H=4, Hkv=2, D=128, ps=32, seed=15), edit=edit).run().check()


@pytest.mark.parametrize("q_len", [1, 60])
def test_a_long_tail_of_small_weights_counts(B, q_len):
    """One key with weight 1 and 4095 equal ones of weight 2^-22 each against it: together a thousandth."""
    n = 4095 + q_len

    def edit(c):
        c.kc[:], c.vc[:] = 0, 0x38                       # zeros; value 1
        c.ks[:], c.vs[:] = 127, 127
        c.q[:] = 0
        c.q[..., 0] = 1.0
        first = c.b.table[0, 0]
        c.kc[first, :, 0, 0] = ora.encode(15.0)          # score 15, weight e^15 = 2^21.6 times the others'
        c.vc[first, :, 0, :] = ora.encode(-1.0)
    c = Call(B, Batch([q_len], [n], H=1, Hkv=1, D=64, ps=64, seed=16), edit=edit, scale=1.0, causal=False).run().check()
    tail = (n - 1) * np.exp(-15.0)
    assert abs(float(c.lse[0, 0]) - (15.0 + np.log1p(tail))) < 1e-5


# Maxima that come late: scores that rise (fall) with the token, slowly and by far more than fp16 holds, and a last key
# above all others.
@pytest.mark.parametrize("q_len", [1, 3, 60])
@pytest.mark.parametrize("ramp", [1.0, 8.0, -1.0, -8.0, "last"])
@pytest.mark.parametrize("causal", [True, False])
def test_scores_that_rise_along_the_sequence(B, q_len, ramp, causal):
    n = 1500

    def edit(c):
        c.kc[:] = 0
        c.ks[:], c.vs[:] = 127, 121
        c.q[:] = 0
        c.q[..., 0] = 1.0 if ramp == "last" else float(ramp)
        for j in range(n):
            page, slot = c.b.table[0, j // 64], j % 64
            x = (14.0 if j == n - 1 else 0.0) if ramp == "last" else 16.0 * j / n - 8.0
            c.kc[page, :, slot, 0] = ora.encode(x)
    b = Batch([q_len], [n], H=4, Hkv=1, D=128, ps=64, seed=19)
    Call(B, b, edit=edit, scale=1.0, causal=causal, max_q_len=q_len).run().check()


def test_scale_byte_255_is_nan(B):
    def edit(c):
        c.ks[c.b.table[0, 0]] = 255
        c.vs[c.b.table[1, 0]] = 255
    c = Call(B, Batch([1, 1, 1], [20, 20, 20], seed=17, **LAYOUTS[0]), edit=edit).run()
    out = f64(c.out)
    assert np.isnan(out[:2]).all() and not np.isnan(out[2]).any()


@pytest.mark.parametrize("q_len", [1, 100])
@pytest.mark.parametrize("what", ["page", "page negative", "length", "cu"])
def test_bad_batches_are_reported_and_stay_inside(B, what, q_len):
    """As for appending: each index is checked in the kernel before it is used."""
    b = Batch([q_len] * 3, [130, 140, 190], seed=18, **LAYOUTS[0])
    c = Call(B, b)
    cu, lens, table = c.args
    if what == "page":
        table[1, 1] = b.pages
    elif what == "page negative":
        table[1, 0] = -1
    elif what == "length":
        lens[1] = 64 * b.cols + 1
        table[1] = table[1].clamp(min=0)
    elif what == "cu":
        cu[2] = 100000
    c.run()
    code, where = B.tl_query_status(c.sig)
    assert code == B.TL_ERR_INVALID and where in (1, 2)
    want, lse, vmax, smax = expected_attention(b, f64(c.q), c.kc, c.ks, c.vc, c.vs, True, b.D ** -0.5)
    rows = slice(0, q_len)
    check_attention(f64(c.out)[rows], f64(c.lse)[:, rows], want[rows], lse[:, rows], vmax[rows], smax[rows])
    # the workspace is in order: the next call is right
    c.args = b.device()
    c.run().check()


@pytest.mark.parametrize("q", [[1, 1, 1, 1], [1, 40, 2, 130]])
def test_same_bits_again_on_a_stream_and_in_a_graph(B, q):
    c = Call(B, Batch(q, [500, 70, 1300, 131], seed=19, **LAYOUTS[0])).run().check()
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


def test_one_workspace_for_many_calls(B):
    calls = [Call(B, Batch(q, n, seed=21, **LAYOUTS[i])) for i, q, n in
             ((0, [1, 1], [900, 30]), (1, [200, 3], [500, 400]), (0, [300], [1500]), (4, [2] * 9, [77] * 9), (1, [1], [3000]))]
    ws = max((c.ws for c in calls), key=lambda w: w.numel()).clone()
    for c in calls + calls[::-1]:
        c.ws = ws
        c.run().check()


def test_binding_refuses_wrong_tensors(B):
    b = Batch([2, 1], [30, 5], seed=22, **LAYOUTS[0])
    c = Call(B, b)
    cu, lens, table = c.args
    out, lse = torch.empty_like(c.dq), torch.empty(b.H, b.n, device="cuda")
    good = dict(q=c.dq, cache=c.cache, out=out, cu_seqlens=cu, seq_lens=lens, page_table=table, workspace=c.ws,
                signals=c.sig, lse=lse)
    B.tl_kv_attn(**good)
    for bad in (dict(q=c.dq.float()), dict(q=c.dq[..., :64]), dict(q=c.dq.cpu()), dict(out=out[:1]), dict(cu_seqlens=cu.long()),
                dict(cu_seqlens=cu[:2]), dict(seq_lens=lens.cpu()), dict(page_table=table.long()), dict(lse=lse.t()),
                dict(page_table=table.repeat(1, 2)[:, ::2])):
        with pytest.raises(ValueError):
            B.tl_kv_attn(**{**good, **bad})
    with pytest.raises(B.TLError):
        B.tl_kv_attn(**{**good, "workspace": c.ws[:256]})
    rows = torch.zeros(b.n, b.Hkv, b.D, dtype=torch.bfloat16, device="cuda")
    cos = torch.zeros(64, 64, device="cuda")
    good = dict(cache=c.cache, k=rows, v=rows, cu_seqlens=cu, seq_lens=lens, page_table=table, signals=c.sig)
    for bad in (dict(k=rows.half()), dict(v=rows[:, :1]), dict(q=rows), dict(cos=cos), dict(cos=cos, sin=cos.double()),
                dict(q=rows, q_out=rows.float()), dict(k=rows.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            B.tl_kv_append(**{**good, **bad})
    assert B.tl_query_status(c.sig)[0] == 0


def test_offsets_past_32_bits(B):
    """A pool of more than 4 GiB, the sequence's pages at its far end."""
    D, ps = 128, 256
    pages = (1 << 32) // (D * ps) + 8
    b = Batch([1], [700], H=2, Hkv=1, D=D, ps=ps, seed=20)
    kc, ks = b.random_codes()
    vc, vs = b.random_codes()
    pool = torch.zeros(pages, 1, ps, D, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(2, pages, 1, dtype=torch.uint8, device="cuda")
    far = pages - b.pages
    pool[far:] = torch.from_numpy(kc).cuda()
    scale[0, far:] = torch.from_numpy(ks).cuda()
    vpool = torch.zeros_like(pool)
    vpool[far:] = torch.from_numpy(vc).cuda()
    scale[1, far:] = torch.from_numpy(vs).cuda()
    cache = B.KvCache(pool, vpool, scale[0], scale[1])
    q = b.bf16(1, 2, D)
    cu, lens, table = b.device()
    out, lse = torch.empty(1, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 1, device="cuda")
    ws = torch.zeros(B.tl_kv_attn_workspace_size(1, 1, 2, 1, D), dtype=torch.uint8, device="cuda")
    sig = B.Signals(1)
    B.tl_kv_attn(q.cuda(), cache, out, cu, lens, torch.where(table >= 0, table + far, table), ws, sig, lse=lse)
    assert B.tl_query_status(sig)[0] == 0
    check_attention(f64(out), f64(lse), *expected_attention(b, f64(q), kc, ks, vc, vs, True, D ** -0.5))
    # a token appended there: the last page's next slot
    b.q, b.lens = [1], [701]
    rows = b.bf16(1, 1, D)
    cu, lens, table = b.device()
    B.tl_kv_append(cache, rows.cuda(), rows.cuda(), cu, lens, torch.where(table >= 0, table + far, table), sig)
    assert B.tl_query_status(sig)[0] == 0
    wk, wks = ora.append(kc, ks, f64(rows), [0, 1], [701], b.table)
    assert np.array_equal(pool[far:].cpu().numpy(), wk) and np.array_equal(scale[0, far:].cpu().numpy(), wks)
