"""The calls for drafts and beams together, as a decoder uses them, against their oracles step by step."""
import numpy as np
import pytest
import torch

from tests.kv_cases import check_attention, f64, tables
from oracle import beam as beams
from oracle import kv_cache as ora
from oracle import kv_pages

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Decoder:
    """Some sequences' pages and some layers' caches, on the device and for the oracle."""

    def __init__(self, B, rows, *, layers=2, H=8, Hkv=2, D=64, ps=16, pages=200, columns=24, most=40, seed=0, pad=0):
        self.pad = pad  # rows behind the last sequence's in every batch
        self.B, self.rng, self.rows, self.n_layers, self.H, self.Hkv, self.D, self.ps = B, np.random.default_rng(seed), rows, layers, H, Hkv, D, ps
        self.codes = np.zeros((layers, 2, pages, Hkv, ps, D), np.uint8)
        self.scales = np.zeros(self.codes.shape[:4], np.uint8)
        self.d, self.ds = torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scales).cuda()
        self.layers = B.KvLayers([B.KvCache(self.d[l, 0], self.d[l, 1], self.ds[l, 0], self.ds[l, 1]) for l in range(layers)])
        self.table, self.lens, self.refs = np.zeros((rows, columns), np.int32), np.zeros(rows, np.int32), np.zeros(pages, np.int32)
        self.d_table, self.d_lens, self.d_refs = i32(self.table), i32(self.lens), i32(self.refs)
        self.cos, self.sin = tables(600, D)
        self.d_cos, self.d_sin = torch.from_numpy(self.cos).cuda(), torch.from_numpy(self.sin).cuda()
        bf = lambda *s: torch.from_numpy(self.rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16)
        self.wq, self.wk = bf(D), bf(D)
        self.bf, self.sig = bf, B.Signals(1)
        byte = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
        self.ws_pages = byte(max(B.tl_kv_resize_workspace_size(rows), B.tl_kv_fork_workspace_size(rows, rows)))
        self.ws_attn = byte(B.tl_kv_attn_workspace_size(rows * most + pad, rows, H, Hkv, D))

    def resize(self, new):
        """To these lengths: an array, or a device tensor with the array."""
        d_new, new = (new if isinstance(new, tuple) else (i32(new), np.asarray(new, np.int32)))
        self.B.tl_kv_resize(self.d_table, self.d_lens, d_new, self.d_refs, self.d_refs, self.ws_pages, self.sig, page_size=self.ps)
        self.table, self.refs = kv_pages.resize(self.table, self.lens, new, self.refs, self.ps)
        self.lens, self.d_lens = new.copy(), d_new.clone()

    def append(self, q, positions=None):
        """q[s] new tokens behind each sequence (already made room for): random rows through every layer; the attention's
        queries and the batch's boundaries."""
        cu = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        n, H, Hkv = int(cu[-1]), self.H, self.Hkv
        pos = np.concatenate([np.arange(l - m, l) for l, m in zip(self.lens, q)]) if positions is None else positions
        d_cu = i32(cu)
        q_out = torch.full((n + self.pad, H, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        if positions is not None:
            positions = np.concatenate([positions, np.full(self.pad, -5)])
        for l, cache in enumerate(self.layers.caches):
            x = self.bf(n + self.pad, H + 2 * Hkv, self.D)
            dx = x.cuda()
            self.B.tl_kv_append_norm(cache, dx[:, H:H + Hkv], dx[:, H + Hkv:], d_cu, self.d_lens, self.d_table, self.sig, q=dx[:, :H],
                                     q_out=q_out, q_weight=self.wq.cuda(), k_weight=self.wk.cuda(), eps=EPS, cos=self.d_cos,
                                     sin=self.d_sin, positions=None if positions is None else i32(positions), max_q_len=int(max(q)))
            k = ora.normed(f64(x)[:n, H:H + Hkv], f64(self.wk), EPS)
            k = np.stack([ora.rotate(k[t], p, self.cos, self.sin, False) for t, p in enumerate(pos[:n])])
            for i, rows in enumerate((k, f64(x)[:n, H + Hkv:])):
                self.codes[l, i], self.scales[l, i] = ora.append(self.codes[l, i], self.scales[l, i], rows, cu, self.lens, self.table)
        assert (q_out[n:] == 7).all()
        return q_out, cu, d_cu

    def check_cache(self):
        assert self.B.tl_query_status(self.sig)[0] == 0
        assert np.array_equal(self.d_lens.cpu().numpy(), self.lens) and np.array_equal(self.d_refs.cpu().numpy(), self.refs)
        table = self.d_table.cpu().numpy()
        held = np.zeros_like(self.refs)
        for s, n in enumerate(self.lens):
            k = -(-int(n) // self.ps)
            assert np.array_equal(table[s, :k], self.table[s, :k])
            np.add.at(held, table[s, :k], 1)
        assert np.array_equal(held, self.refs)  # every page is held as often as it is counted
        got, scales = self.d.cpu().numpy(), self.ds.cpu().numpy()
        for l in range(self.n_layers):
            for i in range(2):
                for s, n in enumerate(self.lens):
                    if n:
                        want = ora.values(self.codes[l, i], self.scales[l, i], self.table[s], int(n))
                        assert np.array_equal(ora.values(got[l, i], scales[l, i], table[s], int(n)), want)

    def attend(self, q_out, cu, d_cu, tree=None, sees=None):
        """Attention over the last layer's cache, against the oracle."""
        n = int(cu[-1])
        q = f64(q_out)[:n]
        out, lse = torch.full_like(q_out, 9.0), torch.full((self.H, n + self.pad), 9.0, device="cuda")
        if tree is None:
            self.B.tl_kv_attn(q_out, self.layers.caches[-1], out, d_cu, self.d_lens, self.d_table, self.ws_attn, self.sig, lse=lse)
        else:
            self.B.tl_kv_tree_attn(q_out, self.layers.caches[-1], out, d_cu, self.d_lens, self.d_table, tree, self.ws_attn, self.sig,
                                   lse=lse)
        want, wl, vmax, smax = np.zeros(q.shape), np.zeros((self.H, n)), np.zeros((n, self.H, 1)), np.zeros((n, self.H, 1))
        for s in range(self.rows):
            rows = slice(cu[s], cu[s + 1])
            if cu[s] == cu[s + 1]:
                continue
            k, v = (ora.values(self.codes[-1, i], self.scales[-1, i], self.table[s], int(self.lens[s])) for i in range(2))
            m = cu[s + 1] - cu[s]
            mask = np.tri(m, dtype=bool) if sees is None else sees[s]
            want[rows], wl[:, rows] = ora.tree_attention(q[rows], k, v, mask, self.D ** -0.5)
            kk, vv = (np.abs(x).repeat(self.H // self.Hkv, 1) for x in (k, v))
            vmax[rows] = vv.max((0, 2))[None, :, None]
            smax[rows] = self.D ** -0.5 * np.einsum("thd,jhd->thj", np.abs(q[rows]), kk).max(2)[:, :, None]
        assert (out[n:] == 9).all() and (lse[:, n:] == 9).all()
        check_attention(f64(out)[:n], f64(lse)[:, :n], want, wl, vmax, smax)


@pytest.mark.parametrize("pad", [0, 13])
def test_drafted_trees(B, pad):
    """Room for the drafts, the drafts appended by depth, seen along their paths, an accepted path kept, the rest given back."""
    rows = 4
    d = Decoder(B, rows, seed=1, pad=pad)
    d.resize([20, 33, 5, 47])
    q = d.append([20, 33, 5, 47])
    d.attend(*q)
    d.check_cache()
    for step in range(5):
        start = d.lens.copy()
        n = [int(d.rng.integers(1, 30)) for _ in range(rows)]
        if step == 2:
            n[1] = 0  # a sequence that drafts nothing
        parents = [[-1 if i == 0 else int(d.rng.integers(-1, i)) for i in range(m)] for m in n]
        sees, depth = [np.zeros((m, m), bool) for m in n], [np.zeros(m, int) for m in n]
        for s in range(rows):
            for i, p in enumerate(parents[s]):
                if p >= 0:
                    sees[s][i] = sees[s][p]
                    depth[s][i] = depth[s][p] + 1
                sees[s][i, i] = True
        d.resize(start + n)
        positions = np.concatenate([start[s] + depth[s] for s in range(rows)]).astype(np.int32)
        q_out, cu, d_cu = d.append(n, positions)
        bits = np.zeros((sum(n) + pad, 32), bool)
        for s in range(rows):
            bits[cu[s]:cu[s + 1], :n[s]] = sees[s]
        tree = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).cuda()
        d.attend(q_out, cu, d_cu, tree, sees)
        d.check_cache()
        kept = []
        for s in range(rows):
            i = int(d.rng.integers(-1, n[s])) if n[s] else -1  # the path to a random draft, or none accepted
            kept.append(np.flatnonzero(sees[s][i]).tolist() if i >= 0 else [])
        table = np.zeros((rows, 32), np.int32)
        for s, path in enumerate(kept):
            table[s, :len(path)] = path
        after = torch.empty(rows, dtype=torch.int32, device="cuda")
        B.tl_kv_compact(d.layers, i32(table), i32([len(p) for p in kept]), d_cu, d.d_lens, d.d_table, after, d.sig)
        for l in range(d.n_layers):
            for i in range(2):
                d.codes[l, i], d.scales[l, i], new = kv_pages.compact(d.codes[l, i], d.scales[l, i], kept, cu, d.lens, d.table)
        d.resize((after, new))
        d.check_cache()


@pytest.mark.parametrize("pad", [0, 5])
def test_beams(B, pad):
    """Beams chosen, their pages shared and copied, a token appended to each, attention; some beams end on the way."""
    users, K, V, T = 3, 4, 600, 9
    rows = users * K
    d = Decoder(B, rows, seed=2, pad=pad)
    lens = np.repeat([18, 32, 7], K)
    first = np.where(np.arange(rows) % K == 0, lens, 0)  # one beam of each user to begin with
    d.resize(first)
    d.attend(*d.append(first.tolist()))
    scores = np.where(np.arange(K) == 0, 0.0, -np.inf)[None].repeat(users, 0)
    done = np.zeros((users, K), np.uint8)
    history = np.full((rows, T), -1, np.int32)
    d_scores, d_done, d_history = torch.from_numpy(scores.astype(np.float32)).cuda(), torch.from_numpy(done).cuda(), i32(history)
    ws = torch.zeros(B.tl_beam_select_workspace_size(users, K, K, V), dtype=torch.uint8, device="cuda")
    for step in range(T):
        logits = torch.from_numpy(d.rng.standard_normal((rows, V)).astype(np.float32) * 3).cuda()
        if step in (2, 5):
            logits[K + 1, 9] = 25.0  # a beam of the second user ends
        x = f64(logits).reshape(users, K, V)
        parents, tokens = torch.empty(users, K, dtype=torch.int32, device="cuda"), torch.empty(users, K, dtype=torch.int32, device="cuda")
        new_scores, new_done, new_history = torch.empty_like(d_scores), torch.empty_like(d_done), torch.full_like(d_history, -1)
        B.tl_beam_select(logits, d_scores, parents, tokens, new_scores, ws, done=d_done, done_out=new_done, eos=9, history=d_history,
                         history_out=new_history, length=step)
        total = beams.totals(x, f64(d_scores), d_done.cpu().numpy(), 9)[0]
        want = beams.select(total, K)
        p, t = parents.cpu().numpy(), tokens.cpu().numpy()
        for u in range(users):
            assert [(int(a) - u * K, int(b)) for a, b in zip(p[u], t[u])] == [w[:2] for w in want[u]]
            assert np.allclose(f64(new_scores)[u], [w[2] for w in want[u]], rtol=1e-6, atol=1e-5)
        old = d_history.cpu().numpy()
        d_scores, d_done, d_history = new_scores, new_done, new_history
        assert np.array_equal(d_history.cpu().numpy()[:, :step], old[p.ravel(), :step])
        assert np.array_equal(d_history.cpu().numpy()[:, step], t.ravel())
        # their pages
        table, lens_out = torch.zeros_like(d.d_table), torch.empty_like(d.d_lens)
        copies, count = torch.zeros(3, rows, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        B.tl_kv_fork(d.d_table, d.d_lens, d.d_refs, parents.view(-1), table, lens_out, d.d_refs, copies, count, d.ws_pages, d.sig,
                     page_size=d.ps)
        B.tl_kv_copy_pages(d.layers, copies[0], copies[1], d.sig, slots=copies[2], count=count)
        d.table, d.lens, d.refs, made = kv_pages.fork(d.table, d.lens, d.refs, p.ravel(), d.ps, np.zeros_like(d.table))
        for l in range(d.n_layers):
            for i in range(2):
                d.codes[l, i], d.scales[l, i] = kv_pages.copy_pages(d.codes[l, i], d.scales[l, i], made)
        d.d_table, d.d_lens = table, lens_out
        assert count.item() == len(made)
        d.check_cache()
        # a token for each beam that goes on
        more = 1 - d_done.cpu().numpy().ravel().astype(int)
        d.resize(d.lens + more)
        d.attend(*d.append(more.tolist()))
        d.check_cache()
    assert d_done.cpu().numpy()[1].any()
    d.resize(np.zeros(rows))
    d.check_cache()
    assert (d.refs == 0).all()
