"""One decoder layer serving a ragged batch: prompts in chunks, then a token or a tree of drafts at a time.

    python examples/serve_layer.py [--steps 32] [--drafts 0] [--check]

The layer's calls, all on one stream and all on the caller's buffers:

    qkv = x Wqkv                      tl_gemm
    rotate q and k, append k and v    tl_kv_append     (8-bit paged cache)
    o = attention over the cache      tl_kv_attn
    x += o Wo                         tl_gemm
    logits = x Wr                     tl_gemm          (fp32 out)
    x += experts of the top k         tl_moe_decode    (up to 64 tokens a call)

Pages are dealt out by the host as sequences grow.  With --drafts N the layer norms its
queries and keys, pages are dealt out on the device, and each step tries a tree of N
drafted tokens for each sequence, of which a path is kept:

    pages for the drafts              tl_kv_resize
    norm, rotate by depth, append     tl_kv_append_norm
    each draft sees its path          tl_kv_tree_attn
    the kept path moves together      tl_kv_compact
    pages behind it are freed         tl_kv_resize

--check runs the same layer in plain
fp32 torch over an unquantised cache and prints how far the results are apart: the cache's
8 bits (a relative step of 2^-4 in each key and value) are what separates them.
"""
import argparse
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tile_centric_gemm_gb300 import binding as B  # noqa: E402


class Layer:
    """Weights, cache and workspaces of one layer; all allocated here, none during the calls."""

    def __init__(self, *, hidden=512, H=8, H_kv=2, D=64, E=8, inter=256, topk=2, pages=64, page=64, max_tokens=512,
                 max_seqs=8, max_pages=16, max_pos=1024, theta=10000.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-2] ** -0.5).to(torch.bfloat16)
        self.hidden, self.H, self.H_kv, self.D, self.E, self.topk, self.page = hidden, H, H_kv, D, E, topk, page
        self.w_qkv, self.w_o, self.w_r = bf(hidden, (H + 2 * H_kv) * D), bf(H * D, hidden), bf(hidden, E)
        self.w1, self.w2 = bf(E, hidden, 2 * inter), bf(E, inter, hidden)
        self.experts = B.MoeWeights(list(self.w1), list(self.w2))
        codes = lambda: torch.zeros(pages, H_kv, page, D, dtype=torch.uint8, device="cuda")
        scales = lambda: torch.zeros(pages, H_kv, dtype=torch.uint8, device="cuda")
        self.cache = B.KvCache(codes(), codes(), scales(), scales())
        f = theta ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * f  # far positions: angles in 64 bits
        self.cos, self.sin = a.cos().float(), a.sin().float()
        self.signals = B.Signals(1)
        ws = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")
        self.ws_attn = ws(B.tl_kv_attn_workspace_size(max_tokens, max_seqs, H, H_kv, D))
        self.ws_moe = ws(B.tl_moe_decode_workspace_size(64, topk, E, hidden, inter, hidden))
        self.table = torch.zeros(max_seqs, max_pages, dtype=torch.int32)
        self.free = list(range(pages))[::-1]
        self.lens = [0] * max_seqs

    def room(self, new):
        """Pages for new[s] more tokens of sequence s; the batch's boundaries, lengths and page table on the device."""
        for s, k in enumerate(new):
            for p in range(-(-self.lens[s] // self.page), -(-(self.lens[s] + k) // self.page)):
                self.table[s, p] = self.free.pop()
            self.lens[s] += k
        cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        return cu, torch.tensor(self.lens[:len(new)], dtype=torch.int32).cuda(), self.table[:len(new)].cuda()

    def append(self, q, k, v, q_out, batch, most, positions):
        B.tl_kv_append(self.cache, k, v, *batch, self.signals, q=q, q_out=q_out, cos=self.cos, sin=self.sin, max_q_len=most)

    def attention(self, q, o, batch, most, tree):
        B.tl_kv_attn(q, self.cache, o, *batch, self.ws_attn, self.signals, max_q_len=most)

    def __call__(self, x, new, positions=None, tree=None):
        """x [n, hidden] bf16: the new tokens of all sequences, new[s] of sequence s.  Returns x after the layer."""
        n, H, Hkv, D = x.shape[0], self.H, self.H_kv, self.D
        batch = self.room(new)
        new_bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
        qkv = new_bf16(n, (H + 2 * Hkv) * D)
        B.tl_gemm(x, self.w_qkv, qkv, self.signals)
        heads = qkv.view(n, H + 2 * Hkv, D)
        q, o = new_bf16(n, H, D), new_bf16(n, H, D)
        most = max(new)
        self.append(heads[:, :H], heads[:, H:H + Hkv], heads[:, H + Hkv:], q, batch, most, positions)
        self.attention(q, o, batch, most, tree)
        y = new_bf16(n, self.hidden)
        B.tl_gemm(o.view(n, H * D), self.w_o, y, self.signals)
        x = x + y
        logits = torch.empty(n, self.E, device="cuda")
        B.tl_gemm(x, self.w_r, None, self.signals, C_f32=logits)
        y, ids = new_bf16(n, self.hidden), torch.empty(n, self.topk, dtype=torch.int32, device="cuda")
        gates = torch.empty(n, self.topk, device="cuda")
        for t in range(0, n, 64):
            part = slice(t, min(t + 64, n))
            B.tl_moe_decode(x[part], logits[part], self.experts, y[part], ids[part], gates[part], self.ws_moe)
        return x + y

    def status(self):
        code, where = B.tl_query_status(self.signals)
        if code:
            raise RuntimeError(f"{B.STATUS_NAMES.get(code, code)} at {where}")


class DraftLayer(Layer):
    """The layer with normed queries and keys, for trees of drafts; lengths and pages are the device's."""
    eps = 1e-6

    def __init__(self, seqs, **kw):
        super().__init__(**kw)
        g = torch.Generator(device="cuda").manual_seed(2)
        self.q_norm, self.k_norm = ((0.5 + torch.rand(self.D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
        self.layers = B.KvLayers([self.cache])
        self.refs = torch.zeros(len(self.free), dtype=torch.int32, device="cuda")
        self.pages = self.table[:seqs].cuda()
        self.d_lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.ws_pages = torch.zeros(B.tl_kv_resize_workspace_size(seqs), dtype=torch.uint8, device="cuda")

    def resize(self, lens):
        B.tl_kv_resize(self.pages, self.d_lens, lens, self.refs, self.refs, self.ws_pages, self.signals, page_size=self.page)
        self.d_lens = lens

    def room(self, new):
        more = torch.tensor(new, dtype=torch.int32).cuda()
        self.resize(self.d_lens + more)
        self.cu = torch.nn.functional.pad(more.cumsum(0, dtype=torch.int32), (1, 0))
        return self.cu, self.d_lens, self.pages

    def append(self, q, k, v, q_out, batch, most, positions):
        B.tl_kv_append_norm(self.cache, k, v, *batch, self.signals, q=q, q_out=q_out, q_weight=self.q_norm, k_weight=self.k_norm,
                            eps=self.eps, cos=self.cos, sin=self.sin, positions=positions, max_q_len=most)

    def attention(self, q, o, batch, most, tree):
        if tree is None:
            super().attention(q, o, batch, most, tree)
        else:
            B.tl_kv_tree_attn(q, self.cache, o, *batch, tree, self.ws_attn, self.signals, max_q_len=most)

    def keep(self, kept, n_kept):
        """Of each sequence's last drafts those that kept names: int32 [sequences, most] and [sequences], on the device."""
        lens = torch.empty_like(self.d_lens)
        B.tl_kv_compact(self.layers, kept, n_kept, self.cu, self.d_lens, self.pages, lens, self.signals)
        self.resize(lens)


def draft_tree(n, rng):
    """n drafts behind parents of lower number (-1: behind the last token): their masks as words, depths, and a path."""
    words, depth, paths = [], [], []
    for i in range(n):
        p = rng.randrange(-1, i)
        paths.append((paths[p] if p >= 0 else []) + [i])
        depth.append(len(paths[i]) - 1)
        row = [0] * -(-n // 32)
        for j in paths[i]:
            row[j // 32] |= 1 << j % 32
        words.append([w - (1 << 32) if w >> 31 else w for w in row])
    return words, depth, rng.choice(paths)


class Plain:
    """The same layer in fp32 torch, keys and values kept as they are."""

    def __init__(self, layer):
        self.l, self.k, self.v = layer, {}, {}

    def rotate(self, x, pos):
        c, s, h = self.l.cos[pos][:, None], self.l.sin[pos][:, None], self.l.D // 2
        return torch.cat([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], -1)

    def __call__(self, x, new):
        l, x = self.l, x.float()
        qkv = (x @ l.w_qkv.float()).view(-1, l.H + 2 * l.H_kv, l.D)
        if isinstance(l, DraftLayer):
            norm = lambda t, w: t * (t.square().mean(-1, keepdim=True) + l.eps).rsqrt() * w.float()
            qkv = torch.cat([norm(qkv[:, :l.H], l.q_norm), norm(qkv[:, l.H:l.H + l.H_kv], l.k_norm), qkv[:, l.H + l.H_kv:]], 1)
        out, at = [], 0
        for s, n in enumerate(new):
            q, k, v = qkv[at:at + n, :l.H], qkv[at:at + n, l.H:l.H + l.H_kv], qkv[at:at + n, l.H + l.H_kv:]
            start = len(self.k.get(s, ()))
            pos = torch.arange(start, start + n, device="cuda")
            if n:
                self.k[s] = torch.cat([self.k[s], self.rotate(k, pos)]) if s in self.k else self.rotate(k, pos)
                self.v[s] = torch.cat([self.v[s], v]) if s in self.v else v
                kk, vv = (t.repeat_interleave(l.H // l.H_kv, 1) for t in (self.k[s], self.v[s]))
                w = torch.einsum("thd,jhd->htj", self.rotate(q, pos), kk) * l.D ** -0.5
                w = w.masked_fill(torch.arange(len(kk), device="cuda") > pos[:, None], -torch.inf)
                out.append(torch.einsum("htj,jhd->thd", w.softmax(-1), vv).reshape(n, -1))
            at += n
        x = x + torch.cat(out) @ l.w_o.float()
        logits = x @ l.w_r.float()
        top, ids = logits.topk(l.topk, 1)
        gates = torch.zeros_like(logits).scatter_(1, ids, top.softmax(1))
        i = l.w2.shape[1]
        h = torch.einsum("th,ehi->eti", x, l.w1.float())
        y = torch.einsum("eti,eih->eth", torch.nn.functional.silu(h[..., :i]) * h[..., i:], l.w2.float())
        return x + torch.einsum("te,eth->th", gates, y), logits


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--drafts", type=int, default=0, help="drafted tokens of a sequence in each step (0: none)")
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    layer = DraftLayer(4) if a.drafts else Layer()
    plain = Plain(layer) if a.check else None
    g = torch.Generator(device="cuda").manual_seed(1)
    rng = random.Random(1)
    batches = [[100, 3, 257, 0], [60, 90, 1, 130]] + [[a.drafts or 1] * 4] * a.steps  # two rounds of chunks, then steps
    lens = [0] * 4
    worst = 0.0
    for step, new in enumerate(batches):
        x = torch.randn(sum(new), layer.hidden, generator=g, device="cuda").to(torch.bfloat16)
        if a.drafts and step >= 2:
            trees = [draft_tree(a.drafts, rng) for _ in new]
            positions = torch.tensor([n + d for n, (_, depth, _) in zip(lens, trees) for d in depth], dtype=torch.int32)
            masks = torch.tensor([w for words, _, _ in trees for w in words], dtype=torch.int32)
            y = layer(x, new, positions.cuda(), masks.cuda())
            paths = [path for _, _, path in trees]
            new = [len(p) for p in paths]
            layer.keep(torch.tensor([p + [0] * (a.drafts - len(p)) for p in paths], dtype=torch.int32).cuda(),
                       torch.tensor(new, dtype=torch.int32).cuda())
            rows = torch.tensor([s * a.drafts + i for s, p in enumerate(paths) for i in p]).cuda()
            x, y = x[rows], y[rows]  # what goes on
        else:
            y = layer(x, new)
        lens = [n + k for n, k in zip(lens, new)]
        if plain:
            want, logits = plain(x, new)
            # where two experts' logits are closer than the cache's steps move them, another may be chosen: left out
            top = logits.sort(1, descending=True).values
            clear = top[:, layer.topk - 1] - top[:, layer.topk] > 0.25
            if clear.any():
                worst = max(worst, float(((y.float() - want)[clear].norm(dim=1) / want[clear].norm(dim=1)).max()))
    layer.status()
    print(f"{len(batches)} calls, lengths {lens}" + (f", worst relative distance {worst:.4f}" if plain else ""))
    return worst


if __name__ == "__main__":
    main()
