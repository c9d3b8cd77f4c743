"""One decoder layer serving a ragged batch: prompts in chunks, then a token at a time.

    python examples/serve_layer.py [--steps 32] [--check]

The layer's calls, all on one stream and all on the caller's buffers:

    qkv = x Wqkv                      tl_gemm
    rotate q and k, append k and v    tl_kv_append     (8-bit paged cache)
    o = attention over the cache      tl_kv_attn
    x += o Wo                         tl_gemm
    logits = x Wr                     tl_gemm          (fp32 out)
    x += experts of the top k         tl_moe_decode    (up to 64 tokens a call)

Pages are dealt out by the host as sequences grow.  --check runs the same layer in plain
fp32 torch over an unquantised cache and prints how far the results are apart: the cache's
8 bits (a relative step of 2^-4 in each key and value) are what separates them.
"""
import argparse
import os
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

    def __call__(self, x, new):
        """x [n, hidden] bf16: the new tokens of all sequences, new[s] of sequence s.  Returns x after the layer."""
        n, H, Hkv, D = x.shape[0], self.H, self.H_kv, self.D
        for s, k in enumerate(new):
            for p in range(-(-self.lens[s] // self.page), -(-(self.lens[s] + k) // self.page)):
                self.table[s, p] = self.free.pop()
            self.lens[s] += k
        cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        lens, table = torch.tensor(self.lens[:len(new)], dtype=torch.int32).cuda(), self.table[:len(new)].cuda()
        new_bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
        qkv = new_bf16(n, (H + 2 * Hkv) * D)
        B.tl_gemm(x, self.w_qkv, qkv, self.signals)
        heads = qkv.view(n, H + 2 * Hkv, D)
        q, o = new_bf16(n, H, D), new_bf16(n, H, D)
        most = max(new)
        B.tl_kv_append(self.cache, heads[:, H:H + Hkv], heads[:, H + Hkv:], cu, lens, table, self.signals, q=heads[:, :H],
                       q_out=q, cos=self.cos, sin=self.sin, max_q_len=most)
        B.tl_kv_attn(q, self.cache, o, cu, lens, table, self.ws_attn, self.signals, max_q_len=most)
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
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    layer = Layer()
    plain = Plain(layer) if a.check else None
    g = torch.Generator(device="cuda").manual_seed(1)
    batches = [[100, 3, 257, 0], [60, 90, 1, 130]] + [[1, 1, 1, 1]] * a.steps  # two rounds of chunks, then tokens
    worst = 0.0
    for new in batches:
        x = torch.randn(sum(new), layer.hidden, generator=g, device="cuda").to(torch.bfloat16)
        y = layer(x, new)
        if plain:
            want, logits = plain(x, new)
            # where two experts' logits are closer than the cache's steps move them, another may be chosen: left out
            top = logits.sort(1, descending=True).values
            clear = top[:, layer.topk - 1] - top[:, layer.topk] > 0.25
            if clear.any():
                worst = max(worst, float(((y.float() - want)[clear].norm(dim=1) / want[clear].norm(dim=1)).max()))
    layer.status()
    print(f"{len(batches)} calls, lengths {layer.lens[:4]}" + (f", worst relative distance {worst:.4f}" if plain else ""))
    return worst


if __name__ == "__main__":
    main()
