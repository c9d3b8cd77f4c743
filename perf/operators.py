"""What the serving operators are measured on: appending to the 8-bit paged key/value cache (tl_kv_append), attention over
it (tl_kv_attn) and the mixture-of-experts layer for a few tokens (tl_moe_decode).

``run`` is one pass: with ``own`` false the operators' plain form (elementary torch operations in 32 bits, 64 where a value
is rounded next to a border), with ``own`` true the library's call.  ``exact`` is each operator's definition in 64 bits.

Cache format: float8 e4m3 codes [page, kv head, token in page, dim] and one E8M0 scale byte b for each page and kv head,
keys and values apart; the value is code * 2^(b-127).  Lengths, page tables and positions go by the case alone (they are
ragged, from a generator of the case's own sizes), values by the seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
THETA = 500000.0


# ------------------------------------------------------------------ the cases
def listed():
    layer = dict(H=32, Hkv=8, D=128, page=64)   # the grouped-head layout of the attention benchmark
    append = dict(op="append", rot=128, interleaved=False, **layer)
    attn = dict(op="attn", causal=True, **layer)
    experts = dict(op="moe", hidden=4096, inter=1408, E=32, topk=2, normalize=True)  # the MoE benchmark's layer
    return [
        # one user's next token: nothing but latency
        dict(append, name="append_1", B=1, q=1, ctx=1000, ragged=False),
        # the next token of a full batch
        dict(append, name="append_256", B=256, q=1, ctx=1500, ragged=True),
        # a long prompt's chunk into an empty cache
        dict(append, name="append_prompt", B=1, q=8192, ctx=8192, ragged=False),
        # ragged prompt chunks that begin and end inside pages; small pages and heads, neighbouring pairs, half the dims rotated
        dict(append, name="append_ragged", B=24, q=301, ctx=777, ragged=True, H=12, Hkv=4, D=64, page=16, rot=32,
             interleaved=True),
        # one user's next token over a medium context: latency again
        dict(attn, name="attn_1", B=1, q=1, ctx=4099, ragged=False),
        # the next token of a batch in mid-conversation
        dict(attn, name="attn_64", B=64, q=1, ctx=8192, ragged=True),
        # few users with long documents
        dict(attn, name="attn_long", B=3, q=1, ctx=131072, ragged=True),
        # a draft of four tokens checked for each sequence
        dict(attn, name="attn_draft", B=16, q=4, ctx=6001, ragged=True),
        # a prompt's chunk over what went before
        dict(attn, name="attn_prompt", B=2, q=2048, ctx=12289, ragged=True),
        # one token through the experts: two of 32 are read
        dict(experts, name="moe_1", T=1),
        # a batch's tokens through most of the experts
        dict(experts, name="moe_27", T=27),
        # a full batch: every expert is read, several tokens each; many narrow experts, eight of them to a token
        dict(experts, name="moe_64_top8", T=64, hidden=2048, inter=1000, E=64, topk=8, normalize=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "moe"])
    if op == "moe":
        E = rng.choice([8, 16, 32, 64])
        hidden = 8 * _log(rng, 64, 512)
        inter = 8 * _log(rng, 24, min(176, 32 * 4096 * 1408 // (8 * E * hidden)))
        return dict(op=op, T=_log(rng, 1, 64), hidden=hidden, inter=inter, E=E,
                    topk=rng.choice([k for k in (1, 2, 4, 6, 8) if k <= E]), normalize=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 4, 8])
    layout = dict(Hkv=Hkv, H=Hkv * rng.choice([1, 2, 3, 4, 8]), D=rng.choice([64, 128]),
                  page=rng.choice([16, 32, 64, 128]), ragged=rng.random() < 0.7)
    if op == "append":
        B = _log(rng, 1, 256)
        q = _log(rng, 1, 8192 // B)
        ctx = min(q + _log(rng, 1, 4096), max(q, 400000 // B))
        D = layout["D"]
        return dict(op=op, B=B, q=q, ctx=ctx, rot=rng.choice([D, D, D // 2, 0]), interleaved=rng.random() < 0.5, **layout)
    if rng.random() < 0.6:  # single tokens and drafts
        B = _log(rng, 1, 128)
        q = rng.choice([1, 1, 1, 2, 3, 5])
        ctx = _log(rng, 16, 400000 // B)
    else:  # chunks of prompts
        B = rng.choice([1, 1, 2, 3])
        q = _log(rng, 16, 2048)
        ctx = q + _log(rng, 1, 10000 // B)
    return dict(op=op, B=B, q=q, ctx=max(q, ctx), causal=rng.random() < 0.8, **layout)


def _lengths(c):
    """(new tokens, length with them) of each sequence."""
    r = random.Random(c["B"] * 1000003 + c["q"] * 1009 + c["ctx"])
    if not c["ragged"]:
        return [c["q"]] * c["B"], [c["ctx"]] * c["B"]
    q = [c["q"]] + [r.randint(max(1, c["q"] // 2), c["q"]) for _ in range(c["B"] - 1)]
    n = [c["ctx"]] + [r.randint(c["ctx"] // 2, c["ctx"]) for _ in range(c["B"] - 1)]
    return q, [max(a, b) for a, b in zip(q, n)]


def work(c):
    if c["op"] == "moe":
        T, k, E, h, i = c["T"], c["topk"], c["E"], c["hidden"], c["inter"]
        active = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token chooses, on average
        return {"bytes": active * 3 * h * i * 2 + T * (h * 2 * 2 + E * 4 + k * 8), "flops": 6.0 * T * k * h * i}
    q, n = _lengths(c)
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    if c["op"] == "append":
        per = 2 * Hkv * D * (2 + 1) + H * D * (2 + 2) + c["rot"] * 4
        return {"bytes": float(sum(q) * per + c["B"] * 8), "flops": 3.0 * sum(q) * (H + Hkv) * c["rot"]}
    pairs = sum(a * b - (a * (a - 1) // 2 if c["causal"] else 0) for a, b in zip(q, n))
    pages = sum(-(-b // c["page"]) for b in n)
    return {"bytes": float(sum(n) * Hkv * D * 2 + pages * (4 + 2 * Hkv) + sum(q) * H * (D * 4 + 4)),
            "flops": 4.0 * H * D * pairs}


# ------------------------------------------------------------------ inputs
def _pow2(e):
    """2^e in 64 bits, exactly (ldexp and pow are not exact on every device)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _need(amax):
    """The least scale byte b with amax <= 448 * 2^(b-127)."""
    m, e = torch.frexp(amax)
    b = e.to(torch.int64) - 9 + (m > 0.875).to(torch.int64) + 127
    return torch.where(amax > 0, b, torch.zeros_like(b)).clamp(0, 254)


def _e4m3(x):
    """e4m3 code of each value of x (64 bits), rounded once to nearest even, above 448 to 448."""
    x = x.clamp(-E4M3_MAX, E4M3_MAX)
    _, e = torch.frexp(x)
    step = _pow2(torch.clamp(e - 1, min=-6) - 3)
    return (torch.round(x / step) * step).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


def _random_cache(g, c, pages):
    """Codes and scales of a pool that is full: rows of N(0, 1) in every head, some heads and dims larger."""
    shape = (pages, c["Hkv"], c["page"], c["D"])
    codes, scales = torch.empty(shape, dtype=torch.uint8, device="cuda"), torch.empty(shape[:2], dtype=torch.uint8, device="cuda")
    dims = torch.exp(0.4 * torch.randn(1, c["Hkv"], 1, c["D"], generator=g, device="cuda"))
    step = max(1, (1 << 26) // (c["Hkv"] * c["page"] * c["D"]))
    for p in range(0, pages, step):
        x = torch.randn((min(step, pages - p),) + shape[1:], generator=g, device="cuda") * dims
        b = _need(x.abs().amax((2, 3)))
        codes[p:p + step] = (x * _pow2(127 - b[:, :, None, None]).float()).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[p:p + step] = b.to(torch.uint8)
    return codes, scales


def _bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    s = {"case": c}
    if c["op"] == "moe":
        T, h, i, E = c["T"], c["hidden"], c["inter"], c["E"]
        s["x"] = _bf16(g, T, h)
        s["logits"] = torch.randn(T, E, generator=g, device="cuda")
        s["W1"] = _bf16(g, E, h, 2 * i, scale=h ** -0.5)  # each expert's gate columns, then its up columns
        s["W2"] = _bf16(g, E, i, h, scale=i ** -0.5)
        s["out"] = torch.empty(T, h, dtype=torch.bfloat16, device="cuda")
        s["ids"] = torch.empty(T, c["topk"], dtype=torch.int32, device="cuda")
        s["gates"] = torch.empty(T, c["topk"], dtype=torch.float32, device="cuda")
        if own:
            from tile_centric_gemm_gb300 import binding as B
            s["w"] = B.MoeWeights(list(s["W1"]), list(s["W2"]))
            s["ws"] = torch.zeros(B.tl_moe_decode_workspace_size(T, c["topk"], E, h, i, h), dtype=torch.uint8, device="cuda")
        return s
    q, n = _lengths(c)
    H, Hkv, D, ps, nB, N = c["H"], c["Hkv"], c["D"], c["page"], c["B"], sum(q)
    need = [-(-b // ps) for b in n]
    order = list(range(sum(need)))
    random.Random(sum(need)).shuffle(order)  # the pages of a sequence lie anywhere in the pool
    table, at = [], 0
    for k in need:
        table.append(order[at:at + k] + [0] * (max(need) - k))
        at += k
    s["cu"] = torch.tensor([sum(q[:b]) for b in range(nB + 1)], dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    s["k"], s["ks"] = _random_cache(g, c, sum(need))
    s["v"], s["vs"] = _random_cache(g, c, sum(need))
    s["qmax"] = c["q"]
    if c["op"] == "append":
        # one row of the fused projection for each new token: queries, keys, values; some tokens larger than the rest
        rows = torch.randn(N, H + 2 * Hkv, D, generator=g, device="cuda")
        rows *= torch.exp(0.5 * torch.randn(N, 1, 1, generator=g, device="cuda"))
        rows = rows.to(torch.bfloat16)
        s["q_new"], s["k_new"], s["v_new"] = rows[:, :H], rows[:, H:H + Hkv], rows[:, H + Hkv:]
        s["q_out"] = torch.empty(N, H, D, dtype=torch.bfloat16, device="cuda")
        if c["rot"]:
            f = THETA ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
            a = torch.arange(max(n), dtype=torch.float64, device="cuda")[:, None] * f
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
        else:
            s["cos"] = s["sin"] = None
    else:
        s["q_new"] = _bf16(g, N, H, D, scale=1.5)
        s["out"] = torch.empty(N, H, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(H, N, dtype=torch.float32, device="cuda")
    if own:
        from tile_centric_gemm_gb300 import binding as B
        s["cache"] = B.KvCache(s["k"], s["v"], s["ks"], s["vs"])
        s["signals"] = B.Signals(1)
        if c["op"] == "attn":
            s["ws"] = torch.zeros(B.tl_kv_attn_workspace_size(N, nB, H, Hkv, D), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"append": _append, "attn": _attn, "moe": _moe}[s["case"]["op"]](s)


def _run_own(s):
    from tile_centric_gemm_gb300 import binding as B
    c = s["case"]
    if c["op"] == "append":
        B.tl_kv_append(s["cache"], s["k_new"], s["v_new"], s["cu"], s["lens"], s["table"], s["signals"], q=s["q_new"],
                       q_out=s["q_out"], cos=s["cos"], sin=s["sin"], interleaved=c["interleaved"], max_q_len=s["qmax"])
        return _cache_out(s, s["q_out"])
    if c["op"] == "attn":
        B.tl_kv_attn(s["q_new"], s["cache"], s["out"], s["cu"], s["lens"], s["table"], s["ws"], s["signals"],
                     causal=c["causal"], max_q_len=s["qmax"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    B.tl_moe_decode(s["x"], s["logits"], s["w"], s["out"], s["ids"], s["gates"], s["ws"], normalize=c["normalize"])
    return {"out": s["out"], "ids": s["ids"], "gates": s["gates"]}


def _cache_out(s, q):
    """The cache's codes as the e4m3 values they are, its scale bytes, and the rotated queries."""
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "ks": s["ks"], "vs": s["vs"], "q": q}


def _tokens(s):
    """For every new token its sequence, its number there and its position; for every sequence its first new position."""
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(s["q_new"].shape[0], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    start = lens - (cu[1:] - cu[:-1])
    i = t - cu[b]
    return b, i, start[b] + i, start


def _rotate(x, cos, sin, interleaved):
    """x [tokens, heads, dims] with its first dims rotated; cos, sin [tokens, pairs]."""
    r = 2 * cos.shape[1]
    c, s, y = cos[:, None], sin[:, None], x.clone()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, b * c + a * s
    return y


def _append(s):
    c = s["case"]
    b, _, pos, start = _tokens(s)
    k, v, q = s["k_new"].double(), s["v_new"].double(), s["q_new"].float()
    if s["cos"] is not None:
        cos, sin = s["cos"][pos], s["sin"][pos]
        k = _rotate(k, cos.double(), sin.double(), c["interleaved"])  # 64 bits: the codes are decided next to borders
        q = _rotate(q, cos, sin, c["interleaved"])
    s["q_out"].copy_(q)
    ps, nB = c["page"], c["B"]
    first = start // ps
    span = c["q"] // ps + 2  # pages that a sequence's new tokens can touch
    j = first[:, None] + torch.arange(span, device="cuda")
    touched = j * ps < s["lens"].long()[:, None]
    page = s["table"].long().gather(1, j.clamp(max=s["table"].shape[1] - 1))
    older = (start[:, None] - j * ps).clamp(0, ps)  # slots of the page that were filled before
    cell = b * span + pos // ps - first[b]
    own_page, slot = s["table"].long()[b, pos // ps], pos % ps
    for x, codes, scales in ((k, s["k"], s["ks"]), (v, s["v"], s["vs"])):
        amax = torch.zeros(nB * span, c["Hkv"], dtype=torch.float64, device="cuda")
        amax.index_reduce_(0, cell, x.abs().amax(2), "amax")
        before = torch.where((older > 0)[:, :, None], scales[page].long(), 0)
        after = torch.maximum(before, _need(amax).view(nB, span, -1))
        at = page[touched]
        old = codes[at].view(torch.float8_e4m3fn).double()
        shifted = _e4m3(old * _pow2((before - after)[touched][:, :, None, None]))
        filled = torch.arange(ps, device="cuda") < older[touched][:, None]
        codes[at] = torch.where(filled[:, None, :, None], shifted, codes[at])
        scales[at] = after[touched].to(torch.uint8)
        codes[own_page, :, slot] = _e4m3(x * _pow2(127 - after.view(nB * span, -1)[cell][:, :, None]))
    return _cache_out(s, s["q_out"])


def _values(codes, scales, table):
    """The cache's values for each sequence: [sequence, kv head, token, dim], in 32 bits."""
    x = codes[table].view(torch.float8_e4m3fn).float()
    x = x * _pow2(scales[table].long()[..., None, None] - 127).float()
    nB, np_, hk, ps, d = x.shape
    return x.transpose(1, 2).reshape(nB, hk, np_ * ps, d)


def _attn(s):
    c = s["case"]
    b, i, _, start = _tokens(s)
    lens, table = s["lens"].long(), s["table"].long()
    nB, Q, H, Hkv, D = c["B"], c["q"], c["H"], c["Hkv"], c["D"]
    q = torch.zeros(nB, Q, H, D, device="cuda")
    q[b, i] = s["q_new"].float()
    q = q.view(nB, Q, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(nB, Hkv, -1, D)
    k = _values(s["k"], s["ks"], table)
    w = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(nB, Hkv, H // Hkv, Q, -1)
    del k
    key = torch.arange(w.shape[-1], device="cuda")
    end = lens[:, None].expand(nB, Q)
    if c["causal"]:
        end = torch.minimum(end, start[:, None] + torch.arange(Q, device="cuda") + 1)
    w.masked_fill_((key >= end[:, :, None])[:, None, None], -math.inf)
    m = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    l = w.sum(-1, keepdim=True)
    v = _values(s["v"], s["vs"], table)
    o = torch.matmul(w.view(nB, Hkv, -1, w.shape[-1]), v).view(nB, Hkv, H // Hkv, Q, D) / l.clamp(min=1e-38)
    out = o.permute(0, 3, 1, 2, 4).reshape(nB, Q, H, D)[b, i].to(torch.bfloat16)
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(nB, Q, H)[b, i].t().contiguous()
    return {"out": out, "lse": lse}


def _moe(s):
    c = s["case"]
    x, T, E, i = s["x"].float(), c["T"], c["E"], c["inter"]
    top, ids = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    top, ids = top[:, :c["topk"]], ids[:, :c["topk"]]
    full = s["logits"] if not c["normalize"] else top
    m = full.amax(1, keepdim=True)
    gates = (top - m).exp() / (full - m).exp().sum(1, keepdim=True)
    weight = torch.zeros(T, E, device="cuda").scatter_(1, ids, gates)
    h = torch.matmul(x, s["W1"].float())  # [E, T, 2 inter]
    h = h[..., :i] / (1.0 + (-h[..., :i]).exp()) * h[..., i:]
    y = torch.matmul(h, s["W2"].float())
    out = (y * weight.t()[:, :, None]).sum(0).to(torch.bfloat16)
    return {"out": out, "ids": ids.int(), "gates": gates}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "moe": _exact_moe}[case["op"]](s, case)


def _exact_e4m3(x):
    """The e4m3 number nearest to each x, ties to the even code: by a search among the 127 magnitudes."""
    grid = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    a = x.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 126)
    lo = hi - 1
    up = a - grid[lo]
    down = grid[hi] - a
    pick = torch.where((up > down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[pick], x)


def _exact_append(s, c):
    q_lens, n = _lengths(c)
    ps = c["page"]
    k, v = s["k"].view(torch.float8_e4m3fn).double(), s["v"].view(torch.float8_e4m3fn).double()
    ks, vs = s["ks"].clone(), s["vs"].clone()
    q_out = s["q_new"].double().clone()
    tables, at = s["table"].tolist(), 0
    half = c["rot"] // 2

    def turned(x, pos):
        if not half:
            return x
        first = [2 * d for d in range(half)] if c["interleaved"] else list(range(half))
        second = [d + (1 if c["interleaved"] else half) for d in first]
        z = torch.complex(x[..., first], x[..., second]) * torch.complex(s["cos"][pos].double(), s["sin"][pos].double())[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    for b in range(c["B"]):
        begin, end = n[b] - q_lens[b], n[b]
        pos = torch.arange(begin, end, device="cuda")
        rows = slice(at, at + q_lens[b])
        at += q_lens[b]
        q_out[rows] = turned(s["q_new"][rows].double(), pos)
        new = (turned(s["k_new"][rows].double(), pos), s["v_new"][rows].double())
        for j in range(begin // ps, (end - 1) // ps + 1):
            lo, hi, p = max(begin, j * ps), min(end, (j + 1) * ps), tables[b][j]
            for x, codes, scales in ((new[0], k, ks), (new[1], v, vs)):
                part = x[lo - begin:hi - begin].transpose(0, 1)  # [kv head, token, dim]
                amax = part.abs().amax((1, 2))
                need = torch.ceil(torch.log2(amax.clamp(min=1e-30) / E4M3_MAX)).clamp(-127, 127)
                need = torch.where(amax > E4M3_MAX * torch.exp2(need), need + 1, need)
                need = torch.where(amax <= E4M3_MAX * torch.exp2(need - 1), need - 1, need).clamp(-127, 127)
                old = scales[p].double() - 127 if lo > j * ps else torch.full_like(need, -127.0)
                e = torch.maximum(need, old)
                codes[p, :, :lo - j * ps] = _exact_e4m3(codes[p, :, :lo - j * ps] * torch.exp2(old - e)[:, None, None])
                codes[p, :, lo - j * ps:hi - j * ps] = _exact_e4m3(part * torch.exp2(-e)[:, None, None])
                scales[p] = (e + 127).to(torch.uint8)
    return {"k": k, "v": v, "ks": ks, "vs": vs, "q": q_out}


def _exact_attn(s, c):
    q_lens, n = _lengths(c)
    group, at = c["H"] // c["Hkv"], 0
    N = sum(q_lens)
    out = torch.zeros(N, c["H"], c["D"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["H"], N), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        pages = s["table"][b, :-(-n[b] // c["page"])].long()
        for h in range(c["Hkv"]):
            k = s["k"][pages, h].view(torch.float8_e4m3fn).double() * torch.exp2(s["ks"][pages, h].double() - 127)[:, None, None]
            v = s["v"][pages, h].view(torch.float8_e4m3fn).double() * torch.exp2(s["vs"][pages, h].double() - 127)[:, None, None]
            k, v = k.reshape(-1, c["D"])[:n[b]], v.reshape(-1, c["D"])[:n[b]]
            for t in range(0, q_lens[b], 512):
                rows = s["q_new"][at + t:at + min(t + 512, q_lens[b]), h * group:(h + 1) * group].double()
                z = torch.einsum("tgd,nd->gtn", rows, k) / math.sqrt(c["D"])
                if c["causal"]:
                    last = n[b] - q_lens[b] + t + torch.arange(rows.shape[0], device="cuda")
                    z = z.masked_fill(torch.arange(n[b], device="cuda") > last[:, None], -math.inf)
                whole = slice(at + t, at + t + rows.shape[0])
                lse[h * group:(h + 1) * group, whole] = torch.logsumexp(z, 2)
                out[whole, h * group:(h + 1) * group] = torch.einsum("gtn,nd->tgd", torch.softmax(z, 2), v)
        at += q_lens[b]
    return {"out": out, "lse": lse}


def _exact_moe(s, c):
    logits = s["logits"].double()
    ids = torch.empty(c["T"], c["topk"], dtype=torch.int64, device="cuda")
    left = logits.clone()
    for j in range(c["topk"]):
        ids[:, j] = torch.max(left, 1).indices
        left.scatter_(1, ids[:, j:j + 1], -math.inf)
    gates = torch.softmax(logits, 1).gather(1, ids)
    if c["normalize"]:
        gates = gates / gates.sum(1, keepdim=True)
    out = torch.zeros(c["T"], c["hidden"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            z = s["x"][t].double() @ s["W1"][e].double()
            z = torch.nn.functional.silu(z[:, :c["inter"]]) * z[:, c["inter"]:]
            out.index_add_(0, t, gates[t, j][:, None] * (z @ s["W2"][e].double()))
    return {"out": out, "ids": ids.int(), "gates": gates}
