"""What the calls for drafts and beams are measured on: appending normed and rotated keys to the 8-bit paged key/value cache
(tl_kv_append_norm), attention of a tree of drafts over it (tl_kv_tree_attn), its pages shared, copied, compacted and freed
(tl_kv_fork, tl_kv_copy_pages, tl_kv_compact, tl_kv_resize) and beam search's selection (tl_beam_select).

``run`` is one pass: with ``own`` false the operators' plain form (elementary torch operations in 32 bits, 64 where a value
is rounded or compared next to a border), with ``own`` true the library's calls.  ``exact`` is each operator's definition in
64 bits.

Cache format: float8 e4m3 codes [page, kv head, token in page, dim] and one E8M0 scale byte b for each page and kv head,
keys and values apart; the value is code * 2^(b-127).  Lengths, page tables, trees and parents go by the case alone (from a
generator of the case's own sizes), values by the seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
THETA = 500000.0
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    layer = dict(H=32, Hkv=8, D=128, page=64)   # the grouped-head layout of the attention benchmark
    norm = dict(op="norm", rot=128, interleaved=False, **layer)
    tree = dict(op="tree", **layer)
    pool = dict(Hkv=8, D=128)
    return [
        # one user's next token: nothing but latency
        dict(norm, name="norm_1", B=1, q=1, ctx=1000, ragged=False, drafts=False),
        # a batch's drafted trees, rotated by their depth
        dict(norm, name="norm_tree", B=32, q=60, ctx=2000, ragged=True, drafts=True),
        # a long prompt's chunk into an empty cache
        dict(norm, name="norm_prompt", B=1, q=8192, ctx=8192, ragged=False, drafts=False),
        # one user's small tree of drafts over a medium context: latency again
        dict(tree, name="tree_1", B=1, q=26, ctx=4099, ragged=False),
        # a batch's large trees in mid-conversation
        dict(tree, name="tree_16", B=16, q=64, ctx=6001, ragged=True),
        # many users' few drafts; small pages and heads, three queries to a key
        dict(tree, name="tree_96", B=96, q=5, ctx=3500, ragged=True, H=12, Hkv=4, D=64, page=16),
        # one user's four beams: part-filled pages copied in every layer
        dict(pool, op="fork", name="fork_4", B=1, K=4, prompt=900, ctx=1000, page=64, layers=16),
        # many users' beams
        dict(pool, op="fork", name="fork_512", B=64, K=8, prompt=700, ctx=911, page=32, layers=4),
        # one user's accepted drafts
        dict(pool, op="compact", name="compact_1", B=1, q=26, ctx=4099, page=64, layers=16, ragged=False),
        # a batch's accepted drafts
        dict(pool, op="compact", name="compact_64", B=64, q=60, ctx=1000, page=64, layers=8, ragged=True),
        # one user's beams over a small vocabulary
        dict(op="beam", name="beam_1", B=1, K=4, N=8, V=32000, half=True, done=False),
        # many users' beams over an odd vocabulary, some of them ended
        dict(op="beam", name="beam_64", B=64, K=8, N=16, V=50001, half=False, done=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["norm", "tree", "tree", "fork", "compact", "beam"])
    if op == "beam":
        V = _log(rng, 500, 140000)
        K = rng.choice([1, 2, 3, 4, 5, 8, 16])
        return dict(op=op, B=_log(rng, 1, max(1, min(64, 64 * 8 * 50001 // (K * V)))), K=K, N=rng.choice([K, 2 * K]), V=V,
                    half=rng.random() < 0.5, done=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 4, 8])
    pool = dict(Hkv=Hkv, D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]))
    if op == "fork":
        B, K = _log(rng, 1, 64), rng.choice([2, 3, 4, 5, 8])
        prompt = _log(rng, 1, 700)
        return dict(op=op, B=B, K=K, prompt=prompt, ctx=prompt + _log(rng, 1, 200), layers=rng.choice([1, 2, 4]), **pool)
    if op == "compact":
        B, q = _log(rng, 1, 64), _log(rng, 1, 120)
        return dict(op=op, B=B, q=q, ctx=q + _log(rng, 1, 900), layers=rng.choice([1, 2, 4, 8]), ragged=rng.random() < 0.7, **pool)
    layout = dict(H=Hkv * rng.choice([1, 2, 3, 4, 8]), ragged=rng.random() < 0.7, **pool)
    if op == "norm":
        B, D = _log(rng, 1, 256), layout["D"]
        drafts = rng.random() < 0.5
        q = _log(rng, 1, min(8192 // B, 128 if drafts else 8192))
        ctx = min(q + _log(rng, 1, 4096), max(q, 400000 // B))
        return dict(op=op, B=B, q=q, ctx=ctx, rot=rng.choice([D, D, D // 2, 0]), interleaved=rng.random() < 0.5, drafts=drafts,
                    **layout)
    B, q = _log(rng, 1, 96), _log(rng, 1, 128)
    ctx = _log(rng, 16, min(30000, 16 * 64 * 32 * 6001 // (B * q * layout["H"]), 400000 // B))
    return dict(op=op, B=B, q=q, ctx=max(q, ctx), **layout)


def _lengths(c):
    """(new tokens, length with them) of each sequence."""
    r = random.Random(c["B"] * 1000003 + c["q"] * 1009 + c["ctx"])
    if not c["ragged"]:
        return [c["q"]] * c["B"], [c["ctx"]] * c["B"]
    q = [c["q"]] + [r.randint(max(1, c["q"] // 2), c["q"]) for _ in range(c["B"] - 1)]
    n = [c["ctx"]] + [r.randint(c["ctx"] // 2, c["ctx"]) for _ in range(c["B"] - 1)]
    return q, [max(a, b) for a, b in zip(q, n)]


def _trees(c):
    """Each sequence's drafts as a tree: for each token its parent among them (-1: the last token before them)."""
    r = random.Random(c["B"] * 31 + c["q"])
    return [[-1 if i == 0 else r.randint(max(-1, i - 7), i - 1) for i in range(n)] for n in _lengths(c)[0]]


def _kept(c):
    """The drafts that each sequence accepts: a path from a root, in order."""
    r = random.Random(c["B"] + 7 * c["q"])
    out = []
    for tree in _trees(c):
        path = [r.randrange(len(tree))]
        while tree[path[-1]] >= 0:
            path.append(tree[path[-1]])
        out.append(path[::-1])
    return out


def _beams(c):
    """Beams' lengths, page tables, how many hold each page, and each new beam's parent.

    A user's beams share the prompt's full pages; what came after lies in pages of their own, some of them shared by two."""
    r = random.Random(c["B"] * 1009 + c["K"] * 13 + c["ctx"])
    ps, table, lens, at = c["page"], [], [], 0
    refs = []
    for _ in range(c["B"]):
        n = c["ctx"] - (r.randint(0, c["page"]) if c["B"] > 1 else 0)
        n = max(n, c["prompt"], 1)
        shared = list(range(at, at + c["prompt"] // ps))
        at += len(shared)
        refs += [c["K"]] * len(shared)
        last = None
        for k in range(c["K"]):
            more = -(-n // ps) - len(shared)
            mine = list(range(at, at + more))
            if last and more > 1 and r.random() < 0.4:  # all but the last page with the beam before
                mine = last[:-1] + [at]
                for p in mine[:-1]:
                    refs[p] += 1
            at += sum(p >= at for p in mine)
            refs += [1] * (at - len(refs))
            table.append(shared + mine)
            lens.append(n)
            last = mine
    rows = c["B"] * c["K"]
    pages = at + rows + 5  # room for every beam's part-filled page, and more
    order = list(range(pages))
    r.shuffle(order)
    held = [0] * pages
    for p, n in enumerate(refs):
        held[order[p]] = n
    width = max(len(t) for t in table) + 2
    table = [[order[p] for p in t] + [-1] * (width - len(t)) for t in table]
    parents = []
    for b in range(c["B"]):
        parents += [b * c["K"] + min(r.randrange(c["K"]), r.randrange(c["K"])) for _ in range(c["K"])]
    return lens, table, held, parents


def _forked(c):
    """What fork makes of _beams, row by row: tables, lengths, holders, and (from, to, filled slots) of each copy."""
    lens, table, held, parents = _beams(c)
    ps = c["page"]
    free = [p for p, n in enumerate(held) if n == 0]
    out, copies, seen = [], [], set()
    refs = list(held)
    for t, n in zip(table, lens):
        for p in t[:-(-n // ps)]:
            refs[p] -= 1
    for b in parents:
        row, n = list(table[b]), lens[b]
        if n % ps:
            if b in seen or held[row[n // ps]] != 1:
                copies.append((row[n // ps], free[len(copies)], n % ps))
                row[n // ps] = copies[-1][1]
            seen.add(b)
        for p in row[:-(-n // ps)]:
            refs[p] += 1
        out.append(row)
    return out, [lens[b] for b in parents], refs, copies


def work(c):
    if c["op"] == "beam":
        ended = sum(_ended(c))
        rows = c["B"] * c["K"]
        e = 2 if c["half"] else 4
        return {"bytes": float((rows - ended) * c["V"] * e + rows * 9 + c["B"] * c["N"] * 13), "flops": 3.0 * (rows - ended) * c["V"]}
    Hkv, D, ps = c["Hkv"], c["D"], c["page"]
    if c["op"] == "fork":
        lens, _, held, _ = _beams(c)
        copies = _forked(c)[3]
        moved = sum(n for _, _, n in copies) * Hkv * D * 2 + len(copies) * Hkv * 2
        entries = 2 * sum(-(-n // ps) for n in lens)
        return {"bytes": float(2 * moved * c["layers"] + 4 * entries + 8 * len(held) + 12 * len(lens) + 24 * len(copies)),
                "flops": 0.0}
    q, n = _lengths(c)
    if c["op"] == "compact":
        kept = _kept(c)
        moved = sum(i != k for path in kept for i, k in enumerate(path)) * Hkv * D * 2
        pages = sum(-(-b // ps) for b in n)
        return {"bytes": float(2 * moved * c["layers"] + 8 * pages + sum(map(len, kept)) * 4 + 16 * c["B"]), "flops": 0.0}
    H = c["H"]
    if c["op"] == "norm":
        per = 2 * Hkv * D * (2 + 1) + H * D * (2 + 2) + c["rot"] * 4 + (4 if c["drafts"] else 0)
        return {"bytes": float(sum(q) * per + c["B"] * 8 + 4 * D), "flops": sum(q) * (H + Hkv) * (4.0 * D + 3.0 * c["rot"])}
    seen = sum(a * (b - a) + _seen(t) for a, b, t in zip(q, n, _trees(c)))
    pages = sum(-(-b // ps) for b in n)
    words = -(-c["q"] // 32)
    return {"bytes": float(sum(n) * Hkv * D * 2 + pages * (4 + 2 * Hkv) + sum(q) * (H * (D * 4 + 4) + 4 * words)),
            "flops": 4.0 * H * D * seen}


def _depths(tree):
    d = []
    for p in tree:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _seen(tree):
    return sum(_depths(tree)) + len(tree)


def _masks(tree, words):
    """For each token the tokens on its path, itself included, as bits of `words` signed 32-bit numbers."""
    m = []
    for i, p in enumerate(tree):
        m.append((m[p] if p >= 0 else 0) | 1 << i)
    return [[((x >> 32 * w & 0xFFFFFFFF) ^ 0x80000000) - 0x80000000 for w in range(words)] for x in m]


def _ended(c):
    r = random.Random(c["B"] * 100 + c["K"])
    return [c["done"] and r.random() < 0.15 for _ in range(c["B"] * c["K"])]


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
    """Codes and scales of a pool that is full: rows of N(0, 1) in every head, some pages, heads and dims larger."""
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


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _layers(s, g, c, pages):
    """The layers' caches: codes [layer, page, ...] and scales, each layer's values its own."""
    parts = [_random_cache(g, c, pages * c["layers"]) for _ in range(2)]
    for name, (codes, scales) in zip("kv", parts):
        s[name], s[name + "s"] = codes.unflatten(0, (c["layers"], pages)), scales.unflatten(0, (c["layers"], pages))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    s = {"case": c}
    if c["op"] == "beam":
        B, K, N, V = c["B"], c["K"], c["N"], c["V"]
        x = torch.randn(B * K, V, generator=g, device="cuda") * 2.5
        s["logits"] = x.to(torch.bfloat16) if c["half"] else x
        s["scores"] = -20.0 * torch.rand(B, K, generator=g, device="cuda")
        s["done"] = torch.tensor(_ended(c), device="cuda").view(B, K).to(torch.uint8) if c["done"] else None
        s["parents"], s["tokens"] = (torch.empty(B, N, dtype=torch.int32, device="cuda") for _ in range(2))
        s["scores_out"] = torch.empty(B, N, device="cuda")
        s["lse"] = torch.zeros(B, K, device="cuda")
        if own:
            from tile_centric_gemm_gb300 import binding as L
            s["ws"] = torch.zeros(L.tl_beam_select_workspace_size(B, K, N, V), dtype=torch.uint8, device="cuda")
        return s
    if c["op"] == "fork":
        lens, table, held, parents = _beams(c)
        s["lens"], s["table"], s["refs"], s["parents"] = _i32(lens), _i32(table), _i32(held), _i32(parents)
        s["lens_out"], s["table_out"], s["refs_out"] = _i32(lens), _i32(table), _i32(held)
        s["copies"], s["count"] = torch.zeros(3, len(lens), dtype=torch.int32, device="cuda"), _i32([0])
        _layers(s, g, c, len(held))
        if own:
            from tile_centric_gemm_gb300 import binding as L
            s["signals"] = L.Signals(1)
            s["caches"] = L.KvLayers([L.KvCache(*t) for t in zip(s["k"], s["v"], s["ks"], s["vs"])])
            s["ws"] = torch.zeros(L.tl_kv_fork_workspace_size(len(lens), len(lens)), dtype=torch.uint8, device="cuda")
        return s
    q, n = _lengths(c)
    D, ps, nB, N = c["D"], c["page"], c["B"], sum(q)
    need = [-(-b // ps) for b in n]
    order = list(range(sum(need)))
    random.Random(sum(need)).shuffle(order)  # the pages of a sequence lie anywhere in the pool
    table, at = [], 0
    for k in need:
        table.append(order[at:at + k] + [0] * (max(need) - k))
        at += k
    s["cu"] = _i32([sum(q[:b]) for b in range(nB + 1)])
    s["lens"], s["table"] = _i32(n), _i32(table)
    s["qmax"] = c["q"]
    if c["op"] == "compact":
        kept = _kept(c)
        s["kept"] = _i32([path + [0] * (c["q"] - len(path)) for path in kept])
        s["n_kept"] = _i32([len(path) for path in kept])
        s["lens_out"] = _i32([0] * nB)
        s["refs"], s["refs_out"] = _i32([1] * sum(need)), _i32([1] * sum(need))
        s["table_out"] = s["table"].clone()
        _layers(s, g, c, sum(need))
        if own:
            from tile_centric_gemm_gb300 import binding as L
            s["signals"] = L.Signals(1)
            s["caches"] = L.KvLayers([L.KvCache(*t) for t in zip(s["k"], s["v"], s["ks"], s["vs"])])
            s["ws"] = torch.zeros(L.tl_kv_resize_workspace_size(nB), dtype=torch.uint8, device="cuda")
        return s
    H, Hkv = c["H"], c["Hkv"]
    s["k"], s["ks"] = _random_cache(g, c, sum(need))
    s["v"], s["vs"] = _random_cache(g, c, sum(need))
    if c["op"] == "norm":
        # one row of the fused projection for each new token: queries, keys, values; some tokens larger than the rest
        rows = torch.randn(N, H + 2 * Hkv, D, generator=g, device="cuda")
        rows *= torch.exp(0.5 * torch.randn(N, 1, 1, generator=g, device="cuda"))
        rows = rows.to(torch.bfloat16)
        s["q_new"], s["k_new"], s["v_new"] = rows[:, :H], rows[:, H:H + Hkv], rows[:, H + Hkv:]
        s["q_out"] = torch.empty(N, H, D, dtype=torch.bfloat16, device="cuda")
        s["q_weight"], s["k_weight"] = (torch.exp(0.3 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
        s["cos"] = s["sin"] = s["positions"] = None
        if c["rot"]:
            f = THETA ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
            a = torch.arange(max(n), dtype=torch.float64, device="cuda")[:, None] * f
            s["cos"], s["sin"] = a.cos().float(), a.sin().float()
        if c["drafts"]:
            s["positions"] = _i32([b - a + d for a, b, t in zip(q, n, _trees(c)) for d in _depths(t)])
    else:
        s["q_new"] = _bf16(g, N, H, D, scale=1.5)
        s["out"] = torch.empty(N, H, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(H, N, dtype=torch.float32, device="cuda")
        s["tree"] = _i32([m for t in _trees(c) for m in _masks(t, -(-c["q"] // 32))])
    if own:
        from tile_centric_gemm_gb300 import binding as L
        s["cache"] = L.KvCache(s["k"], s["v"], s["ks"], s["vs"])
        s["signals"] = L.Signals(1)
        if c["op"] == "tree":
            s["ws"] = torch.zeros(L.tl_kv_attn_workspace_size(N, nB, H, Hkv, D), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    return {"norm": _norm, "tree": _tree, "fork": _fork, "compact": _compact, "beam": _beam}[s["case"]["op"]](s)


def _run_own(s):
    from tile_centric_gemm_gb300 import binding as L
    c = s["case"]
    if c["op"] == "norm":
        L.tl_kv_append_norm(s["cache"], s["k_new"], s["v_new"], s["cu"], s["lens"], s["table"], s["signals"], q=s["q_new"],
                            q_out=s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, cos=s["cos"], sin=s["sin"],
                            positions=s["positions"], interleaved=c["interleaved"], max_q_len=s["qmax"])
        return {**_cache_out(s), "q": s["q_out"]}
    if c["op"] == "tree":
        L.tl_kv_tree_attn(s["q_new"], s["cache"], s["out"], s["cu"], s["lens"], s["table"], s["tree"], s["ws"], s["signals"],
                          max_q_len=s["qmax"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "fork":
        L.tl_kv_fork(s["table"], s["lens"], s["refs"], s["parents"], s["table_out"], s["lens_out"], s["refs_out"], s["copies"],
                     s["count"], s["ws"], s["signals"], page_size=c["page"])
        L.tl_kv_copy_pages(s["caches"], s["copies"][0], s["copies"][1], s["signals"], slots=s["copies"][2], count=s["count"])
        return _fork_out(s)
    if c["op"] == "compact":
        L.tl_kv_compact(s["caches"], s["kept"], s["n_kept"], s["cu"], s["lens"], s["table"], s["lens_out"], s["signals"])
        L.tl_kv_resize(s["table_out"], s["lens"], s["lens_out"], s["refs"], s["refs_out"], s["ws"], s["signals"], page_size=c["page"])
        return {**_cache_out(s), "lens": s["lens_out"], "refs": s["refs_out"], "table": s["table_out"]}
    L.tl_beam_select(s["logits"], s["scores"], s["parents"], s["tokens"], s["scores_out"], s["ws"], done=s["done"],
                     eos=2 if c["done"] else -1, lse=s["lse"])
    return {"parents": s["parents"], "tokens": s["tokens"], "scores": s["scores_out"], "lse": s["lse"]}


def _cache_out(s):
    """The cache's codes as the e4m3 values they are, and its scale bytes."""
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "ks": s["ks"], "vs": s["vs"]}


def _fork_out(s):
    return {**_cache_out(s), "table": s["table_out"], "lens": s["lens_out"], "refs": s["refs_out"], "copies": s["copies"],
            "count": s["count"]}


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


def _normed(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _norm(s):
    c = s["case"]
    b, _, pos, start = _tokens(s)
    v = s["v_new"].double()
    k = _normed(s["k_new"].double(), s["k_weight"].double())  # 64 bits: the codes are decided next to borders
    q = _normed(s["q_new"].float(), s["q_weight"].float())
    if s["cos"] is not None:
        at = pos if s["positions"] is None else s["positions"].long()
        cos, sin = s["cos"][at], s["sin"][at]
        k = _rotate(k, cos.double(), sin.double(), c["interleaved"])
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

    def put(x, codes, scales):
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

    put(k, s["k"], s["ks"])
    put(v, s["v"], s["vs"])
    return {**_cache_out(s), "q": s["q_out"]}


def _values(codes, scales, table):
    """The cache's values for each sequence: [sequence, kv head, token, dim], in 32 bits."""
    x = codes[table].view(torch.float8_e4m3fn).float()
    x = x * _pow2(scales[table].long()[..., None, None] - 127).float()
    nB, np_, hk, ps, d = x.shape
    return x.transpose(1, 2).reshape(nB, hk, np_ * ps, d)


def _tree(s):
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
    j = key - start[:, None]  # a key's number among its sequence's drafts
    bits = torch.zeros(nB, Q, s["tree"].shape[1], dtype=torch.int64, device="cuda")
    bits[b, i] = s["tree"].long()
    word = bits.gather(2, (j.clamp(0, Q - 1) // 32)[:, None].expand(nB, Q, -1))
    sees = (j < 0)[:, None] | ((word >> (j.clamp(0, Q - 1) % 32)[:, None]) & 1 == 1) & (key < lens[:, None])[:, None]
    w.masked_fill_(~sees[:, None, None], -math.inf)
    m = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    l = w.sum(-1, keepdim=True)
    v = _values(s["v"], s["vs"], table)
    o = torch.matmul(w.view(nB, Hkv, -1, w.shape[-1]), v).view(nB, Hkv, H // Hkv, Q, D) / l.clamp(min=1e-38)
    out = o.permute(0, 3, 1, 2, 4).reshape(nB, Q, H, D)[b, i].to(torch.bfloat16)
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(nB, Q, H)[b, i].t().contiguous()
    return {"out": out, "lse": lse}


def _holders(refs, table, lens, ps, sign):
    """refs with `sign` added for each page that a row of the table holds."""
    held = torch.arange(table.shape[1], device="cuda") < (lens[:, None] + ps - 1) // ps
    return refs.index_add(0, table.clamp(min=0).flatten(), held.flatten().to(torch.int32) * sign)


def _fork(s):
    ps, lens, table, parents = s["case"]["page"], s["lens"].long(), s["table"].long(), s["parents"].long()
    rows = torch.arange(len(parents), device="cuda")
    first = torch.full_like(lens, len(parents)).scatter_reduce(0, parents, rows, "amin")
    n, out = lens[parents], table[parents]
    last = out.gather(1, (n // ps)[:, None])[:, 0]
    need = (n % ps > 0) & ((first[parents] != rows) | (s["refs"][last.clamp(min=0)] != 1))
    free = torch.sort((s["refs"] != 0).int(), stable=True).indices  # the free pages come first, in order
    rank = torch.cumsum(need, 0) - 1
    new = free[rank.clamp(min=0)]
    s["table_out"].copy_(torch.where(need[:, None] & (torch.arange(out.shape[1], device="cuda") == (n // ps)[:, None]), new[:, None], out))
    s["lens_out"].copy_(n)
    refs = _holders(s["refs"], table, lens, ps, -1)
    s["refs_out"].copy_(_holders(refs, s["table_out"].long(), n, ps, 1))
    src, dst, slots = last[need], new[need], (n % ps)[need]
    s["copies"][:, :len(src)] = torch.stack([src, dst, slots]).int()
    s["count"].copy_(need.sum()[None])
    filled = (torch.arange(ps, device="cuda") < slots[:, None])[None, :, None, :, None]
    s["k"][:, dst] = torch.where(filled, s["k"][:, src], s["k"][:, dst])
    s["v"][:, dst] = torch.where(filled, s["v"][:, src], s["v"][:, dst])
    s["ks"][:, dst], s["vs"][:, dst] = s["ks"][:, src], s["vs"][:, src]
    return _fork_out(s)


def _compact(s):
    c = s["case"]
    ps, lens, table, cu = c["page"], s["lens"].long(), s["table"].long(), s["cu"].long()
    start, nB, Q = lens - (cu[1:] - cu[:-1]), c["B"], c["q"]
    i = torch.arange(Q, device="cuda")
    valid = i < s["n_kept"][:, None]
    b = torch.arange(nB, device="cuda")[:, None].expand(nB, Q)[valid]
    to, of = (start[:, None] + i)[valid], (start[:, None] + s["kept"].long())[valid]
    to_page, of_page = table[b, to // ps], table[b, of // ps]
    begun = (start % ps > 0).nonzero()[:, 0]  # sequences whose page in work holds earlier tokens
    old_page = table[begun, start[begun] // ps]
    pages = s["k"].shape[1]
    earlier = torch.zeros(pages, dtype=torch.int64, device="cuda").index_add(0, old_page, start[begun] % ps)
    seq_pages = torch.cat([to_page, old_page])

    def move(codes, scales):
        before = scales.long()
        after = torch.zeros_like(before)
        after.index_reduce_(1, to_page, before[:, of_page], "amax")
        after.index_reduce_(1, old_page, before[:, old_page], "amax")
        shift = (before[:, of_page] - after[:, to_page]).transpose(0, 1)[..., None]
        moved = _e4m3(codes[:, of_page, :, of % ps].view(torch.float8_e4m3fn).double() * _pow2(shift))  # [token, layer, head, dim]
        kept = _e4m3(codes[:, old_page].view(torch.float8_e4m3fn).double() * _pow2((before - after)[:, old_page])[..., None, None])
        filled = (torch.arange(ps, device="cuda") < earlier[old_page][:, None])[None, :, None, :, None]
        codes[:, old_page] = torch.where(filled, kept, codes[:, old_page])
        codes[:, to_page, :, to % ps] = moved
        scales[:, seq_pages] = after[:, seq_pages].to(torch.uint8)

    move(s["k"], s["ks"])
    move(s["v"], s["vs"])
    s["lens_out"].copy_(start + s["n_kept"])
    refs = _holders(s["refs"], table, lens, ps, -1)
    s["refs_out"].copy_(_holders(refs, table, s["lens_out"].long(), ps, 1))
    return {**_cache_out(s), "lens": s["lens_out"], "refs": s["refs_out"], "table": s["table_out"]}


def _beam(s):
    c = s["case"]
    B, K, N, V = c["B"], c["K"], c["N"], c["V"]
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    lse = m.double() + (x - m).exp().sum(1, keepdim=True, dtype=torch.float64).log()  # 64 bits: beams are compared by it
    score = s["scores"].double().view(-1, 1) + (x.double() - lse)
    if s["done"] is not None:
        done = s["done"].view(-1, 1) != 0
        score.masked_fill_(done, -math.inf)
        score[:, 2] = torch.where(done[:, 0], s["scores"].double().flatten(), score[:, 2])
        lse = torch.where(done, 0.0, lse)
    top, at = torch.sort(score.view(B, K * V), dim=1, descending=True, stable=True)
    top, at = top[:, :N], at[:, :N]
    some = top > -math.inf
    rows = torch.arange(B, device="cuda")[:, None] * K + at // V
    return {"parents": torch.where(some, rows, -1).int(), "tokens": torch.where(some, at % V, -1).int(), "scores": top.float(),
            "lse": lse.view(B, K).float()}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "tree": _exact_tree, "fork": _exact_fork, "compact": _exact_compact, "beam": _exact_beam}[case["op"]](s, case)


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


def _exact_norm(s, c):
    q_lens, n = _lengths(c)
    ps = c["page"]
    k, v = s["k"].view(torch.float8_e4m3fn).double(), s["v"].view(torch.float8_e4m3fn).double()
    ks, vs = s["ks"].clone(), s["vs"].clone()
    q_out = torch.empty(s["q_new"].shape, dtype=torch.float64, device="cuda")
    tables, trees, at = s["table"].tolist(), _trees(c), 0
    half = c["rot"] // 2

    def turned(x, w, pos):
        x = x.double()
        x = w.double() * x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["D"] + EPS)
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
        if c["drafts"]:
            pos = begin + torch.tensor(_depths(trees[b]), device="cuda")
        rows = slice(at, at + q_lens[b])
        at += q_lens[b]
        q_out[rows] = turned(s["q_new"][rows], s["q_weight"], pos)
        new = (turned(s["k_new"][rows], s["k_weight"], pos), s["v_new"][rows].double())
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


def _exact_tree(s, c):
    q_lens, n = _lengths(c)
    group, at = c["H"] // c["Hkv"], 0
    N = sum(q_lens)
    out = torch.zeros(N, c["H"], c["D"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["H"], N), -math.inf, dtype=torch.float64, device="cuda")
    for b, tree in enumerate(_trees(c)):
        pages = s["table"][b, :-(-n[b] // c["page"])].long()
        paths = []
        for i, p in enumerate(tree):
            paths.append((paths[p] if p >= 0 else set()) | {i})
        sees = torch.ones(len(tree), n[b], dtype=torch.bool)
        sees[:, n[b] - len(tree):] = torch.tensor([[j in p for j in range(len(tree))] for p in paths])
        sees = sees.cuda()
        whole = slice(at, at + len(tree))
        for h in range(c["Hkv"]):
            k = s["k"][pages, h].view(torch.float8_e4m3fn).double() * torch.exp2(s["ks"][pages, h].double() - 127)[:, None, None]
            v = s["v"][pages, h].view(torch.float8_e4m3fn).double() * torch.exp2(s["vs"][pages, h].double() - 127)[:, None, None]
            k, v = k.reshape(-1, c["D"])[:n[b]], v.reshape(-1, c["D"])[:n[b]]
            rows = s["q_new"][whole, h * group:(h + 1) * group].double()
            z = torch.einsum("tgd,nd->gtn", rows, k) / math.sqrt(c["D"])
            z = z.masked_fill(~sees, -math.inf)
            lse[h * group:(h + 1) * group, whole] = torch.logsumexp(z, 2)
            out[whole, h * group:(h + 1) * group] = torch.einsum("gtn,nd->tgd", torch.softmax(z, 2), v)
        at += len(tree)
    return {"out": out, "lse": lse}


def _exact_fork(s, c):
    table, lens, refs, copies = _forked(c)
    k, v = s["k"].view(torch.float8_e4m3fn).double(), s["v"].view(torch.float8_e4m3fn).double()
    ks, vs, listed_copies = s["ks"].clone(), s["vs"].clone(), torch.zeros_like(s["copies"])
    for i, (src, dst, n) in enumerate(copies):
        for x in (k, v):
            x[:, dst, :, :n] = x[:, src, :, :n]
        for x in (ks, vs):
            x[:, dst] = x[:, src]
        listed_copies[:, i] = _i32([src, dst, n])
    return {"k": k, "v": v, "ks": ks, "vs": vs, "table": _i32(table), "lens": _i32(lens), "refs": _i32(refs),
            "copies": listed_copies, "count": _i32([len(copies)])}


def _exact_compact(s, c):
    q_lens, n = _lengths(c)
    ps, tables, new = c["page"], s["table"].tolist(), []
    k, v = s["k"].view(torch.float8_e4m3fn).double(), s["v"].view(torch.float8_e4m3fn).double()
    ks, vs = s["ks"].clone(), s["vs"].clone()
    refs = [1] * s["refs"].numel()
    for b, path in enumerate(_kept(c)):
        start = n[b] - q_lens[b]
        new.append(start + len(path))
        for p in tables[b][-(-new[b] // ps):-(-n[b] // ps)]:
            refs[p] -= 1
        for codes, scales in ((k, ks), (v, vs)):
            rows = [(tables[b][(start + i) // ps], (start + i) % ps) for i in path]
            was = [(codes[:, p, :, r].clone(), scales[:, p].double()) for p, r in rows]
            for j in range(start // ps, (new[b] - 1) // ps + 1):
                p, lo, hi = tables[b][j], max(start, j * ps), min(new[b], (j + 1) * ps)
                into = [was[t - start][1] for t in range(lo, hi)] + ([scales[:, p].double()] if lo > j * ps else [])
                e = torch.stack(into).amax(0)
                old = codes[:, p, :, :lo - j * ps]
                codes[:, p, :, :lo - j * ps] = _exact_e4m3(old * torch.exp2(scales[:, p].double() - e)[..., None, None])
                for t in range(lo, hi):
                    x, b_x = was[t - start]
                    codes[:, p, :, t - j * ps] = _exact_e4m3(x * torch.exp2(b_x - e)[..., None])
                scales[:, p] = e.to(torch.uint8)
    return {"k": k, "v": v, "ks": ks, "vs": vs, "lens": _i32(new), "refs": _i32(refs), "table": s["table"].clone()}


def _exact_beam(s, c):
    B, K, N, V = c["B"], c["K"], c["N"], c["V"]
    parents, tokens = torch.full((2, B, N), -1, dtype=torch.int32, device="cuda")
    scores = torch.full((B, N), -math.inf, dtype=torch.float64, device="cuda")
    lses = torch.zeros(B, K, dtype=torch.float64, device="cuda")
    ended = _ended(c)
    for b in range(B):
        x = s["logits"][b * K:(b + 1) * K].double()
        lse = torch.logsumexp(x, 1)
        total = torch.log_softmax(x, 1) + s["scores"][b].double()[:, None]
        for k in range(K):
            if ended[b * K + k]:
                total[k], lse[k] = -math.inf, 0.0
                total[k, 2] = s["scores"][b, k].double()
        lses[b] = lse
        best, at = torch.topk(total.flatten(), N)
        order = sorted(zip(best.tolist(), at.tolist()), key=lambda p: (-p[0], p[1]))
        parents[b] = _i32([b * K + i // V if x > -math.inf else -1 for x, i in order])
        tokens[b] = _i32([i % V if x > -math.inf else -1 for x, i in order])
        scores[b] = torch.tensor([x for x, _ in order], dtype=torch.float64)
    return {"parents": parents, "tokens": tokens, "scores": scores, "lse": lses}
