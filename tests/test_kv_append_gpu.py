"""tl_kv_append against the float64 oracle: codes and scale bytes bit for bit, queries to one rounding."""
import numpy as np
import pytest
import torch

from tests.kv_cases import Batch, f64, tables
from oracle import kv_cache as ora

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


def run_append(B, b, *, rot, interleaved, scale=1.0, spread=3, max_q_len=0, edit=None, with_q=True, fused=True,
               times=1):
    kc, ks = b.random_codes(spread)
    vc, vs = b.random_codes(spread)
    rows = b.bf16(b.n, b.H + 2 * b.Hkv, b.D, scale=scale)
    if edit:
        edit(rows)
    cos, sin = tables(max(b.lens + [1]), rot) if rot else (None, None)
    dk, dv = b.both(kc, vc)
    dks, dvs = torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda()
    cache = B.KvCache(dk, dv, dks, dvs)
    sig = B.Signals(1)
    d = rows.cuda()
    q, k, v = d[:, :b.H], d[:, b.H:b.H + b.Hkv], d[:, b.H + b.Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q_out = torch.full((b.n, b.H, b.D), 7.0, dtype=torch.bfloat16, device="cuda")
    dc = None if cos is None else torch.from_numpy(cos).cuda()
    ds = None if sin is None else torch.from_numpy(sin).cuda()
    for _ in range(times):
        B.tl_kv_append(cache, k, v, *b.device(), sig, q=q if with_q else None, q_out=q_out if with_q else None, cos=dc,
                       sin=ds, interleaved=interleaved, max_q_len=max_q_len)
    assert B.tl_query_status(sig)[0] == 0
    x = f64(rows)
    pos = np.concatenate([np.arange(n - m, n) for m, n in zip(b.q, b.lens)]).astype(int) if b.n else []
    if rot:
        x = np.stack([np.concatenate([ora.rotate(x[t, :b.H + b.Hkv], p, cos, sin, interleaved), x[t, b.H + b.Hkv:]])
                      for t, p in enumerate(pos)]) if b.n else x
    want = ora.append(kc, ks, x[:, b.H:b.H + b.Hkv], b.cu, b.lens, b.table) + \
        ora.append(vc, vs, x[:, b.H + b.Hkv:], b.cu, b.lens, b.table)
    got = (dk.cpu().numpy(), dks.cpu().numpy(), dv.cpu().numpy(), dvs.cpu().numpy())
    for name, g, w in zip(("k", "k scale", "v", "v scale"), got, want):
        assert np.array_equal(g, w), (name, int((g != w).sum()), np.argwhere(g != w)[:4].tolist())
    if with_q:
        # fp32 products and sum (2^-23 of the two terms), then one bf16 rounding; a step of it next to a border
        w, mag = x[:, :b.H], np.abs(f64(rows)).max() if b.n else 0.0
        assert (np.abs(f64(q_out) - w) <= 2.0 ** -8 * np.abs(w) + 2.0 ** -22 * mag).all()
    else:
        assert (q_out == 7.0).all()
    sig.close()


LAYOUTS = [dict(H=4, Hkv=2, D=128, ps=64), dict(H=3, Hkv=3, D=64, ps=16), dict(H=8, Hkv=1, D=128, ps=16),
           dict(H=1, Hkv=1, D=64, ps=256), dict(H=6, Hkv=2, D=128, ps=48)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rot,interleaved", [("all", False), ("all", True), (32, False), (16, True), (0, False)])
def test_ragged_batch(B, layout, rot, interleaved):
    b = Batch([1, 0, 70, 5, 1, 33, 300], [1, 9, 70, 37, 256, 97, 411], seed=1, **layout)
    run_append(B, b, rot=layout["D"] if rot == "all" else rot, interleaved=interleaved)


@pytest.mark.parametrize("layout", LAYOUTS[:3])
@pytest.mark.parametrize("order", ["hnd", "nhd", "kv"])
def test_single_tokens(B, layout, order):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200] * 3
    b = Batch([1] * len(lens), lens, seed=2, order=order, **layout)
    run_append(B, b, rot=layout["D"], interleaved=False, fused=order != "kv")


@pytest.mark.parametrize("max_q_len", [0, 1, 4, 1000])
def test_the_hint_changes_nothing(B, max_q_len):
    b = Batch([3, 1, 40], [3, 65, 200], seed=3, extra_columns=3, **LAYOUTS[0])
    run_append(B, b, rot=128, interleaved=False, max_q_len=max_q_len)


@pytest.mark.parametrize("scale", [1e-30, 1e-4, 30.0, 1e30])
def test_scales_grow_and_old_codes_move(B, scale):
    # old blocks around 2^-6; new rows far below (scale byte kept), and far above (every old code becomes 0)
    b = Batch([1, 3, 20, 64], [40, 70, 90, 100], seed=4, **LAYOUTS[0])
    run_append(B, b, rot=128, interleaved=False, scale=scale, spread=5)


@pytest.mark.parametrize("step", [0, 1, 2, 3, 4, 5, 8, 12])
def test_recoding_by_small_shifts(B, step):
    # one element sets the block's need to exactly 2^step above the old scales
    def edit(rows):
        rows *= 0.01
        rows[:, :, 5] = 448.0 * 2.0 ** (121 + step - 127)
    b = Batch([1, 2], [60, 33], seed=5, **LAYOUTS[0])
    run_append(B, b, rot=0, interleaved=False, spread=0, edit=edit)


def test_called_again_gives_the_same(B):
    b = Batch([1, 20, 7], [64, 90, 7], seed=6, **LAYOUTS[0])
    run_append(B, b, rot=128, interleaved=False, scale=20.0, times=3)


def test_values_at_rounding_borders(B):
    """bf16 values half-way between two codes, and rotations by angles whose products land next to them."""
    def edit(rows):
        n, h, d = rows.shape
        m = torch.arange(n * h * d).reshape(n, h, d) % 128
        rows.copy_(((1 + m.float() / 128) * 2.0 ** ((m % 7) - 3).float()).to(torch.bfloat16))
    b = Batch([64, 3], [64, 67], seed=7, **LAYOUTS[0])
    run_append(B, b, rot=0, interleaved=False, edit=edit)
    b = Batch([64, 3], [64, 67], seed=7, **LAYOUTS[0])
    run_append(B, b, rot=64, interleaved=True, edit=edit)


def test_zeros_infinities_and_nan(B):
    def edit(rows):
        rows[0] = 0.0
        rows[1, :, 3] = float("inf")
        rows[1, :, 4] = float("-inf")
        rows[2, :, 9] = float("nan")
        rows[3] = float("inf")
    b = Batch([1, 1, 1, 1, 1, 2], [1, 20, 33, 5, 64, 66], seed=8, **LAYOUTS[0])
    run_append(B, b, rot=0, interleaved=False, edit=edit, with_q=False)


def test_far_positions_and_no_queries(B):
    b = Batch([2, 1], [5000, 4097], seed=9, H=1, Hkv=1, D=64, ps=32)
    run_append(B, b, rot=64, interleaved=False)
    b = Batch([5], [9], seed=10, H=2, Hkv=2, D=64, ps=32)
    run_append(B, b, rot=64, interleaved=False, with_q=False)


def test_many_sequences(B):
    rng = np.random.default_rng(11)
    lens = rng.integers(1, 90, 700).tolist()
    b = Batch([1 if i % 5 else 0 for i in range(700)], lens, seed=11, H=2, Hkv=2, D=64, ps=16)
    run_append(B, b, rot=64, interleaved=False)


@pytest.mark.parametrize("what", ["page", "page negative", "length", "cu", "position"])
def test_bad_batches_are_reported_and_stay_inside(B, what):
    """What the arrays get wrong is skipped and recorded; the other sequences come out right.  Every access is
    bounded by checks in the kernel (the page against the pool, the length against the table's row, rows
    against n_tokens, positions against max_pos), so nothing here reaches memory outside."""
    b = Batch([2, 3, 4], [10, 20, 40], seed=12, **LAYOUTS[0])
    kc, ks = b.random_codes()
    vc, vs = b.random_codes()
    rows = b.bf16(b.n, b.Hkv, b.D)
    cu, lens, table = b.device()
    cos, sin = (torch.from_numpy(t).cuda() for t in tables(12 if what == "position" else 64, 128))
    if what == "page":
        table[1, 0] = b.pages
    elif what == "page negative":
        table[1, 0] = -5
    elif what == "length":
        lens[1] = 64 * b.cols + 1
    elif what == "cu":
        cu[2] = 100
    cache = B.KvCache(*(b.pool(c) for c in (kc, vc)), torch.from_numpy(ks).cuda(), torch.from_numpy(vs).cuda())
    sig = B.Signals(1)
    B.tl_kv_append(cache, rows.cuda(), rows.cuda(), cu, lens, table, sig, cos=cos, sin=sin)
    code, where = B.tl_query_status(sig)
    assert code == B.TL_ERR_INVALID and where in (1, 2)
    x = f64(rows)
    c, s = tables(64, 128)
    first = np.stack([ora.rotate(x[t], 8 + t, c, s, False) for t in range(2)])
    want, wscale = ora.append(kc, ks, np.concatenate([first, x[2:]]), [0, 2], [10], b.table[:1])
    page = b.table[0, 0]
    assert np.array_equal(cache.k[page].cpu().numpy(), want[page])
    assert np.array_equal(cache.k_scale[page].cpu().numpy(), wscale[page])
    sig.close()


def test_on_another_stream_and_in_a_graph(B):
    b = Batch([1] * 4, [5, 64, 65, 3], seed=13, **LAYOUTS[0])
    kc, ks = b.random_codes()
    rows = b.bf16(b.n, b.Hkv, b.D)
    want = ora.append(kc, ks, f64(rows), b.cu, b.lens, b.table)
    args = b.device()
    sig = B.Signals(1)
    d = rows.cuda()
    make = lambda: B.KvCache(b.pool(kc), b.pool(kc), torch.from_numpy(ks).cuda(), torch.from_numpy(ks).cuda())
    side = torch.cuda.Stream()
    cache = make()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.tl_kv_append(cache, d, d, *args, sig)
    side.synchronize()
    assert np.array_equal(cache.v.cpu().numpy(), want[0])
    cache = make()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.tl_kv_append(cache, d, d, *args, sig)
    assert np.array_equal(cache.k.cpu().numpy(), kc)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(cache.k.cpu().numpy(), want[0]) and np.array_equal(cache.k_scale.cpu().numpy(), want[1])
    sig.close()
