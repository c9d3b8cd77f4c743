"""tl_kv_append where cu_seqlens is wrong in places: every sequence whose rows are in order and nobody else's comes out
right, and the wrong ones are reported.  Every access is bounded in the kernel, whatever the entries say."""
import numpy as np
import pytest
import torch

from oracle import kv_cache as ora
from tests.kv_cases import Batch, f64, tables

pytestmark = pytest.mark.gpu
Q, LENS = [300, 3, 20, 33, 4], [310, 50, 20, 170, 7]  # cu = 0 300 303 323 356 360


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


# which entry, its value, the sequences that stay right.  (Where an entry gives rows to two sequences, the first has them.)
BAD = [(2, 100000, (0, 3, 4)), (2, -5, (0, 3, 4)), (2, 10, (0, 3, 4)), (2, 360, (0,)), (3, 301, (0, 1, 4)),
       (0, -1, (1, 2, 3, 4)), (5, 361, (0, 1, 2, 3)), (1, 2147483647, (2, 3, 4)), (4, -2147483648, (0, 1, 2)),
       (5, 0, (0, 1, 2, 3))]


@pytest.mark.parametrize("entry,value,good", BAD)
@pytest.mark.parametrize("ps,max_q_len,more", [(16, 0, 0), (64, 300, 0), (16, 0, 200)])
def test_the_other_sequences_come_out_right(B, entry, value, good, ps, max_q_len, more):
    # `more` sequences of one token behind them: the bad entry is one of many threads' to find
    b = Batch(Q + [1] * more, LENS + [5] * more, H=4, Hkv=2, D=128, ps=ps, seed=51)
    good = list(good) + list(range(6 if entry == 5 else 5, 5 + more))
    if value == 360 and more:
        good = [0] + list(range(5, 5 + more))
    if value == 361 and more:
        pytest.skip("in order there")
    kc, ks = b.random_codes()
    vc, vs = b.random_codes()
    rows = b.bf16(b.n, b.H + 2 * b.Hkv, b.D)
    cos, sin = tables(320, 128)
    x = f64(rows)
    cu, lens, table = b.device()
    cu[entry] = value
    d = rows.cuda()
    q_out = torch.full((b.n, b.H, b.D), 7.0, dtype=torch.bfloat16, device="cuda")
    cache = B.KvCache(torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), torch.from_numpy(ks).cuda(),
                      torch.from_numpy(vs).cuda())
    sig = B.Signals(1)
    B.tl_kv_append(cache, d[:, b.H:b.H + b.Hkv], d[:, b.H + b.Hkv:], cu, lens, table, sig, q=d[:, :b.H], q_out=q_out,
                   cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda(), max_q_len=max_q_len)
    code, where = B.tl_query_status(sig)
    assert code == B.TL_ERR_INVALID and where not in good
    got_k, got_v, got_ks, got_vs = (t.cpu().numpy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale))
    out = f64(q_out)
    for s in good:
        r = slice(b.cu[s], b.cu[s + 1])
        pos = range(b.lens[s] - b.q[s], b.lens[s])
        turned = np.stack([ora.rotate(x[t, :b.H + b.Hkv], p, cos, sin, False) for t, p in zip(range(r.start, r.stop), pos)])
        one = ([0, b.q[s]], [b.lens[s]], b.table[s:s + 1])
        pages = b.table[s][:-(-b.lens[s] // ps)]
        for name, new, codes, scales, gc, gs in (("k", turned[:, b.H:], kc, ks, got_k, got_ks),
                                                 ("v", x[r, b.H + b.Hkv:], vc, vs, got_v, got_vs)):
            wc, ws = ora.append(codes, scales, new, *one)
            assert np.array_equal(gc[pages], wc[pages]) and np.array_equal(gs[pages], ws[pages]), (s, name)
        # fp32 products and sum (2^-23 of the two terms), then one bf16 rounding; a step of it next to a border
        want, mag = turned[:, :b.H], np.abs(x).max()
        assert (np.abs(out[r] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * mag).all(), s
    sig.close()
