"""tl_kv_append into a page whose scale byte is 255 (NaN): it stays NaN, as the definition's max(need, byte before) says."""
import numpy as np
import pytest
import torch

from oracle import kv_cache as ora
from tests.kv_cases import Batch, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


@pytest.mark.parametrize("scale", [1.0, 1e37])
@pytest.mark.parametrize("q,lens", [([1, 3, 1], [40, 66, 64]), ([40, 70, 64], [45, 130, 129])])
def test_a_nan_block_stays_nan(B, q, lens, scale):
    b = Batch(q, lens, H=4, Hkv=2, D=128, ps=64, seed=61)
    kc, ks = b.random_codes()
    vc, vs = b.random_codes()
    for s in range(len(q)):
        first = b.table[s, (lens[s] - q[s]) // 64]
        ks[first, 0], vs[first, 1] = 255, 255
    rows = b.bf16(b.n, 2 * b.Hkv, b.D, scale=scale)
    cache = B.KvCache(torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), torch.from_numpy(ks).cuda(),
                      torch.from_numpy(vs).cuda())
    sig, d = B.Signals(1), rows.cuda()
    args = b.device()
    for _ in range(2):  # and again: the same
        B.tl_kv_append(cache, d[:, :b.Hkv], d[:, b.Hkv:], *args, sig)
        x = f64(rows)
        for new, codes, scales, got, got_s in ((x[:, :b.Hkv], kc, ks, cache.k, cache.k_scale),
                                               (x[:, b.Hkv:], vc, vs, cache.v, cache.v_scale)):
            want, want_s = ora.append(codes, scales, new, b.cu, b.lens, b.table)
            assert np.array_equal(got_s.cpu().numpy(), want_s)
            assert np.array_equal(got.cpu().numpy(), want)
    query = b.bf16(b.n, b.H, b.D).cuda()
    out = torch.zeros_like(query)
    ws = torch.zeros(B.tl_kv_attn_workspace_size(b.n, len(q), b.H, b.Hkv, b.D), dtype=torch.uint8, device="cuda")
    B.tl_kv_attn(query, cache, out, *args, ws, sig)
    assert B.tl_query_status(sig)[0] == 0
    out = f64(out)
    assert np.isnan(out).all()  # every new token sees the page where the new ones begin, which held older ones
    sig.close()
