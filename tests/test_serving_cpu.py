"""Argument checks of the serving calls (8-bit paged cache, attention over it, experts for a few tokens) that need no device, and the
cache's oracle against torch's own e4m3 and against attention over plain values."""
import ctypes

import numpy as np
import pytest

from oracle import kv_cache as ora


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from tile_centric_gemm_gb300 import binding
    return binding


def cache(B, **kw):
    a = dict(k=4096, v=8192, k_scale=64, v_scale=96, page_stride=8192 * 2, head_stride=8192, token_stride=128,
             num_pages=4, page_size=64, H_kv=2, head_dim=128)
    a.update(kw)
    return B.tl_kv_cache(**a)


CACHE_ERRORS = [(dict(k=None), 1), (dict(v=None), 1), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
                (dict(k=4104), 1), (dict(v=4104), 1), (dict(num_pages=0), 1), (dict(H_kv=0), 1),
                (dict(head_dim=96), 4), (dict(head_dim=0), 4), (dict(page_size=8), 4), (dict(page_size=40), 4),
                (dict(page_size=512), 4), (dict(page_stride=100), 1), (dict(head_stride=-8192), 1),
                (dict(token_stride=64), 1), (dict(token_stride=136), 1), (dict(H_kv=5000), 4)]


def append_args(L, c=None, **kw):
    a = dict(n_tokens=3, B=2, H=4, rot_dim=64, interleaved=0, max_pos=100, max_pages=4, max_q_len=0,
             cache=c or cache(L), k=16, v=32, q=48, k_token_stride=256, k_head_stride=128, v_token_stride=256,
             v_head_stride=128, q_token_stride=512, q_head_stride=128, q_out=64, cos=80, sin=96, cu_seqlens=4,
             seq_lens=4, page_table=4, signals=64)
    a.update(kw)
    return L.tl_kv_append_args(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(n_tokens=-1), 1), (dict(B=0), 1), (dict(B=1 << 21), 1), (dict(max_pages=0), 1), (dict(H=-1), 1),
    (dict(H=0), 1), (dict(q=None), 1), (dict(q_out=None), 1), (dict(rot_dim=-16), 4), (dict(rot_dim=8), 4),
    (dict(rot_dim=144), 4), (dict(interleaved=2), 1), (dict(max_q_len=-1), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(cu_seqlens=None), 1), (dict(seq_lens=None), 1), (dict(page_table=None), 1), (dict(signals=None), 1),
    (dict(cos=None), 1), (dict(sin=None), 1), (dict(max_pos=0), 1), (dict(k=20), 1), (dict(v=20), 1), (dict(q=20), 1),
    (dict(q_out=20), 1), (dict(cos=20), 1), (dict(k_token_stride=4), 1), (dict(v_head_stride=-8), 1),
    (dict(q_token_stride=12), 1)])
def test_append_refuses(B, kw, code):
    a = append_args(B, **kw)
    assert B.lib.tl_kv_append(ctypes.byref(a), None) == code, kw
    assert "tl_kv_append" in B.tl_last_error()


def attn_args(L, c=None, **kw):
    a = dict(n_tokens=3, B=2, H=4, causal=1, max_pages=4, max_q_len=0, scale=0.0, reserved0=0, cache=c or cache(L),
             q=16, q_token_stride=512, q_head_stride=128, out=32, lse=4, cu_seqlens=4, seq_lens=4, page_table=4,
             workspace=256, workspace_bytes=1 << 30, signals=64)
    a.update(kw)
    return L.tl_kv_attn_args(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(n_tokens=-1), 1), (dict(B=0), 1), (dict(max_pages=0), 1), (dict(H=3), 1), (dict(H=0), 1), (dict(causal=2), 1),
    (dict(max_q_len=-2), 1), (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(q=None), 1), (dict(out=None), 1), (dict(workspace=None), 1), (dict(cu_seqlens=None), 1),
    (dict(seq_lens=None), 1), (dict(page_table=None), 1), (dict(signals=None), 1), (dict(q=24), 1), (dict(out=24), 1),
    (dict(workspace=260), 1), (dict(lse=6), 1), (dict(q_token_stride=100), 1), (dict(q_head_stride=-8), 1),
    (dict(n_tokens=1 << 30, H=16), 4)])
def test_attention_refuses(B, kw, code):
    a = attn_args(B, **kw)
    assert B.lib.tl_kv_attn(ctypes.byref(a), None) == code, kw
    assert "tl_kv_attn" in B.tl_last_error()


@pytest.mark.parametrize("kw,code", CACHE_ERRORS)
def test_both_refuse_a_bad_cache(B, kw, code):
    c = cache(B, **kw)
    assert B.lib.tl_kv_append(ctypes.byref(append_args(B, c)), None) == code, kw
    assert B.lib.tl_kv_attn(ctypes.byref(attn_args(B, c, H=c.H_kv or 1)), None) == code, kw


def test_null_and_nothing_to_do(B):
    assert B.lib.tl_kv_append(None, None) == B.TL_ERR_INVALID
    assert B.lib.tl_kv_attn(None, None) == B.TL_ERR_INVALID
    assert B.lib.tl_kv_append(ctypes.byref(append_args(B, n_tokens=0, k=None, v=None, q=None, q_out=None)), None) == 0
    assert B.lib.tl_kv_attn(ctypes.byref(attn_args(B, n_tokens=0, q=None, out=None, workspace=None)), None) == 0


def test_attention_workspace_size(B):
    size = lambda *a: B.tl_kv_attn_workspace_size(*a)
    assert size(1, 1, 32, 8, 128, 152) > 0
    for bad in [(-1, 1, 32, 8, 128, 152), (1, 0, 32, 8, 128, 152), (1, 1, 33, 8, 128, 152), (1, 1, 32, 0, 128, 152),
                (1, 1, 32, 8, 96, 152), (1, 1, 32, 8, 128, -1)]:
        assert size(*bad) == 0
    sizes = [size(n, b, 32, 8, 128, 152) for n, b in [(1, 1), (64, 64), (300, 2), (5000, 2), (5000, 64)]]
    assert sizes == sorted(sizes)


def test_binding_refuses_wrong_tensors(B):
    import torch
    k = torch.zeros(2, 1, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        B.KvCache(k, k, torch.zeros(2, 1, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8))  # not on a GPU


def moe_args(L, **kw):
    import ctypes as ct
    e = kw.get("E", 4)
    ptrs = ct.cast((ct.c_void_p * max(e, 1))(*[16] * max(e, 1)), ct.POINTER(ct.c_void_p))
    a = dict(T=3, H=64, I=32, Hd=64, E=4, topk=2, normalize=1, reserved0=0, x=16, logits=4, W1=ptrs, W2=ptrs, out=32,
             ids=4, gates=8, workspace=256, workspace_bytes=1 << 30)
    a.update(kw)
    return L.tl_moe_decode_args(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(T=65), 4), (dict(H=0), 1), (dict(H=60), 4), (dict(I=12), 4), (dict(Hd=4), 4),
    (dict(E=0), 1), (dict(E=257), 4), (dict(topk=0), 1), (dict(topk=5), 1), (dict(E=32, topk=17), 4),
    (dict(normalize=2), 1), (dict(x=None), 1), (dict(logits=None), 1), (dict(W1=None), 1), (dict(W2=None), 1),
    (dict(out=None), 1), (dict(ids=None), 1), (dict(gates=None), 1), (dict(workspace=None), 1), (dict(x=24), 1),
    (dict(out=40), 1), (dict(workspace=264), 1), (dict(logits=6), 1), (dict(gates=9), 1), (dict(workspace_bytes=4096), 1)])
def test_moe_refuses(B, kw, code):
    a = moe_args(B, **kw)
    assert B.lib.tl_moe_decode(ctypes.byref(a), None) == code, kw
    assert "tl_moe_decode" in B.tl_last_error()


def test_moe_refuses_bad_weight_pointers(B):
    for bad in (None, 24):
        ptrs = ctypes.cast((ctypes.c_void_p * 4)(16, 32, bad, 48), ctypes.POINTER(ctypes.c_void_p))
        for name in ("W1", "W2"):
            assert B.lib.tl_moe_decode(ctypes.byref(moe_args(B, **{name: ptrs})), None) == B.TL_ERR_INVALID
            assert "expert 2" in B.tl_last_error()


def test_moe_null_and_nothing_to_do(B):
    assert B.lib.tl_moe_decode(None, None) == B.TL_ERR_INVALID
    assert B.lib.tl_moe_decode(ctypes.byref(moe_args(B, T=0, x=None, out=None, workspace=None)), None) == 0


def test_moe_workspace_size(B):
    size = B.tl_moe_decode_workspace_size
    assert size(1, 2, 32, 4096, 1408, 4096) >= 2 * (1408 * 4 + 4096 * 4)
    assert size(64, 2, 32, 4096, 1408, 4096) > size(8, 2, 32, 4096, 1408, 4096)
    for bad in [(-1, 2, 8, 64, 64, 64), (65, 2, 8, 64, 64, 64), (1, 9, 8, 64, 64, 64), (1, 2, 8, 60, 64, 64),
                (1, 17, 32, 64, 64, 64), (1, 1, 257, 64, 64, 64)]:
        assert size(*bad) == 0


@pytest.mark.parametrize("name", ["APPEND", "ATTN", "MOE"])
def test_packed_arguments_are_the_structures(B, name):
    fmt = getattr(B, "_" + name)
    cls = {"APPEND": B.tl_kv_append_args, "ATTN": B.tl_kv_attn_args, "MOE": B.tl_moe_decode_args}[name]

    def flat(s):
        for f, _ in s._fields_:
            v = getattr(s, f)
            if isinstance(v, ctypes.Structure):
                yield from flat(v)
            else:
                yield ctypes.cast(v, ctypes.c_void_p).value if isinstance(v, ctypes._Pointer) else v
    n = len(list(flat(cls())))
    want = [float(i + 1) if i == 6 and name == "ATTN" else i + 1 for i in range(n)]
    assert list(flat(cls.from_buffer_copy(fmt.pack(*want)))) == want


# ------------------------------------------------------------------ the oracle
def test_oracle_codes_are_torchs():
    import torch
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ora.TABLE, want, equal_nan=True)
    x = np.random.default_rng(0).standard_normal(5000).astype(np.float32) * 8
    x = np.concatenate([x, (ora.GRID[:-1] + ora.GRID[1:]).astype(np.float32) / 2, [448.0, 464.0, 0.0]]).astype(np.float32)
    got = ora.encode(x)
    ref = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, ref)


def test_oracle_scale_and_recoding_by_hand():
    assert ora.scale_byte(448.0) == 127 and ora.scale_byte(448.5) == 128 and ora.scale_byte(0.0) == 0
    codes = np.zeros((1, 1, 16, 64), np.uint8)
    codes[0, 0, 0, :3] = [0x38, 0x09, 0x03]          # 1, 2^-6 * 9/8, 3 * 2^-9
    scales = np.full((1, 1), 127, np.uint8)
    row = np.zeros((1, 1, 64))
    row[0, 0, 0] = 1792.0                             # needs 2^2
    c, s = ora.append(codes, scales, row, [0, 1], [2], np.zeros((1, 1), np.int32))
    assert s[0, 0] == 129
    # 1/4 exactly; 9 * 2^-9 / 4 = 2.25 steps of 2^-9 -> 2; 3/4 of a step -> 1
    assert c[0, 0, 0, :3].tolist() == [0x28, 0x02, 0x01] and c[0, 0, 1, 0] == 0x7E


def test_oracle_attention_is_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    o, lse = ora.attention(q, k, v, True, 0.5)
    s = np.einsum("ihd,jhd->hij", q, k.repeat(2, 1)) * 0.5
    s[:, np.arange(9)[None, :] > np.arange(6, 9)[:, None]] = -np.inf
    p = np.exp(s)
    assert np.allclose(o, np.einsum("hij,jhd->ihd", p / p.sum(2, keepdims=True), v.repeat(2, 1)), rtol=1e-12)
    assert np.allclose(lse, np.log(p.sum(2)), rtol=1e-12)


def test_oracle_rotation_is_complex_multiplication():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((2, 8))
    a = rng.standard_normal((4, 3))
    cos, sin = np.cos(a), np.sin(a)
    for inter in (False, True):
        first = [0, 2, 4] if inter else [0, 1, 2]
        second = [1, 3, 5] if inter else [3, 4, 5]
        z = (x[:, first] + 1j * x[:, second]) * np.exp(1j * a[2])
        y = ora.rotate(x, 2, cos, sin, inter)
        assert np.allclose(y[:, first], z.real) and np.allclose(y[:, second], z.imag)
        assert np.array_equal(y[:, 6:], x[:, 6:])


def test_oracle_selection():
    from oracle import moe_decode
    l = np.array([[0.0, 2.0, 2.0, -1.0], [np.nan, -np.inf, 1.0, 1.0], [-np.inf] * 4])
    ids, gates = moe_decode.select(l, 3, True)
    assert ids.tolist() == [[1, 2, 0], [2, 3, 1], [0, 1, 2]]
    assert np.allclose(gates[0], np.exp([0, 0, -2]) / np.exp([0, 0, -2]).sum())
    assert np.allclose(gates[1], [0.5, 0.5, 0.0]) and (gates[2] == 0).all()
    assert np.allclose(moe_decode.select(l[:1], 2, False)[1][0], np.exp([0, 0]) / np.exp([-2, 0, 0, -3]).sum())


def test_oracle_layer_by_hand():
    from oracle import moe_decode
    x = np.array([[1.0, 2.0]])
    W1 = [np.array([[1.0, 3.0], [0.5, -1.0]]), np.zeros((2, 2))]
    W2 = [np.array([[2.0, -1.0]]), np.zeros((1, 2))]
    g, u = 2.0, 1.0
    h = g / (1 + np.exp(-g)) * u
    out = moe_decode.layer(x, np.array([[np.log(3.0), 0.0]]), W1, W2, 2, True)[0]
    assert np.allclose(out, 0.75 * h * np.array([[2.0, -1.0]]))
