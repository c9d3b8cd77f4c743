"""Argument checks of the calls for drafts and beams that need no device."""
import ctypes

import pytest

from tests.test_serving_cpu import CACHE_ERRORS, append_args, cache


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from tile_centric_gemm_gb300 import binding
    return binding


def flat(s):
    for f, _ in s._fields_:
        v = getattr(s, f)
        if isinstance(v, ctypes.Structure):
            yield from flat(v)
        else:
            yield ctypes.cast(v, ctypes.c_void_p).value if isinstance(v, ctypes._Pointer) else v


def check_packed(fmt, cls, floats=()):
    n = len(list(flat(cls())))
    want = [float(i + 1) if i in floats else i + 1 for i in range(n)]
    assert list(flat(cls.from_buffer_copy(fmt.pack(*want)))) == want


# ------------------------------------------------------------------ append with norms
def norm_args(L, c=None, **kw):
    a = dict(q_weight=128, k_weight=160, positions=4, eps=1e-6, reserved0=0)
    inner = {k: v for k, v in kw.items() if k not in a}
    a.update({k: v for k, v in kw.items() if k in a})
    return L.tl_kv_append_norm_args(append=append_args(L, c, **inner), **a)


@pytest.mark.parametrize("kw,code", [
    (dict(n_tokens=-1), 1), (dict(B=0), 1), (dict(q=None), 1), (dict(rot_dim=8), 4), (dict(k=20), 1), (dict(signals=None), 1),
    (dict(q_out=48), 1), (dict(q_weight=24), 1), (dict(k_weight=8), 1), (dict(positions=6), 1), (dict(eps=0.0), 1),
    (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(eps=1e-13), 1),
    (dict(H=0, q=None, q_out=None), 1)])
def test_append_norm_refuses(B, kw, code):
    assert B.lib.tl_kv_append_norm(ctypes.byref(norm_args(B, **kw)), None) == code, kw
    assert "tl_kv_append_norm" in B.tl_last_error()


@pytest.mark.parametrize("kw,code", CACHE_ERRORS)
def test_append_norm_refuses_a_bad_cache(B, kw, code):
    assert B.lib.tl_kv_append_norm(ctypes.byref(norm_args(B, cache(B, **kw))), None) == code, kw


def test_append_norm_null_and_nothing_to_do(B):
    assert B.lib.tl_kv_append_norm(None, None) == B.TL_ERR_INVALID
    a = norm_args(B, n_tokens=0, k=None, v=None, q=None, q_out=None)
    assert B.lib.tl_kv_append_norm(ctypes.byref(a), None) == 0


def test_append_norm_packed_arguments_are_the_structure(B):
    n = len(list(flat(B.tl_kv_append_norm_args())))
    check_packed(B._APPEND_NORM, B.tl_kv_append_norm_args, floats=[n - 2])


# ------------------------------------------------------------------ attention of a tree
def tree_args(L, c=None, **kw):
    from tests.test_serving_cpu import attn_args
    a = dict(tree=4, tree_words=2, reserved0=0)
    inner = {"causal": 0, **{k: v for k, v in kw.items() if k not in a}}
    a.update({k: v for k, v in kw.items() if k in a})
    return L.tl_kv_tree_attn_args(attn=attn_args(L, c, **inner), **a)


@pytest.mark.parametrize("kw,code", [
    (dict(n_tokens=-1), 1), (dict(H=3), 1), (dict(causal=1), 1), (dict(scale=-1.0), 1), (dict(q=None), 1), (dict(out=24), 1),
    (dict(workspace=None), 1), (dict(tree=None), 1), (dict(tree=6), 1), (dict(tree_words=0), 4), (dict(tree_words=-3), 4),
    (dict(tree_words=257), 4)])
def test_tree_attention_refuses(B, kw, code):
    assert B.lib.tl_kv_tree_attn(ctypes.byref(tree_args(B, **kw)), None) == code, kw
    assert "tl_kv_tree_attn" in B.tl_last_error()


def test_tree_attention_null_and_nothing_to_do(B):
    assert B.lib.tl_kv_tree_attn(None, None) == B.TL_ERR_INVALID
    assert B.lib.tl_kv_tree_attn(ctypes.byref(tree_args(B, n_tokens=0, q=None, out=None, workspace=None, tree=None)), None) == 0


def test_tree_attention_packed_arguments_are_the_structure(B):
    check_packed(B._TREE, B.tl_kv_tree_attn_args, floats=[6])


# ------------------------------------------------------------------ pages
def fork_args(L, **kw):
    a = dict(B_in=4, B_out=6, max_pages=8, page_size=32, num_pages=100, reserved0=0, page_table=4096, seq_lens=8192, refs=16384,
             parents=4, page_table_out=32768, seq_lens_out=65536, refs_out=16384, copies=4, n_copies=4, workspace=256,
             workspace_bytes=1 << 20, signals=64)
    a.update(kw)
    return L.tl_kv_fork_args(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(B_in=0), 1), (dict(B_out=0), 1), (dict(B_out=1 << 21), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1),
    (dict(page_size=8), 4), (dict(page_size=40), 4), (dict(page_size=512), 4), (dict(max_pages=1 << 28), 4),
    (dict(page_table=None), 1), (dict(seq_lens=None), 1), (dict(refs=None), 1), (dict(parents=None), 1),
    (dict(page_table_out=None), 1), (dict(seq_lens_out=None), 1), (dict(refs_out=None), 1), (dict(copies=None), 1),
    (dict(n_copies=None), 1), (dict(workspace=None), 1), (dict(signals=None), 1), (dict(refs=16388), 1), (dict(workspace=260), 1),
    (dict(workspace_bytes=64), 1), (dict(page_table_out=4096 + 64), 1), (dict(page_table_out=4096 - 64), 1),
    (dict(seq_lens_out=8192), 1), (dict(refs_out=16384 + 16), 1)])
def test_fork_refuses(B, kw, code):
    assert B.lib.tl_kv_fork(ctypes.byref(fork_args(B, **kw)), None) == code, kw
    assert "tl_kv_fork" in B.tl_last_error()


def resize_args(L, **kw):
    a = dict(B=4, max_pages=8, page_size=32, num_pages=100, page_table=4096, seq_lens=8192, new_lens=8192, refs=16384,
             refs_out=16384, workspace=256, workspace_bytes=1 << 20, signals=64)
    a.update(kw)
    return L.tl_kv_resize_args(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1), (dict(page_size=8), 4), (dict(page_table=None), 1),
    (dict(seq_lens=None), 1), (dict(new_lens=None), 1), (dict(refs=None), 1), (dict(refs_out=None), 1), (dict(workspace=None), 1),
    (dict(signals=None), 1), (dict(refs=16388), 1), (dict(workspace=260), 1), (dict(workspace_bytes=64), 1),
    (dict(refs_out=16384 + 396), 1)])
def test_resize_refuses(B, kw, code):
    assert B.lib.tl_kv_resize(ctypes.byref(resize_args(B, **kw)), None) == code, kw
    assert "tl_kv_resize" in B.tl_last_error()


def layers(L, n=2, **kw):
    return (L.tl_kv_cache * n)(*[cache(L, **(kw if i == n - 1 else {})) for i in range(n)])


def test_copy_pages_refuses(B):
    def call(caches, code, **kw):
        a = dict(n_layers=2, n=3, caches=ctypes.addressof(caches) if caches else None, src=4, dst=8, slots=None, count=None, signals=64)
        a.update(kw)
        assert B.lib.tl_kv_copy_pages(ctypes.byref(B.tl_kv_copy_pages_args(**a)), None) == code, kw
        assert code == 0 or "tl_kv_copy_pages" in B.tl_last_error()
    good = layers(B)
    for kw in (dict(n=-1), dict(n_layers=0), dict(src=None), dict(dst=None), dict(signals=None)):
        call(good, 1, **kw)
    call(good, 4, n_layers=5000)
    call(None, 1)
    call(good, 0, n=0, src=None, dst=None)
    for kw, code in CACHE_ERRORS:
        call(layers(B, **kw), code)
    for kw in (dict(num_pages=5), dict(page_size=32), dict(H_kv=1), dict(head_dim=64), dict(token_stride=256)):
        call(layers(B, **kw), 1)  # not laid out as the first
    assert B.lib.tl_kv_copy_pages(None, None) == 1


def test_compact_refuses(B):
    def call(caches, code, **kw):
        a = dict(n_layers=2, B=3, max_pages=4, max_kept=5, caches=ctypes.addressof(caches) if caches else None, kept=4, n_kept=4,
                 cu_seqlens=4, seq_lens=4096, page_table=4, seq_lens_out=8192, signals=64)
        a.update(kw)
        assert B.lib.tl_kv_compact(ctypes.byref(B.tl_kv_compact_args(**a)), None) == code, kw
        assert "tl_kv_compact" in B.tl_last_error()
    good = layers(B)
    for kw in (dict(B=0), dict(max_pages=0), dict(max_kept=0), dict(n_layers=0), dict(kept=None), dict(n_kept=None),
               dict(cu_seqlens=None), dict(seq_lens=None), dict(page_table=None), dict(seq_lens_out=None), dict(signals=None),
               dict(seq_lens_out=4100)):
        call(good, 1, **kw)
    call(None, 1)
    for kw, code in CACHE_ERRORS:
        call(layers(B, **kw), code)
    assert B.lib.tl_kv_compact(None, None) == 1


def test_page_calls_packed_arguments_and_sizes(B):
    for fmt, cls in ((B._FORK, B.tl_kv_fork_args), (B._RESIZE, B.tl_kv_resize_args), (B._COPY_PAGES, B.tl_kv_copy_pages_args),
                     (B._COMPACT, B.tl_kv_compact_args)):
        check_packed(fmt, cls)
    assert B.tl_kv_fork_workspace_size(4, 6) >= 4 * (2 * 4 + 6) and B.tl_kv_resize_workspace_size(1000) >= 4000
    assert not any(B.tl_kv_fork_workspace_size(*a) for a in ((0, 1), (1, 0), (-1, 4), (1 << 21, 1)))
    assert not B.tl_kv_resize_workspace_size(0) and not B.tl_kv_resize_workspace_size(1 << 21)


# ------------------------------------------------------------------ the oracle
def test_oracle_fork_and_resize_by_hand():
    import numpy as np
    from oracle import kv_pages
    table = np.array([[4, 2, 0], [4, 5, 1]], np.int32)
    lens, refs = np.array([20, 40], np.int32), np.array([0, 1, 1, 0, 2, 1, 0], np.int32)
    out, n, new, copies = kv_pages.fork(table, lens, refs, [0, 0, -1, 1], 16, np.full((4, 3), -1, np.int32))
    assert out.tolist() == [[4, 2, -1], [4, 0, -1], [-1, -1, -1], [4, 5, 1]] and n.tolist() == [20, 20, 0, 40]
    assert copies == [(2, 0, 4)] and new.tolist() == [1, 1, 1, 0, 3, 1, 0]
    t, r = kv_pages.resize(table, lens, [33, 16], refs, 16)
    assert t.tolist() == [[4, 2, 0], [4, 5, 1]] and r.tolist() == [1, 0, 1, 0, 2, 0, 0]


def test_oracle_compact_by_hand():
    import numpy as np
    from oracle import kv_pages
    codes = np.zeros((2, 1, 16, 64), np.uint8)
    codes[0, 0, 14:16, 0], codes[1, 0, :3, 0] = [0x38, 0x40], [0x48, 0x38, 0x50]  # 1, 2; 4, 1, 8
    scales = np.array([[127], [129]], np.uint8)
    c, s, n = kv_pages.compact(codes, scales, [[1, 3]], [0, 4], [19], np.array([[0, 1]]))  # tokens 15..18: keep 16, 18
    assert n.tolist() == [17] and s.ravel().tolist() == [129, 129]
    assert c[0, 0, 14, 0] == 0x28 and c[0, 0, 15, 0] == 0x48 and c[1, 0, 0, 0] == 0x50  # 1/4 of 2^2; 4; 8


# ------------------------------------------------------------------ beam selection
def beam_args(L, **kw):
    a = dict(B=2, K=4, N=8, V=1000, dtype=0, eos=-1, history_stride=0, length=0, row_stride=1000, logits=4, scores=4096, done=None,
             parents=4, tokens=4, scores_out=8192, done_out=None, lse=None, history=None, history_out=None, workspace=256,
             workspace_bytes=1 << 24)
    a.update(kw)
    return L.tl_beam_select_args(**a)


HIST = dict(history=1 << 20, history_out=1 << 22, history_stride=10)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 1), (dict(B=20000), 4), (dict(K=0), 1), (dict(K=65), 4), (dict(N=0), 1), (dict(N=65), 4), (dict(V=0), 1),
    (dict(V=1 << 30, row_stride=1 << 30), 4), (dict(dtype=2), 1), (dict(row_stride=999), 1), (dict(eos=1000), 1), (dict(eos=-2), 1),
    (dict(done=1 << 16), 1), (dict(logits=None), 1), (dict(scores=None), 1), (dict(parents=None), 1), (dict(tokens=None), 1),
    (dict(scores_out=None), 1), (dict(workspace=None), 1), (dict(logits=6), 1), (dict(logits=5, dtype=1), 1),
    (dict(workspace=264), 1), (dict(workspace_bytes=1000), 1), (dict(scores_out=4096), 1), (dict(scores_out=4096 - 4), 1),
    (dict(done=1 << 16, done_out=(1 << 16) + 4, eos=1), 1), (dict(history=1 << 20), 1), (dict(HIST, length=10), 1),
    (dict(HIST, length=-1), 1), (dict(HIST, history_out=(1 << 20) + 40), 1)])
def test_beam_select_refuses(B, kw, code):
    assert B.lib.tl_beam_select(ctypes.byref(beam_args(B, **kw)), None) == code, kw
    assert "tl_beam_select" in B.tl_last_error()


def test_beam_select_null_sizes_and_nothing_to_do(B):
    assert B.lib.tl_beam_select(None, None) == 1
    assert B.lib.tl_beam_select(ctypes.byref(beam_args(B, B=0, logits=None, workspace=None)), None) == 0
    check_packed(B._BEAM, B.tl_beam_select_args)
    size = B.tl_beam_select_workspace_size
    assert 0 < size(1, 1, 1, 1) < size(64, 8, 16, 50001) <= size(64, 8, 64, 50001)
    assert not any(size(*a) for a in ((0, 1, 1, 1), (20000, 1, 1, 1), (1, 65, 1, 1), (1, 1, 65, 1), (1, 1, 1, 0), (1, 64, 1, 1 << 26)))


def test_oracle_beams_by_hand():
    import numpy as np
    from oracle import beam
    x = np.log(np.array([[[0.5, 0.25, 0.25], [0.1, 0.8, 0.1]], [[1.0, 1.0, 1.0], [np.nan, 1.0, 1.0]]]))
    total, lse = beam.totals(x, np.array([[0.0, -1.0], [0.0, 5.0]]), None, -1)
    assert np.allclose(lse[0], 0) and np.isclose(lse[1, 0], np.log(3)) and np.isnan(lse[1, 1])
    best = beam.select(total, 4)
    assert [b[:2] for b in best[0]] == [(0, 0), (1, 1), (0, 1), (0, 2)] and np.isclose(best[0][1][2], np.log(0.8) - 1)
    assert [b[:2] for b in best[1]] == [(0, 0), (0, 1), (0, 2), (-1, -1)]
    total, lse = beam.totals(x[:1], np.array([[-0.5, -1.0]]), np.array([[1, 0]]), 2)
    assert [b[:2] for b in beam.select(total, 2)[0]] == [(0, 2), (1, 1)] and lse[0, 0] == 0
