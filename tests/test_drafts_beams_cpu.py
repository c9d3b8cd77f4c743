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
