"""Thin ctypes binding over libtilelink.so with the C ABI's names.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Importing this module loads the library and fails loudly when it is
missing (build it with ``python -m tile_centric_gemm_gb300.build``); there is
no fallback.  Tensors are torch tensors on the device the call runs on; the
stream is torch's current stream unless one is given.
"""
from __future__ import annotations

import ctypes
import os
import struct

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libtilelink.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libtilelink.so not built: {_LIB_PATH} (run python -m tile_centric_gemm_gb300.build)")

lib = ctypes.CDLL(_LIB_PATH)

TL_OK, TL_ERR_INVALID, TL_ERR_CUDA, TL_ERR_TIMEOUT, TL_ERR_UNSUPPORTED, TL_ERR_INTERNAL = range(6)
TL_MODE_PULL, TL_MODE_PUSH = 0, 1
TL_SWIZZLE_ARRIVAL, TL_SWIZZLE_ROWS = 0, 1
TL_RS_BF16_PARTIALS, TL_RS_RING_ORDER = 1, 2
TL_LL_FLAG_IN_DATA, TL_LL_SEPARATE_FLAG = 0, 1
STATUS_NAMES = {0: "TL_OK", 1: "TL_ERR_INVALID", 2: "TL_ERR_CUDA", 3: "TL_ERR_TIMEOUT",
                4: "TL_ERR_UNSUPPORTED", 5: "TL_ERR_INTERNAL"}

# Every symbol the header declares; tests check that the library exports all of them.
EXPORTED = [
    "tl_version", "tl_last_error", "tl_signals_create", "tl_signals_destroy", "tl_signals_flags",
    "tl_signals_reset", "tl_tile_notify", "tl_tile_wait", "tl_query_status",
    "tl_gemm_workspace_size", "tl_gemm", "tl_ag_gemm_workspace_size", "tl_ag_gemm_num_flags",
    "tl_ag_gemm_tile_order", "tl_ag_gemm",
    "tl_gemm_rs_workspace_size", "tl_gemm_rs_num_flags", "tl_gemm_rs", "tl_gemm_rs_noalloc",
    "tl_moe_workspace_size", "tl_moe_num_flags", "tl_moe_ag_gemm", "tl_allgather", "tl_reduce_scatter",
    "tl_moe_down_workspace_size", "tl_moe_down_num_flags", "tl_moe_down",
    "tl_ag_attn_num_flags", "tl_ag_attn", "tl_allgather_ll_link_bytes", "tl_allgather_ll",
    "tl_test_hold_chunks",
    "tl_kv_append", "tl_kv_append_norm", "tl_kv_attn_workspace_size", "tl_kv_attn", "tl_kv_tree_attn",
    "tl_kv_fork_workspace_size", "tl_kv_fork", "tl_kv_resize_workspace_size", "tl_kv_resize", "tl_kv_copy_pages", "tl_kv_compact",
    "tl_beam_select_workspace_size", "tl_beam_select", "tl_moe_decode_workspace_size", "tl_moe_decode",
]


class TLError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


_vp = ctypes.c_void_p


class tl_ag_gemm_args(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("self_rank", ctypes.c_int32), ("M_shard", ctypes.c_int32),
        ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("mode", ctypes.c_int32),
        ("rows_per_barrier", ctypes.c_int32), ("swizzle", ctypes.c_int32),
        ("A_shards", ctypes.POINTER(_vp)), ("B", _vp), ("gathered", _vp), ("C", _vp), ("C_f32", _vp),
        ("signals", _vp), ("src_ready", _vp),
        ("epoch", ctypes.c_uint32), ("reserved1", ctypes.c_uint32),
        ("timeout_ns", ctypes.c_uint64), ("trace", _vp),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class tl_ag_attn_args(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("self_rank", ctypes.c_int32), ("S_shard", ctypes.c_int32),
        ("H", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("causal", ctypes.c_int32), ("scale", ctypes.c_float),
        ("Q", _vp), ("K_shards", ctypes.POINTER(_vp)), ("V_shards", ctypes.POINTER(_vp)),
        ("K_gathered", _vp), ("V_gathered", _vp), ("O", _vp), ("lse", _vp), ("signals", _vp),
        ("epoch", ctypes.c_uint32), ("reserved0", ctypes.c_uint32), ("timeout_ns", ctypes.c_uint64),
    ]


class tl_gemm_args(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("reserved0", ctypes.c_int32),
        ("A", _vp), ("B", _vp), ("C", _vp), ("C_f32", _vp), ("signals", _vp), ("timeout_ns", ctypes.c_uint64),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


class tl_gemm_rs_args(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("M", ctypes.c_int32), ("K_r", ctypes.c_int32), ("N", ctypes.c_int32),
        ("A", ctypes.POINTER(_vp)), ("B", ctypes.POINTER(_vp)), ("out", ctypes.POINTER(_vp)),
        ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("signals", _vp),
        ("epoch", ctypes.c_uint32), ("options", ctypes.c_uint32), ("timeout_ns", ctypes.c_uint64),
        ("trace", _vp),
    ]


class tl_moe_args(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("self_rank", ctypes.c_int32), ("T_r", ctypes.c_int32), ("H", ctypes.c_int32),
        ("N", ctypes.c_int32), ("E", ctypes.c_int32), ("topk", ctypes.c_int32), ("rows_per_barrier", ctypes.c_int32),
        ("X", ctypes.POINTER(_vp)), ("topk_ids", _vp), ("W", ctypes.POINTER(_vp)), ("sorted_tokens", _vp),
        ("Y", _vp), ("perm", _vp), ("expert_offsets", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
        ("signals", _vp), ("epoch", ctypes.c_uint32), ("mode", ctypes.c_int32),
        ("timeout_ns", ctypes.c_uint64), ("trace", _vp),
    ]


class tl_moe_down_args(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("T_r", ctypes.c_int32), ("topk", ctypes.c_int32), ("E", ctypes.c_int32),
        ("I_r", ctypes.c_int32), ("Hd", ctypes.c_int32),
        ("H", ctypes.POINTER(_vp)), ("W2", ctypes.POINTER(_vp)), ("gates", _vp), ("routing", _vp),
        ("out", ctypes.POINTER(_vp)), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t), ("signals", _vp),
        ("epoch", ctypes.c_uint32), ("options", ctypes.c_uint32), ("timeout_ns", ctypes.c_uint64),
    ]


class tl_allgather_args(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("self_rank", ctypes.c_int32), ("M_shard", ctypes.c_int32), ("K", ctypes.c_int32),
        ("mode", ctypes.c_int32), ("rows_per_barrier", ctypes.c_int32), ("A_shards", ctypes.POINTER(_vp)),
        ("gathered", _vp), ("signals", _vp), ("src_ready", _vp), ("epoch", ctypes.c_uint32),
        ("reserved0", ctypes.c_uint32), ("timeout_ns", ctypes.c_uint64),
    ]


class tl_allgather_ll_args(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("self_rank", ctypes.c_int32), ("M_shard", ctypes.c_int32), ("K", ctypes.c_int32),
        ("protocol", ctypes.c_int32), ("rows_per_barrier", ctypes.c_int32), ("A_shards", ctypes.POINTER(_vp)),
        ("link", _vp), ("link_bytes", ctypes.c_size_t), ("gathered", _vp), ("signals", _vp),
        ("send_mask", ctypes.c_uint64), ("epoch", ctypes.c_uint32), ("reserved0", ctypes.c_uint32),
        ("timeout_ns", ctypes.c_uint64),
    ]


class tl_reduce_scatter_args(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int32), ("M", ctypes.c_int32), ("N", ctypes.c_int32), ("reserved0", ctypes.c_int32),
        ("partials", ctypes.POINTER(_vp)), ("out", ctypes.POINTER(_vp)),
    ]


class tl_kv_cache(ctypes.Structure):
    _fields_ = [
        ("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp),
        ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
        ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("H_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
    ]


class tl_kv_append_args(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int32), ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32), ("max_pos", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("max_q_len", ctypes.c_int32), ("cache", tl_kv_cache), ("k", _vp), ("v", _vp), ("q", _vp),
        ("k_token_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
        ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("q_out", _vp), ("cos", _vp), ("sin", _vp), ("cu_seqlens", _vp), ("seq_lens", _vp), ("page_table", _vp),
        ("signals", _vp),
    ]


class tl_kv_append_norm_args(ctypes.Structure):
    _fields_ = [
        ("append", tl_kv_append_args), ("q_weight", _vp), ("k_weight", _vp), ("positions", _vp), ("eps", ctypes.c_float),
        ("reserved0", ctypes.c_int32),
    ]


class tl_kv_attn_args(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int32), ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("causal", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("max_q_len", ctypes.c_int32), ("scale", ctypes.c_float),
        ("reserved0", ctypes.c_int32), ("cache", tl_kv_cache), ("q", _vp),
        ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("out", _vp), ("lse", _vp),
        ("cu_seqlens", _vp), ("seq_lens", _vp), ("page_table", _vp), ("workspace", _vp),
        ("workspace_bytes", ctypes.c_size_t), ("signals", _vp),
    ]


class tl_kv_tree_attn_args(ctypes.Structure):
    _fields_ = [("attn", tl_kv_attn_args), ("tree", _vp), ("tree_words", ctypes.c_int32), ("reserved0", ctypes.c_int32)]


class tl_kv_fork_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B_in", "B_out", "max_pages", "page_size", "num_pages", "reserved0")] + [
        (n, _vp) for n in ("page_table", "seq_lens", "refs", "parents", "page_table_out", "seq_lens_out", "refs_out", "copies",
                           "n_copies", "workspace")] + [("workspace_bytes", ctypes.c_size_t), ("signals", _vp)]


class tl_kv_resize_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "max_pages", "page_size", "num_pages")] + [
        (n, _vp) for n in ("page_table", "seq_lens", "new_lens", "refs", "refs_out", "workspace")] + [
        ("workspace_bytes", ctypes.c_size_t), ("signals", _vp)]


class tl_kv_copy_pages_args(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n", ctypes.c_int32)] + [
        (n, _vp) for n in ("caches", "src", "dst", "slots", "count", "signals")]


class tl_kv_compact_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_layers", "B", "max_pages", "max_kept")] + [
        (n, _vp) for n in ("caches", "kept", "n_kept", "cu_seqlens", "seq_lens", "page_table", "seq_lens_out", "signals")]


class tl_beam_select_args(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "K", "N", "V", "dtype", "eos", "history_stride", "length")] + [
        ("row_stride", ctypes.c_int64)] + [
        (n, _vp) for n in ("logits", "scores", "done", "parents", "tokens", "scores_out", "done_out", "lse", "history",
                           "history_out", "workspace")] + [("workspace_bytes", ctypes.c_size_t)]


class tl_moe_decode_args(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("Hd", ctypes.c_int32),
        ("E", ctypes.c_int32), ("topk", ctypes.c_int32), ("normalize", ctypes.c_int32), ("reserved0", ctypes.c_int32),
        ("x", _vp), ("logits", _vp), ("W1", ctypes.POINTER(_vp)), ("W2", ctypes.POINTER(_vp)), ("out", _vp),
        ("ids", _vp), ("gates", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t),
    ]


def _decl(name, restype, *argtypes):
    f = getattr(lib, name)
    f.restype = restype
    f.argtypes = list(argtypes)
    return f


_i, _u32, _u64, _sz = ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_size_t
_decl("tl_version", _i)
_decl("tl_last_error", ctypes.c_char_p)
_decl("tl_signals_create", _i, _i, ctypes.POINTER(_vp))
_decl("tl_signals_destroy", _i, _vp)
_decl("tl_signals_flags", _i, _vp, ctypes.POINTER(_vp), ctypes.POINTER(_i))
_decl("tl_signals_reset", _i, _vp, _vp)
_decl("tl_tile_notify", _i, _vp, _i, _i, _u32, _vp)
_decl("tl_tile_wait", _i, _vp, _i, _i, _u32, _u64, _vp)
_decl("tl_query_status", _i, _vp, _vp, ctypes.POINTER(_i), ctypes.POINTER(_i))
_decl("tl_gemm_workspace_size", _sz, _i, _i, _i, _i)
_decl("tl_gemm", _i, ctypes.POINTER(tl_gemm_args), _vp)
_decl("tl_ag_gemm_workspace_size", _sz, _i, _i, _i, _i, _i)
_decl("tl_ag_gemm_num_flags", _i, _i, _i, _i, _i, ctypes.POINTER(_i))
_decl("tl_ag_gemm_tile_order", _i, _i, _i, _i, ctypes.POINTER(ctypes.c_int32), _i)
_decl("tl_ag_gemm", _i, ctypes.POINTER(tl_ag_gemm_args), _vp)
_decl("tl_gemm_rs_workspace_size", _sz, _i, _i, _i)
_decl("tl_moe_down_workspace_size", _sz, _i, _i, _i, _i, _i)
_decl("tl_moe_down_num_flags", _i, _i, _i, _i, _i, _i)
_decl("tl_moe_down", _i, ctypes.POINTER(tl_moe_down_args), _vp)
_decl("tl_gemm_rs_num_flags", _i, _i, _i, _i)
_decl("tl_gemm_rs", _i, ctypes.POINTER(tl_gemm_rs_args), _vp)
_decl("tl_gemm_rs_noalloc", _i, ctypes.POINTER(tl_gemm_rs_args), _vp, _vp)
_decl("tl_moe_workspace_size", _sz, _i, _i, _i, _i)
_decl("tl_moe_num_flags", _i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_i))
_decl("tl_moe_ag_gemm", _i, ctypes.POINTER(tl_moe_args), _vp)
_decl("tl_allgather", _i, ctypes.POINTER(tl_allgather_args), _vp)
_decl("tl_reduce_scatter", _i, ctypes.POINTER(tl_reduce_scatter_args), _vp)
_decl("tl_allgather_ll_link_bytes", _sz, _i, _i, _i, _i)
_decl("tl_allgather_ll", _i, ctypes.POINTER(tl_allgather_ll_args), _vp)
_decl("tl_test_hold_chunks", _i, _i, _i, _u64)
_decl("tl_ag_attn_num_flags", _i, _i, _i)
_decl("tl_ag_attn", _i, ctypes.POINTER(tl_ag_attn_args), _vp)
_decl("tl_kv_append", _i, ctypes.POINTER(tl_kv_append_args), _vp)
_decl("tl_kv_attn_workspace_size", _sz, _i, _i, _i, _i, _i, _i)
_decl("tl_kv_attn", _i, ctypes.POINTER(tl_kv_attn_args), _vp)
_decl("tl_kv_append_norm", _i, ctypes.POINTER(tl_kv_append_norm_args), _vp)
_decl("tl_kv_tree_attn", _i, ctypes.POINTER(tl_kv_tree_attn_args), _vp)
_decl("tl_kv_fork_workspace_size", _sz, _i, _i)
_decl("tl_kv_fork", _i, ctypes.POINTER(tl_kv_fork_args), _vp)
_decl("tl_kv_resize_workspace_size", _sz, _i)
_decl("tl_kv_resize", _i, ctypes.POINTER(tl_kv_resize_args), _vp)
_decl("tl_kv_copy_pages", _i, ctypes.POINTER(tl_kv_copy_pages_args), _vp)
_decl("tl_kv_compact", _i, ctypes.POINTER(tl_kv_compact_args), _vp)
_decl("tl_beam_select_workspace_size", _sz, _i, _i, _i, _i)
_decl("tl_beam_select", _i, ctypes.POINTER(tl_beam_select_args), _vp)
_decl("tl_moe_decode_workspace_size", _sz, _i, _i, _i, _i, _i, _i)
_decl("tl_moe_decode", _i, ctypes.POINTER(tl_moe_decode_args), _vp)


def _check(code):
    if code != TL_OK:
        raise TLError(code, lib.tl_last_error().decode(errors="replace"))


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _ptr_array(ts):
    arr = (_vp * len(ts))(*[t.data_ptr() for t in ts])
    return arr


def tl_version():
    return lib.tl_version()


def tl_last_error():
    return lib.tl_last_error().decode(errors="replace")


class Signals:
    """Owner of a tl_signals object (device flags + status word)."""

    def __init__(self, num_flags: int):
        h = _vp()
        _check(lib.tl_signals_create(int(num_flags), ctypes.byref(h)))
        self.handle = h
        self.num_flags = int(num_flags)

    def flags_ptr(self):
        p, n = _vp(), _i()
        _check(lib.tl_signals_flags(self.handle, ctypes.byref(p), ctypes.byref(n)))
        return p.value, n.value

    def flags_tensor(self):
        """A zero-copy torch uint32-as-int32 CUDA view of the flags (memory owned by the library)."""
        ptr, n = self.flags_ptr()
        return _device_view(ptr, n, "<i4")

    def read_flags(self):
        """The flags as a CPU numpy uint32 array (synchronises the device)."""
        import numpy as np
        import torch
        torch.cuda.synchronize()
        return self.flags_tensor().cpu().numpy().view(np.uint32)

    def close(self):
        if self.handle:
            lib.tl_signals_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _device_view(dev_ptr, n, typestr):
    """A torch CUDA tensor viewing n elements at dev_ptr (no copy)."""
    import torch

    class _CAI:
        def __init__(self):
            self.__cuda_array_interface__ = {"shape": (n,), "typestr": typestr, "data": (dev_ptr, False),
                                             "version": 3, "strides": None}
    return torch.as_tensor(_CAI(), device="cuda")


def tl_signals_reset(sig: Signals, stream=None):
    _check(lib.tl_signals_reset(sig.handle, _stream(stream)))


def tl_tile_notify(sig: Signals, first: int, count: int, value: int, stream=None):
    _check(lib.tl_tile_notify(sig.handle, int(first), int(count), int(value) & 0xFFFFFFFF, _stream(stream)))


def tl_tile_wait(sig: Signals, first: int, count: int, value: int, timeout_ns: int = 0, stream=None):
    _check(lib.tl_tile_wait(sig.handle, int(first), int(count), int(value) & 0xFFFFFFFF, int(timeout_ns),
                            _stream(stream)))


def tl_query_status(sig: Signals, stream=None):
    """Returns (code, where); code 0 = no device error.  Clears the status word."""
    code, where = _i(), _i()
    rc = lib.tl_query_status(sig.handle, _stream(stream), ctypes.byref(code), ctypes.byref(where))
    if rc not in (TL_OK,) and code.value == 0:
        _check(rc)
    return code.value, where.value


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def tl_gemm_workspace_size(M, N, K, sm_count=0):
    return int(lib.tl_gemm_workspace_size(M, N, K, sm_count))


def tl_ag_gemm_workspace_size(R, M_shard, K, N, sm_count=0):
    return int(lib.tl_ag_gemm_workspace_size(R, M_shard, K, N, sm_count))


def tl_gemm(A, B, C, signals: Signals, *, C_f32=None, timeout_ns=0, workspace=None, stream=None):
    """C = A . B (bf16 in, fp32 accumulate) with no communication; split over K
    when the tiles leave SMs idle and a (zeroed) workspace is given."""
    M, K = A.shape
    N = B.shape[1]
    a = tl_gemm_args(M=M, N=N, K=K, reserved0=0, A=_ptr(A), B=_ptr(B), C=_ptr(C), C_f32=_ptr(C_f32),
                     signals=signals.handle, timeout_ns=int(timeout_ns), workspace=_ptr(workspace),
                     workspace_bytes=_nbytes(workspace))
    _check(lib.tl_gemm(ctypes.byref(a), _stream(stream)))


def tl_ag_gemm_num_flags(R, M_shard, K, rows_per_barrier=0):
    eff = _i()
    n = lib.tl_ag_gemm_num_flags(R, M_shard, K, rows_per_barrier, ctypes.byref(eff))
    return n, eff.value


def tl_ag_gemm_tile_order(R, self_rank, M_shard):
    Mt = -(-R * M_shard // 256)
    out = (ctypes.c_int32 * Mt)()
    _check(lib.tl_ag_gemm_tile_order(R, self_rank, M_shard, out, Mt))
    return list(out)


def tl_ag_gemm(A_shards, B, gathered, C, signals: Signals, epoch: int, *, self_rank=0, C_f32=None,
               mode=TL_MODE_PUSH, src_ready: Signals | None = None, rows_per_barrier=0, timeout_ns=0,
               trace=None, swizzle=TL_SWIZZLE_ARRIVAL, workspace=None, stream=None):
    """C = [A_0; ...; A_{R-1}] . B, gathered rows written to `gathered` (see tilelink.h)."""
    R = len(A_shards)
    M_shard, K = A_shards[0].shape
    N = B.shape[1]
    ptrs = _ptr_array(A_shards)
    a = tl_ag_gemm_args(R=R, self_rank=self_rank, M_shard=M_shard, K=K, N=N, mode=mode,
                        rows_per_barrier=rows_per_barrier, swizzle=int(swizzle),
                        A_shards=ctypes.cast(ptrs, ctypes.POINTER(_vp)), B=_ptr(B), gathered=_ptr(gathered),
                        C=_ptr(C), C_f32=_ptr(C_f32), signals=signals.handle,
                        src_ready=src_ready.handle if src_ready is not None else None,
                        epoch=int(epoch) & 0xFFFFFFFF, reserved1=0, timeout_ns=int(timeout_ns), trace=_ptr(trace),
                        workspace=_ptr(workspace), workspace_bytes=_nbytes(workspace))
    _check(lib.tl_ag_gemm(ctypes.byref(a), _stream(stream)))


def tl_gemm_rs_workspace_size(R, M, N):
    return int(lib.tl_gemm_rs_workspace_size(R, M, N))


def tl_gemm_rs_num_flags(R, M, N):
    return int(lib.tl_gemm_rs_num_flags(R, M, N))


def tl_gemm_rs(A, B, out, workspace, signals: Signals, epoch: int, *, timeout_ns=0, trace=None, options=0,
               stream=None):
    """out[d] = rows d of sum_r A_r . B_r, rank order unless options say otherwise (see tilelink.h)."""
    R = len(A)
    M, K_r = A[0].shape
    N = B[0].shape[1]
    pa, pb, po = _ptr_array(A), _ptr_array(B), _ptr_array(out)
    a = tl_gemm_rs_args(R=R, M=M, K_r=K_r, N=N, A=ctypes.cast(pa, ctypes.POINTER(_vp)),
                        B=ctypes.cast(pb, ctypes.POINTER(_vp)), out=ctypes.cast(po, ctypes.POINTER(_vp)),
                        workspace=_ptr(workspace), workspace_bytes=workspace.numel() * workspace.element_size(),
                        signals=signals.handle, epoch=int(epoch) & 0xFFFFFFFF, options=int(options),
                        timeout_ns=int(timeout_ns), trace=_ptr(trace))
    _check(lib.tl_gemm_rs(ctypes.byref(a), _stream(stream)))


def tl_gemm_rs_noalloc(A, B, out, epoch: int, *, dev_status=None, timeout_ns=0, options=0, stream=None):
    """GEMM-RS for callers that cannot allocate device memory: the library's
    static device scratch replaces the workspace and the signals object.
    dev_status: optional int32 CUDA tensor of 4 words that receives device errors."""
    R = len(A)
    M, K_r = A[0].shape
    N = B[0].shape[1]
    pa, pb, po = _ptr_array(A), _ptr_array(B), _ptr_array(out)
    a = tl_gemm_rs_args(R=R, M=M, K_r=K_r, N=N, A=ctypes.cast(pa, ctypes.POINTER(_vp)),
                        B=ctypes.cast(pb, ctypes.POINTER(_vp)), out=ctypes.cast(po, ctypes.POINTER(_vp)),
                        workspace=None, workspace_bytes=0, signals=None, epoch=int(epoch) & 0xFFFFFFFF,
                        options=int(options), timeout_ns=int(timeout_ns), trace=None)
    _check(lib.tl_gemm_rs_noalloc(ctypes.byref(a), _ptr(dev_status), _stream(stream)))


def tl_moe_workspace_size(R, T_r, E, topk):
    return int(lib.tl_moe_workspace_size(R, T_r, E, topk))


def tl_moe_num_flags(R, T_r, H, topk, rows_per_barrier=0, mode=TL_MODE_PULL):
    eff = _i()
    n = lib.tl_moe_num_flags(mode, R, T_r, H, topk, rows_per_barrier, ctypes.byref(eff))
    return n, eff.value


def tl_moe_ag_gemm(X, topk_ids, W, sorted_tokens, Y, perm, expert_offsets, workspace, signals: Signals, epoch: int,
                   *, self_rank=0, rows_per_barrier=0, mode=TL_MODE_PULL, timeout_ns=0, trace=None, stream=None):
    """AllGather + grouped MoE GEMM (see tilelink.h): Y rows in expert-sorted order."""
    R = len(X)
    T_r, H = X[0].shape
    E = len(W)
    N = W[0].shape[1]
    topk = topk_ids.shape[1]
    px, pw = _ptr_array(X), _ptr_array(W)
    a = tl_moe_args(R=R, self_rank=self_rank, T_r=T_r, H=H, N=N, E=E, topk=topk, rows_per_barrier=rows_per_barrier,
                    X=ctypes.cast(px, ctypes.POINTER(_vp)), topk_ids=_ptr(topk_ids),
                    W=ctypes.cast(pw, ctypes.POINTER(_vp)), sorted_tokens=_ptr(sorted_tokens), Y=_ptr(Y),
                    perm=_ptr(perm), expert_offsets=_ptr(expert_offsets), workspace=_ptr(workspace),
                    workspace_bytes=workspace.numel() * workspace.element_size(), signals=signals.handle,
                    epoch=int(epoch) & 0xFFFFFFFF, mode=mode, timeout_ns=int(timeout_ns), trace=_ptr(trace))
    _check(lib.tl_moe_ag_gemm(ctypes.byref(a), _stream(stream)))


def tl_allgather(A_shards, gathered, signals: Signals, epoch: int, *, self_rank=0, mode=TL_MODE_PUSH,
                 src_ready: Signals | None = None, rows_per_barrier=0, timeout_ns=0, stream=None):
    """Gather the shards into `gathered`, releasing one flag per chunk (see tilelink.h)."""
    R = len(A_shards)
    M_shard, K = A_shards[0].shape
    ptrs = _ptr_array(A_shards)
    a = tl_allgather_args(R=R, self_rank=self_rank, M_shard=M_shard, K=K, mode=mode,
                          rows_per_barrier=rows_per_barrier, A_shards=ctypes.cast(ptrs, ctypes.POINTER(_vp)),
                          gathered=_ptr(gathered), signals=signals.handle,
                          src_ready=src_ready.handle if src_ready is not None else None,
                          epoch=int(epoch) & 0xFFFFFFFF, reserved0=0, timeout_ns=int(timeout_ns))
    _check(lib.tl_allgather(ctypes.byref(a), _stream(stream)))


def tl_allgather_ll_link_bytes(R, M_shard, K, rows_per_barrier=0):
    return int(lib.tl_allgather_ll_link_bytes(R, M_shard, K, rows_per_barrier))


def tl_allgather_ll(A_shards, link, gathered, signals: Signals, epoch: int, *, self_rank=0,
                    protocol=TL_LL_FLAG_IN_DATA, send_mask=None, rows_per_barrier=0, timeout_ns=0, stream=None):
    """AllGather through the link buffer `link` (pinned host or device tensor) with the
    flag-in-data protocol or the separate-flag one (see tilelink.h).  send_mask None =
    every rank sends in this launch."""
    R = len(A_shards)
    M_shard, K = A_shards[0].shape
    ptrs = _ptr_array(A_shards)
    mask = (1 << R) - 1 if send_mask is None else int(send_mask)
    a = tl_allgather_ll_args(R=R, self_rank=self_rank, M_shard=M_shard, K=K, protocol=int(protocol),
                             rows_per_barrier=rows_per_barrier, A_shards=ctypes.cast(ptrs, ctypes.POINTER(_vp)),
                             link=_ptr(link), link_bytes=_nbytes(link), gathered=_ptr(gathered),
                             signals=signals.handle, send_mask=mask, epoch=int(epoch) & 0xFFFFFFFF, reserved0=0,
                             timeout_ns=int(timeout_ns))
    _check(lib.tl_allgather_ll(ctypes.byref(a), _stream(stream)))


def tl_test_hold_chunks(first_flag, count, hold_ns):
    """Test facility: on this thread, later copy-warp calls move the chunks with flag ids in
    [first_flag, first_flag + count) last, after hold_ns (see tilelink.h).  count 0 = off."""
    _check(lib.tl_test_hold_chunks(int(first_flag), int(count), int(hold_ns)))


def tl_reduce_scatter(partials, out, *, stream=None):
    """out[d] = rows d of the rank-ordered fp32 sum of the partials, bf16."""
    R = len(partials)
    M, N = partials[0].shape
    pp, po = _ptr_array(partials), _ptr_array(out)
    a = tl_reduce_scatter_args(R=R, M=M, N=N, reserved0=0, partials=ctypes.cast(pp, ctypes.POINTER(_vp)),
                               out=ctypes.cast(po, ctypes.POINTER(_vp)))
    _check(lib.tl_reduce_scatter(ctypes.byref(a), _stream(stream)))


def tl_moe_down_workspace_size(R, T_r, topk, E, Hd):
    return int(lib.tl_moe_down_workspace_size(R, T_r, topk, E, Hd))


def tl_moe_down_num_flags(R, T_r, topk, E, Hd):
    return int(lib.tl_moe_down_num_flags(R, T_r, topk, E, Hd))


def tl_moe_down(H, W2, gates, routing, out, workspace, signals: Signals, epoch: int, *, topk, E, timeout_ns=0,
                options=0, stream=None):
    """out[d] = the gate-weighted combine of each token's expert outputs, Y summed over ranks
    (see tilelink.h); routing is the workspace of the matching tl_moe_ag_gemm call."""
    R = len(H)
    P, I_r = H[0].shape
    Hd = W2[0].shape[1]
    T_r = out[0].shape[0]
    ph, pw, po = _ptr_array(H), _ptr_array(W2), _ptr_array(out)
    a = tl_moe_down_args(R=R, T_r=T_r, topk=topk, E=E, I_r=I_r, Hd=Hd, H=ctypes.cast(ph, ctypes.POINTER(_vp)),
                         W2=ctypes.cast(pw, ctypes.POINTER(_vp)), gates=_ptr(gates), routing=_ptr(routing),
                         out=ctypes.cast(po, ctypes.POINTER(_vp)), workspace=_ptr(workspace),
                         workspace_bytes=workspace.numel() * workspace.element_size(), signals=signals.handle,
                         epoch=int(epoch) & 0xFFFFFFFF, options=int(options), timeout_ns=int(timeout_ns))
    _check(lib.tl_moe_down(ctypes.byref(a), _stream(stream)))


def tl_ag_attn_num_flags(R, S_shard):
    return int(lib.tl_ag_attn_num_flags(R, S_shard))


def tl_ag_attn(Q, K_shards, V_shards, K_gathered, V_gathered, O, signals: Signals, epoch: int, *, self_rank=0,
               causal=False, scale=0.0, lse=None, timeout_ns=0, stream=None):
    """O = softmax(scale Q Kg^T) Vg per head over the gathered key/value shards,
    K_gathered / V_gathered written (see tilelink.h).  Q [S_shard, H, D],
    K_r / V_r [S_shard, H_kv, D], lse optional float [H, S_shard]."""
    R = len(K_shards)
    S_shard, H, D = Q.shape
    H_kv = K_shards[0].shape[1]
    pk, pv = _ptr_array(K_shards), _ptr_array(V_shards)
    a = tl_ag_attn_args(R=R, self_rank=self_rank, S_shard=S_shard, H=H, H_kv=H_kv, head_dim=D,
                        causal=int(bool(causal)), scale=float(scale), Q=_ptr(Q),
                        K_shards=ctypes.cast(pk, ctypes.POINTER(_vp)), V_shards=ctypes.cast(pv, ctypes.POINTER(_vp)),
                        K_gathered=_ptr(K_gathered), V_gathered=_ptr(V_gathered), O=_ptr(O), lse=_ptr(lse),
                        signals=signals.handle, epoch=int(epoch) & 0xFFFFFFFF, reserved0=0,
                        timeout_ns=int(timeout_ns))
    _check(lib.tl_ag_attn(ctypes.byref(a), _stream(stream)))


# ---------------------------------------------------------------- serving: the 8-bit paged cache, experts for a few tokens
# A decode step's calls take a few microseconds on the GPU, so their marshalling is kept short: the arguments are packed
# in one go, laid out as the C structures above.

_APPEND = struct.Struct("@8i4P3q4i3P6q7P")
_APPEND_NORM = struct.Struct(_APPEND.format + "3Pfi")
_ATTN = struct.Struct("@6ifi4P3q4iP2q6PNP")
_TREE = struct.Struct(_ATTN.format + "P2i")
_FORK = struct.Struct("@6i10PNP")
_RESIZE = struct.Struct("@4i6PNP")
_COPY_PAGES = struct.Struct("@2i6P")
_COMPACT = struct.Struct("@4i8P")
_BEAM = struct.Struct("@8iq11PN")
_MOE = struct.Struct("@8i8PN")
assert _APPEND.size == ctypes.sizeof(tl_kv_append_args) and \
    _APPEND_NORM.size == ctypes.sizeof(tl_kv_append_norm_args) and _TREE.size == ctypes.sizeof(tl_kv_tree_attn_args) and _ATTN.size == ctypes.sizeof(tl_kv_attn_args) and \
    _MOE.size == ctypes.sizeof(tl_moe_decode_args) and _FORK.size == ctypes.sizeof(tl_kv_fork_args) and \
    _RESIZE.size == ctypes.sizeof(tl_kv_resize_args) and _COPY_PAGES.size == ctypes.sizeof(tl_kv_copy_pages_args) and \
    _COMPACT.size == ctypes.sizeof(tl_kv_compact_args) and _BEAM.size == ctypes.sizeof(tl_beam_select_args)


def _packed(name):
    """The library's function, taking its argument structure as packed bytes."""
    f = lib[name]
    f.restype, f.argtypes = _i, [ctypes.c_char_p, _vp]
    return f


_kv_append, _kv_attn, _moe_decode = _packed("tl_kv_append"), _packed("tl_kv_attn"), _packed("tl_moe_decode")
_kv_append_norm, _kv_tree_attn = _packed("tl_kv_append_norm"), _packed("tl_kv_tree_attn")
_kv_fork, _kv_resize = _packed("tl_kv_fork"), _packed("tl_kv_resize")
_kv_copy_pages, _kv_compact, _beam_select = _packed("tl_kv_copy_pages"), _packed("tl_kv_compact"), _packed("tl_beam_select")
_torch = None


def _place(stream):
    """(The stream's handle, the number of the current device): where a call's kernels run, and its tensors have to be."""
    global _torch
    if _torch is None:
        import torch
        torch.cuda.init()
        _torch = torch
    dev = _torch._C._cuda_getDevice()
    return (_torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)), dev


def _mistyped(t, what, dtype, shape, dev):
    raise ValueError(f"{what}: a tensor on device cuda:{dev} of {dtype} and shape {tuple(shape)}, not {t.dtype} "
                     f"{tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def _typed(t, what, dtype, shape, dev):
    """t is a contiguous tensor of this type and shape on CUDA device `dev`; its address."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _mistyped(t, what, dtype, shape, dev)
    return t.data_ptr()


def _rows(t, what, dtype, shape, dev):
    """A tensor [tokens, heads, dim] on CUDA device `dev` whose dims lie next to one another: its address and outer strides."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _mistyped(t, what, dtype, shape, dev)
    a, b, c = t.stride()
    if c != 1:
        raise ValueError(f"{what}: the dims of a head must lie next to one another")
    return t.data_ptr(), a, b


def _scratch(t, dev):
    """Address and size of a call's workspace."""
    if t is None:
        return 0, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on device cuda:{dev}, not on {t.device}"
                         f"{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr(), t.numel() * t.element_size()


def _held(x, dev):
    """A cache or weights whose tensors are on CUDA device `dev`."""
    if x.device != dev:
        raise ValueError(f"{type(x).__name__}: its tensors are on cuda:{x.device}, the current device is cuda:{dev}")


class KvCache:
    """The paged 8-bit cache (see tilelink.h): k and v are uint8 or float8_e4m3fn tensors of codes
    [num_pages, H_kv, page_size, head_dim] (any strides that are multiples of 16 and the same for both,
    dims next to one another: views of one buffer will do), k_scale and v_scale the E8M0 bytes
    [num_pages, H_kv].  Holds the tensors."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        for t in (k, v):
            if t.dim() != 4 or t.element_size() != 1 or not t.is_cuda:
                raise ValueError("KvCache: codes are 4-D CUDA tensors of 8-bit elements")
            if t.stride(3) != 1:
                raise ValueError("KvCache: the dims of a code tensor must lie next to one another")
        if k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("KvCache: k and v must have the same shape and strides")
        for t in (k_scale, v_scale):
            if tuple(t.shape) != tuple(k.shape[:2]) or t.element_size() != 1 or not t.is_contiguous() or not t.is_cuda:
                raise ValueError("KvCache: scales are contiguous [num_pages, H_kv] CUDA tensors of bytes")
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, k.get_device()
        if any(t.get_device() != self.device for t in (v, k_scale, v_scale)):
            raise ValueError("KvCache: codes and scales must be on one device")
        self.num_pages, self.H_kv, self.page_size, self.head_dim = k.shape
        self.fields = (k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k.stride(0), k.stride(1),
                       k.stride(2), self.num_pages, self.page_size, self.H_kv, self.head_dim)


def _batch(cu_seqlens, seq_lens, page_table, int32, dev):
    """(B, columns of the page table, the three addresses) of a ragged batch, its arrays' types checked."""
    B, max_pages = page_table.shape
    return (B, max_pages, _typed(cu_seqlens, "cu_seqlens", int32, (B + 1,), dev), _typed(seq_lens, "seq_lens", int32, (B,), dev),
            _typed(page_table, "page_table", int32, (B, max_pages), dev))


def _append_fields(dev, cache, k, v, cu_seqlens, seq_lens, page_table, signals, q, q_out, cos, sin, interleaved, max_q_len):
    """tl_kv_append_args, field by field."""
    bf16, f32 = _torch.bfloat16, _torch.float32
    n, D = k.shape[0], cache.head_dim
    _held(cache, dev)
    B, max_pages, cu, lens, table = _batch(cu_seqlens, seq_lens, page_table, _torch.int32, dev)
    kp, ka, kb = _rows(k, "k", bf16, (n, cache.H_kv, D), dev)
    vp, va, vb = _rows(v, "v", bf16, (n, cache.H_kv, D), dev)
    H = qp = qa = qb = out = rot = max_pos = cp = sp = 0
    if q is not None or q_out is not None:
        if q is None or q_out is None:
            raise ValueError("q and q_out go together")
        H = q.shape[1]
        qp, qa, qb = _rows(q, "q", bf16, (n, H, D), dev)
        out = _typed(q_out, "q_out", bf16, (n, H, D), dev)
    if cos is not None or sin is not None:
        if cos is None or sin is None:
            raise ValueError("cos and sin go together")
        max_pos, rot = cos.shape
        cp, sp = _typed(cos, "cos", f32, (max_pos, rot), dev), _typed(sin, "sin", f32, (max_pos, rot), dev)
        rot *= 2
    return (n, B, H, rot, bool(interleaved), max_pos, max_pages, max_q_len, *cache.fields, kp, vp, qp, ka, kb, va, vb, qa, qb,
            out, cp, sp, cu, lens, table, signals.handle.value)


def tl_kv_append(cache: KvCache, k, v, cu_seqlens, seq_lens, page_table, signals: Signals, *, q=None, q_out=None,
                 cos=None, sin=None, interleaved=False, max_q_len=0, stream=None):
    """Append k, v [n, H_kv, D] (bf16; views of a fused projection will do) to the cache, k rotated by the
    tables cos, sin [positions, rot_dim/2] at each token's position; q [n, H, D] rotated into q_out
    (see tilelink.h).  No tables: no rotation."""
    st, dev = _place(stream)
    code = _kv_append(_APPEND.pack(*_append_fields(dev, cache, k, v, cu_seqlens, seq_lens, page_table, signals, q, q_out, cos,
                                                   sin, interleaved, max_q_len)), st)
    if code:
        _check(code)


def tl_kv_append_norm(cache: KvCache, k, v, cu_seqlens, seq_lens, page_table, signals: Signals, *, q=None, q_out=None,
                      q_weight=None, k_weight=None, eps=1e-6, cos=None, sin=None, positions=None, interleaved=False,
                      max_q_len=0, stream=None):
    """tl_kv_append with each head's queries and keys normed by the weights q_weight, k_weight [D] (bf16; None: not
    normed) before the rotation, and the tables read at positions [n] (int32; None: the tokens' own; see tilelink.h)."""
    st, dev = _place(stream)
    bf16, i32, D = _torch.bfloat16, _torch.int32, cache.head_dim
    fields = _append_fields(dev, cache, k, v, cu_seqlens, seq_lens, page_table, signals, q, q_out, cos, sin, interleaved,
                            max_q_len)
    code = _kv_append_norm(_APPEND_NORM.pack(*fields, 0 if q_weight is None else _typed(q_weight, "q_weight", bf16, (D,), dev),
                                             0 if k_weight is None else _typed(k_weight, "k_weight", bf16, (D,), dev),
                                             0 if positions is None else _typed(positions, "positions", i32, (k.shape[0],), dev),
                                             eps, 0), st)
    if code:
        _check(code)


def tl_kv_attn_workspace_size(n_tokens, B, H, H_kv, head_dim, sm_count=0):
    return int(lib.tl_kv_attn_workspace_size(n_tokens, B, H, H_kv, head_dim, sm_count))


def _attn_fields(dev, q, cache, out, cu_seqlens, seq_lens, page_table, workspace, signals, causal, scale, max_q_len, lse):
    """tl_kv_attn_args, field by field."""
    bf16 = _torch.bfloat16
    n, H, D = q.shape
    if D != cache.head_dim:
        raise ValueError(f"q: head dim {D}, the cache's is {cache.head_dim}")
    _held(cache, dev)
    B, max_pages, cu, lens, table = _batch(cu_seqlens, seq_lens, page_table, _torch.int32, dev)
    qp, qa, qb = _rows(q, "q", bf16, (n, H, D), dev)
    return (n, B, H, causal, max_pages, max_q_len, scale, 0, *cache.fields, qp, qa, qb, _typed(out, "out", bf16, (n, H, D), dev),
            0 if lse is None else _typed(lse, "lse", _torch.float32, (H, n), dev), cu, lens, table, *_scratch(workspace, dev),
            signals.handle.value)


def tl_kv_attn(q, cache: KvCache, out, cu_seqlens, seq_lens, page_table, workspace, signals: Signals, *, causal=True,
               scale=0.0, max_q_len=0, lse=None, stream=None):
    """out [n, H, D] = attention of q [n, H, D] over each sequence's keys and values in the cache, the new
    tokens' included; lse optional float [H, n] (see tilelink.h)."""
    st, dev = _place(stream)
    code = _kv_attn(_ATTN.pack(*_attn_fields(dev, q, cache, out, cu_seqlens, seq_lens, page_table, workspace, signals,
                                             bool(causal), scale, max_q_len, lse)), st)
    if code:
        _check(code)


def tl_kv_tree_attn(q, cache: KvCache, out, cu_seqlens, seq_lens, page_table, tree, workspace, signals: Signals, *, scale=0.0,
                    max_q_len=0, lse=None, stream=None):
    """tl_kv_attn for a tree of drafts: tree [n, words] (int32 bits) says which of its sequence's new tokens each new
    token sees beside those before them (see tilelink.h)."""
    st, dev = _place(stream)
    words = tree.shape[1]
    fields = _attn_fields(dev, q, cache, out, cu_seqlens, seq_lens, page_table, workspace, signals, 0, scale, max_q_len, lse)
    code = _kv_tree_attn(_TREE.pack(*fields, _typed(tree, "tree", _torch.int32, (q.shape[0], words), dev), words, 0), st)
    if code:
        _check(code)


class KvLayers:
    """The caches of the layers that share one page table, all laid out alike.  Holds them."""

    def __init__(self, caches):
        if not caches:
            raise ValueError("KvLayers: one cache at least")
        self.caches, self.device = list(caches), caches[0].device
        if any(c.fields[4:] != caches[0].fields[4:] or c.device != self.device for c in self.caches):
            raise ValueError("KvLayers: the caches must have the same sizes and strides, on one device")
        self.array = (tl_kv_cache * len(self.caches))(*(tl_kv_cache(*c.fields) for c in self.caches))
        self.address = ctypes.addressof(self.array)


def tl_kv_fork_workspace_size(B_in, B_out):
    return int(lib.tl_kv_fork_workspace_size(B_in, B_out))


def tl_kv_fork(page_table, seq_lens, refs, parents, page_table_out, seq_lens_out, refs_out, copies, n_copies, workspace,
               signals: Signals, *, page_size, stream=None):
    """Row o of page_table_out [B_out, max_pages] goes on from row parents[o] of page_table [B_in, max_pages]: pages are
    shared, part-filled ones listed in copies [3, B_out] and n_copies [1] for tl_kv_copy_pages; refs [pages] count the
    holders (all int32; see tilelink.h)."""
    st, dev = _place(stream)
    i32 = _torch.int32
    (B, max_pages), n, pages = page_table.shape, parents.shape[0], refs.shape[0]
    code = _kv_fork(_FORK.pack(
        B, n, max_pages, page_size, pages, 0, _typed(page_table, "page_table", i32, (B, max_pages), dev),
        _typed(seq_lens, "seq_lens", i32, (B,), dev), _typed(refs, "refs", i32, (pages,), dev),
        _typed(parents, "parents", i32, (n,), dev), _typed(page_table_out, "page_table_out", i32, (n, max_pages), dev),
        _typed(seq_lens_out, "seq_lens_out", i32, (n,), dev), _typed(refs_out, "refs_out", i32, (pages,), dev),
        _typed(copies, "copies", i32, (3, n), dev), _typed(n_copies, "n_copies", i32, (1,), dev), *_scratch(workspace, dev),
        signals.handle.value), st)
    if code:
        _check(code)


def tl_kv_resize_workspace_size(B):
    return int(lib.tl_kv_resize_workspace_size(B))


def tl_kv_resize(page_table, seq_lens, new_lens, refs, refs_out, workspace, signals: Signals, *, page_size, stream=None):
    """Sequences go from seq_lens [B] to new_lens [B] tokens: pages are taken into page_table [B, max_pages], or given
    back; refs [pages] count the holders (all int32; see tilelink.h)."""
    st, dev = _place(stream)
    i32 = _torch.int32
    (B, max_pages), pages = page_table.shape, refs.shape[0]
    code = _kv_resize(_RESIZE.pack(
        B, max_pages, page_size, pages, _typed(page_table, "page_table", i32, (B, max_pages), dev),
        _typed(seq_lens, "seq_lens", i32, (B,), dev), _typed(new_lens, "new_lens", i32, (B,), dev),
        _typed(refs, "refs", i32, (pages,), dev), _typed(refs_out, "refs_out", i32, (pages,), dev), *_scratch(workspace, dev),
        signals.handle.value), st)
    if code:
        _check(code)


def tl_kv_copy_pages(layers: KvLayers, src, dst, signals: Signals, *, slots=None, count=None, stream=None):
    """In every layer's cache the first slots[i] tokens (None: all) of page src[i] go to page dst[i], i below count [1]
    (None: all of src [n]; all int32; see tilelink.h)."""
    st, dev = _place(stream)
    i32 = _torch.int32
    _held(layers, dev)
    n, = src.shape
    code = _kv_copy_pages(_COPY_PAGES.pack(
        len(layers.caches), n, layers.address, _typed(src, "src", i32, (n,), dev), _typed(dst, "dst", i32, (n,), dev),
        0 if slots is None else _typed(slots, "slots", i32, (n,), dev),
        0 if count is None else _typed(count, "count", i32, (1,), dev), signals.handle.value), st)
    if code:
        _check(code)


def tl_kv_compact(layers: KvLayers, kept, n_kept, cu_seqlens, seq_lens, page_table, seq_lens_out, signals: Signals, *,
                  stream=None):
    """Of each sequence's new tokens those that kept [B, max_kept] names, n_kept [B] of them, move together behind the
    earlier ones, in every layer's cache; seq_lens_out [B] are the lengths then (all int32; see tilelink.h)."""
    st, dev = _place(stream)
    i32 = _torch.int32
    _held(layers, dev)
    B, max_pages, cu, lens, table = _batch(cu_seqlens, seq_lens, page_table, i32, dev)
    max_kept = kept.shape[1]
    code = _kv_compact(_COMPACT.pack(
        len(layers.caches), B, max_pages, max_kept, layers.address, _typed(kept, "kept", i32, (B, max_kept), dev),
        _typed(n_kept, "n_kept", i32, (B,), dev), cu, lens, table, _typed(seq_lens_out, "seq_lens_out", i32, (B,), dev),
        signals.handle.value), st)
    if code:
        _check(code)


def tl_beam_select_workspace_size(B, K, N, V):
    return int(lib.tl_beam_select_workspace_size(B, K, N, V))


def tl_beam_select(logits, scores, parents, tokens, scores_out, workspace, *, done=None, done_out=None, eos=-1, lse=None,
                   history=None, history_out=None, length=0, stream=None):
    """The N best continuations of each user's K beams: logits [B * K, V] (float or bf16, rows any distance apart), scores
    [B, K]; parents (rows of logits), tokens (int32) and scores_out [B, N] written (see tilelink.h)."""
    st, dev = _place(stream)
    i32, f32, u8 = _torch.int32, _torch.float32, _torch.uint8
    (B, K), N, (rows, V) = scores.shape, parents.shape[1], logits.shape
    half = logits.dtype is _torch.bfloat16
    if rows != B * K or logits.get_device() != dev or not (half or logits.dtype is f32):
        _mistyped(logits, "logits", "float32 or bfloat16", (B * K, V), dev)
    stride = logits.stride(0) if rows > 1 else V
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("logits: a row's elements must lie next to one another")
    hist = hist_out = width = 0
    if history is not None or history_out is not None:
        if history is None or history_out is None:
            raise ValueError("history and history_out go together")
        width = history.shape[1]
        hist = _typed(history, "history", i32, (B * K, width), dev)
        hist_out = _typed(history_out, "history_out", i32, (B * N, width), dev)
    code = _beam_select(_BEAM.pack(
        B, K, N, V, half, eos, width, length, stride, logits.data_ptr(), _typed(scores, "scores", f32, (B, K), dev),
        0 if done is None else _typed(done, "done", u8, (B, K), dev), _typed(parents, "parents", i32, (B, N), dev),
        _typed(tokens, "tokens", i32, (B, N), dev), _typed(scores_out, "scores_out", f32, (B, N), dev),
        0 if done_out is None else _typed(done_out, "done_out", u8, (B, N), dev),
        0 if lse is None else _typed(lse, "lse", f32, (B, K), dev), hist, hist_out, *_scratch(workspace, dev)), st)
    if code:
        _check(code)


class MoeWeights:
    """The experts of tl_moe_decode: E contiguous bf16 matrices W1[e] [H, 2*I] (gate columns, then up columns) and
    W2[e] [I, Hd].  Holds the tensors and their pointers."""

    def __init__(self, W1, W2):
        import torch
        if len(W1) != len(W2) or not W1:
            raise ValueError("MoeWeights: as many W1 as W2, one at least")
        self.E, (self.H, two_I), (self.I, self.Hd) = len(W1), W1[0].shape, W2[0].shape
        if two_I != 2 * self.I:
            raise ValueError(f"MoeWeights: W1 has {two_I} columns, W2 has {self.I} rows: twice as many are wanted")
        self.device = W1[0].get_device()
        if self.device < 0:
            raise ValueError("MoeWeights: the matrices are on a CUDA device")
        for w1, w2 in zip(W1, W2):
            _typed(w1, "W1", torch.bfloat16, (self.H, two_I), self.device)
            _typed(w2, "W2", torch.bfloat16, (self.I, self.Hd), self.device)
        self.W1, self.W2 = W1, W2
        self.pointers = _ptr_array(W1), _ptr_array(W2)
        self.addresses = tuple(ctypes.addressof(p) for p in self.pointers)


def tl_moe_decode_workspace_size(T, topk, E, H, I, Hd):
    return int(lib.tl_moe_decode_workspace_size(T, topk, E, H, I, Hd))


def tl_moe_decode(x, logits, weights: MoeWeights, out, ids, gates, workspace, *, normalize=True, stream=None):
    """out [T, Hd] = the mixture-of-experts layer of x [T, H] under the router's logits [T, E]; the chosen experts
    and their gates into ids and gates [T, topk] (see tilelink.h)."""
    st, dev = _place(stream)
    bf16, f32, w = _torch.bfloat16, _torch.float32, weights
    T, topk = ids.shape
    _held(w, dev)
    code = _moe_decode(_MOE.pack(T, w.H, w.I, w.Hd, w.E, topk, bool(normalize), 0, _typed(x, "x", bf16, (T, w.H), dev),
                                 _typed(logits, "logits", f32, (T, w.E), dev), *w.addresses,
                                 _typed(out, "out", bf16, (T, w.Hd), dev), _typed(ids, "ids", _torch.int32, (T, topk), dev),
                                 _typed(gates, "gates", f32, (T, topk), dev), *_scratch(workspace, dev)), st)
    if code:
        _check(code)
