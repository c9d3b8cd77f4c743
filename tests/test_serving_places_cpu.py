"""The serving calls' binding takes tensors of the current CUDA device only, workspaces among them: a pointer to anywhere
else would be followed by a kernel.  Checked without a device, on stand-ins that say where they are."""
import pytest
import torch

from tests.test_serving_cpu import B  # noqa: F401


class Tensor:
    """As much of a tensor as the binding asks for."""

    def __init__(self, dtype, *shape, device=0, contiguous=True):
        self.dtype, self.shape, self.where, self.contiguous = dtype, torch.Size(shape), device, contiguous

    def get_device(self):
        return self.where

    @property
    def is_cuda(self):
        return self.where >= 0

    @property
    def device(self):
        return "cpu" if self.where < 0 else f"cuda:{self.where}"

    def is_contiguous(self):
        return self.contiguous

    def stride(self, i=None):
        s, n = [], 1
        for d in reversed(self.shape):
            s.insert(0, n)
            n *= d
        return tuple(s) if i is None else s[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 4096


class Signals:
    class handle:
        value = 64


bf16, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture
def calls(B, monkeypatch):  # noqa: F811
    """The binding with its library calls and the current device (0) replaced; what was called."""
    made = []
    for name in ("_kv_append", "_kv_attn", "_moe_decode"):
        monkeypatch.setattr(B, name, lambda args, st, name=name: made.append(name) or 0)
    monkeypatch.setattr(B, "_torch", torch)
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.setattr(torch._C, name, lambda *a: 0, raising=False)
    monkeypatch.setattr(B, "_ptr_array", lambda ts: (B._vp * len(ts))())
    return made


def cache(B, device=0, **one):  # noqa: F811
    t = dict(k=Tensor(u8, 4, 2, 16, 64, device=device), v=Tensor(u8, 4, 2, 16, 64, device=device),
             k_scale=Tensor(u8, 4, 2, device=device), v_scale=Tensor(u8, 4, 2, device=device))
    return B.KvCache(**{**t, **one})


def batch():
    return dict(cu_seqlens=Tensor(i32, 3), seq_lens=Tensor(i32, 2), page_table=Tensor(i32, 2, 2))


def append(B):  # noqa: F811
    return B.tl_kv_append, dict(cache=cache(B), k=Tensor(bf16, 5, 2, 64), v=Tensor(bf16, 5, 2, 64), **batch(), signals=Signals,
                                q=Tensor(bf16, 5, 4, 64), q_out=Tensor(bf16, 5, 4, 64), cos=Tensor(f32, 9, 32),
                                sin=Tensor(f32, 9, 32))


def attn(B):  # noqa: F811
    return B.tl_kv_attn, dict(q=Tensor(bf16, 5, 4, 64), cache=cache(B), out=Tensor(bf16, 5, 4, 64), **batch(),
                              workspace=Tensor(u8, 4096), signals=Signals, lse=Tensor(f32, 4, 5))


def moe(B):  # noqa: F811
    w = B.MoeWeights([Tensor(bf16, 16, 16)] * 3, [Tensor(bf16, 8, 16)] * 3)
    return B.tl_moe_decode, dict(x=Tensor(bf16, 5, 16), logits=Tensor(f32, 5, 3), weights=w, out=Tensor(bf16, 5, 16),
                                 ids=Tensor(i32, 5, 2), gates=Tensor(f32, 5, 2), workspace=Tensor(u8, 4096))


CALLS = {"append": append, "attn": attn, "moe": moe}
PLACED = [("append", n) for n in ("k", "v", "cu_seqlens", "seq_lens", "page_table", "q", "q_out", "cos", "sin")] + \
    [("attn", n) for n in ("q", "out", "cu_seqlens", "seq_lens", "page_table", "workspace", "lse")] + \
    [("moe", n) for n in ("x", "logits", "out", "ids", "gates", "workspace")]


@pytest.mark.parametrize("call", CALLS)
def test_all_in_place(B, calls, call):  # noqa: F811
    f, a = CALLS[call](B)
    f(**a)
    assert len(calls) == 1


@pytest.mark.parametrize("call,name", PLACED)
@pytest.mark.parametrize("device", [-1, 1])
def test_a_tensor_of_another_device(B, calls, call, name, device):  # noqa: F811
    f, a = CALLS[call](B)
    a[name] = Tensor(a[name].dtype, *a[name].shape, device=device)
    with pytest.raises(ValueError, match=name):
        f(**a)
    assert not calls


@pytest.mark.parametrize("call", ["attn", "moe"])
def test_a_workspace_with_holes(B, calls, call):  # noqa: F811
    f, a = CALLS[call](B)
    a["workspace"] = Tensor(u8, 4096, contiguous=False)
    with pytest.raises(ValueError, match="workspace"):
        f(**a)
    assert not calls


def test_caches_and_weights_of_another_device(B, calls):  # noqa: F811
    for make in (append, attn):
        f, a = make(B)
        a["cache"] = cache(B, device=1)
        with pytest.raises(ValueError, match="KvCache"):
            f(**a)
    f, a = moe(B)
    a["weights"] = B.MoeWeights([Tensor(bf16, 16, 16, device=1)] * 3, [Tensor(bf16, 8, 16, device=1)] * 3)
    with pytest.raises(ValueError, match="MoeWeights"):
        f(**a)
    assert not calls


@pytest.mark.parametrize("device", [-1, 1])
def test_parts_of_a_cache_or_of_weights_elsewhere(B, calls, device):  # noqa: F811
    for name, shape in (("k", (4, 2, 16, 64)), ("v", (4, 2, 16, 64)), ("k_scale", (4, 2)), ("v_scale", (4, 2))):
        with pytest.raises(ValueError):
            cache(B, **{name: Tensor(u8, *shape, device=device)})
    one = Tensor(bf16, 16, 16), Tensor(bf16, 8, 16)
    with pytest.raises(ValueError):
        B.MoeWeights([one[0], Tensor(bf16, 16, 16, device=device)], [one[1]] * 2)
    with pytest.raises(ValueError):
        B.MoeWeights([one[0]] * 2, [one[1], Tensor(bf16, 8, 16, device=device)])
    if device < 0:
        with pytest.raises(ValueError):
            B.MoeWeights([Tensor(bf16, 16, 16, device=-1)], [Tensor(bf16, 8, 16, device=-1)])
