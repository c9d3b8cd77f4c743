"""tl_moe_decode against the float64 oracle: the experts chosen exactly, gates and outputs within counted bounds."""
import numpy as np
import pytest
import torch

from oracle import moe_decode as ora

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


class Call:
    def __init__(self, B, T, H, I, Hd, E, topk, *, normalize=True, seed=0, logits=None, scale=1.0):
        self.B, self.normalize, self.topk = B, normalize, topk
        rng = np.random.default_rng(seed)
        bf = lambda s, *shape: (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * s).to(torch.bfloat16)
        self.x = bf(scale, T, H)
        self.logits = rng.standard_normal((T, E)).astype(np.float32) if logits is None else np.asarray(logits, np.float32)
        self.W1 = [bf(H ** -0.5, H, 2 * I) for _ in range(E)]
        self.W2 = [bf(I ** -0.5, I, Hd) for _ in range(E)]
        chosen = set(ora.select(self.logits.astype(np.float64), topk, normalize)[0].ravel().tolist())
        nan = lambda w: torch.full_like(w, float("nan"))  # the weights that nobody chose are not to be read
        self.w = B.MoeWeights([(w if e in chosen else nan(w)).cuda() for e, w in enumerate(self.W1)],
                              [(w if e in chosen else nan(w)).cuda() for e, w in enumerate(self.W2)])
        self.dx, self.dl = self.x.cuda(), torch.from_numpy(self.logits).cuda()
        self.out = torch.full((T, Hd), 7.0, dtype=torch.bfloat16, device="cuda")
        self.ids = torch.full((T, topk), -1, dtype=torch.int32, device="cuda")
        self.gates = torch.full((T, topk), 7.0, device="cuda")
        self.ws = torch.zeros(B.tl_moe_decode_workspace_size(T, topk, E, H, I, Hd), dtype=torch.uint8, device="cuda")

    def run(self):
        self.B.tl_moe_decode(self.dx, self.dl, self.w, self.out, self.ids, self.gates, self.ws, normalize=self.normalize)
        return self

    def check(self):
        f = lambda t: t.cpu().double().numpy()
        want, ids, gates, slack = ora.layer(f(self.x), self.logits.astype(np.float64), [f(w) for w in self.W1],
                                            [f(w) for w in self.W2], self.topk, self.normalize)
        assert np.array_equal(self.ids.cpu().numpy(), ids)
        # exponentials to 2^-22, their argument (a difference of logits of magnitude below 2^6) to 2^-18, one division
        assert (np.abs(f(self.gates) - gates) <= 2.0 ** -17 * gates + 1e-38).all()
        slack = slack + 2.0 ** -17 * np.abs(want)
        bad = ~(np.abs(f(self.out) - want) <= 2.0 ** -8 * np.abs(want) + slack)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), f(self.out)[bad][:4], want[bad][:4])
        return self


@pytest.mark.parametrize("T", [1, 2, 3, 7, 15, 16, 17, 31, 32, 33, 50, 64])
@pytest.mark.parametrize("normalize", [True, False])
def test_token_counts(B, T, normalize):
    Call(B, T, 256, 96, 128, 8, 2, normalize=normalize, seed=T).run().check()


@pytest.mark.parametrize("H,I,Hd", [(8, 8, 8), (128, 64, 128), (136, 72, 200), (1000, 56, 264), (64, 1000, 72),
                                    (512, 128, 1024), (24, 16, 8)])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_odd_sizes(B, H, I, Hd, T):
    Call(B, T, H, I, Hd, 4, 3, seed=H + I).run().check()


@pytest.mark.parametrize("E,topk", [(1, 1), (2, 2), (5, 5), (16, 16), (33, 4), (64, 8), (256, 6), (100, 16)])
@pytest.mark.parametrize("T", [1, 20, 64])
def test_experts_and_topk(B, E, topk, T):
    Call(B, T, 64, 24, 40, E, topk, normalize=T != 20, seed=E).run().check()


def test_one_large_layer(B):
    Call(B, 3, 4096, 1408, 4096, 4, 2, seed=1).run().check()


@pytest.mark.parametrize("T", [17, 33, 64])
def test_all_tokens_choose_the_same_experts(B, T):
    logits = np.tile(np.array([0.0, 3.0, 1.0, 2.0, -1.0]), (T, 1))
    Call(B, T, 160, 72, 136, 5, 2, logits=logits, seed=2).run().check()


def test_ties_go_to_the_lower_index(B):
    logits = np.zeros((6, 40))
    logits[1, 35] = logits[1, 3] = 1.0
    logits[2] = -0.0
    logits[3, ::2] = -5.0
    logits[4, :] = np.arange(40) // 4
    logits[5, 33:36] = 7.0
    Call(B, 6, 64, 16, 16, 40, 4, logits=logits, seed=3).run().check()


def test_masked_experts(B):
    inf = np.inf
    logits = np.random.default_rng(4).standard_normal((4, 8))
    logits[0, [1, 3, 5]] = -inf
    logits[1, :7] = -inf          # fewer finite logits than topk: gates of the rest are 0
    logits[2] = -inf              # nothing left: all gates 0, output 0
    for normalize in (True, False):
        c = Call(B, 4, 64, 16, 24, 8, 3, logits=logits, normalize=normalize, seed=4).run().check()
        assert (c.out[2] == 0).all() and (c.gates[2] == 0).all()
        assert c.gates[1].tolist() == [1.0, 0.0, 0.0]


def test_nan_logits_rank_last(B):
    logits = np.random.default_rng(5).standard_normal((3, 6))
    logits[0, [0, 2]] = np.nan
    logits[1, [1, 5]] = np.nan
    logits[1, 3] = -np.inf
    Call(B, 3, 64, 16, 24, 6, 3, logits=logits, seed=5).run().check()
    logits[2, :4] = np.nan        # two numbers for three places: the lowest NaN comes third, and the gates are NaN
    c = Call(B, 3, 64, 16, 24, 6, 3, logits=logits, seed=5).run()
    order = sorted((4, 5), key=lambda e: -logits[2, e])
    assert c.ids[2].tolist() == order + [0] and torch.isnan(c.gates[2]).all() and torch.isnan(c.out[2]).all()
    assert not torch.isnan(c.out[:2]).any()


@pytest.mark.parametrize("scale", [1e-15, 1e-3, 1e4])
def test_small_and_large_tokens(B, scale):
    Call(B, 5, 256, 64, 72, 4, 2, seed=6, scale=scale).run().check()


@pytest.mark.parametrize("T", [1, 30])
def test_same_bits_again_on_a_stream_and_in_a_graph(B, T):
    c = Call(B, T, 512, 200, 264, 8, 2, seed=7).run().check()
    first = c.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.out.zero_()
        c.run()
    side.synchronize()
    assert torch.equal(c.out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
        c.run()
    for _ in range(3):
        c.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, first)


def test_one_workspace_for_many_sizes(B):
    """A workspace of the largest size serves the smaller calls in turn, and back."""
    calls = [Call(B, T, 128, 48, 136, 8, k, seed=T) for T, k in ((1, 1), (64, 4), (7, 2), (33, 8), (2, 3))]
    ws = max((c.ws for c in calls), key=lambda w: w.numel()).clone()
    for c in calls + calls[::-1]:
        c.ws = ws
        c.run().check()
