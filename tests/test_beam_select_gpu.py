"""tl_beam_select against the float64 oracle."""
import numpy as np
import pytest
import torch

from tests.kv_cases import f64
from oracle import beam as ora

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from tile_centric_gemm_gb300 import binding
    return binding


class Case:
    def __init__(self, L, logits, scores, N, *, done=None, eos=-1, history=None, length=0, place=None):
        """logits [B, K, V] (float or bf16, on the host); place: where its rows go (a strided device tensor [B K, V])."""
        self.L, self.N, self.eos, self.length = L, N, eos, length
        self.B, self.K, self.V = logits.shape
        self.logits, self.scores, self.done = logits, scores, done
        rows = logits.reshape(-1, self.V)
        self.d = rows.cuda() if place is None else place
        if place is not None:
            place.copy_(rows)
        self.ds = torch.from_numpy(scores.astype(np.float32)).cuda()
        self.dd = None if done is None else torch.from_numpy(done.astype(np.uint8)).cuda()
        self.ws = torch.zeros(L.tl_beam_select_workspace_size(self.B, self.K, N, self.V), dtype=torch.uint8, device="cuda")
        self.history = None if history is None else torch.from_numpy(history).cuda()

    def run(self, stream=None):
        i32 = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")
        self.parents, self.tokens = i32(self.B, self.N), i32(self.B, self.N)
        self.out = torch.full((self.B, self.N), 9.0, device="cuda")
        self.lse = torch.full((self.B, self.K), 9.0, device="cuda")
        self.done_out = torch.full((self.B, self.N), 9, dtype=torch.uint8, device="cuda")
        self.history_out = None if self.history is None else i32(self.B * self.N, self.history.shape[1])
        self.L.tl_beam_select(self.d, self.ds, self.parents, self.tokens, self.out, self.ws, done=self.dd, done_out=self.done_out,
                              eos=self.eos, lse=self.lse, history=self.history, history_out=self.history_out, length=self.length,
                              stream=stream)
        return self

    def check(self):
        x, scores = f64(self.logits), self.scores.astype(np.float32).astype(np.float64)
        total, lse = ora.totals(x, scores, self.done, self.eos)
        # A logit's distance from its thread's reference, and the reference's from the maximum, d + 2 together (d the logit's
        # distance from the maximum; references lie up to 1 below a maximum), are rounded to 2^-24 of them, and so are their
        # products with log2 e, itself off by as much: 3 (d + 2) 2^-24 in the exponent.  Exponentials are off by 2^-22 of
        # their result: a logit's, the reference's, and those of references that were raised (what came before is e times
        # less each time): 4 of them at most.  Sums: four in a chain and two more, 2^-24 each (pairs and 64 bits from there
        # on), and as much for the products.  lse is off by the mean of that over the softmax.
        with np.errstate(all="ignore"):
            w = np.exp(x - lse[..., None])
            d = np.where(w > 0, x.max(2, keepdims=True) - x, 0.0)
            tol = np.nan_to_num((w * (d + 2)).sum(2) * 3 * 2.0 ** -24 + 4 * 2.0 ** -22 + 12 * 2.0 ** -24, nan=0.0, posinf=0.0, neginf=0.0)
        got_lse = f64(self.lse)
        same = np.isclose(got_lse, lse, rtol=0, atol=0, equal_nan=True) & ~np.isfinite(lse)
        fine = np.isfinite(lse)
        assert (same | fine).all(), (got_lse[~(same | fine)], lse[~(same | fine)])
        assert (np.abs(got_lse - lse)[fine] <= (tol + 2.0 ** -24 * np.abs(lse))[fine]).all()
        tol = tol[..., None] * np.ones_like(total)
        if self.done is not None:
            tol[self.done != 0] = 0.0
        parents, tokens, out = self.parents.cpu().numpy(), self.tokens.cpu().numpy(), f64(self.out)
        done_out = self.done_out.cpu().numpy()
        for b in range(self.B):
            t, e = total[b].ravel(), tol[b].ravel()
            n = min(self.N, int((t > -np.inf).sum()))
            assert (parents[b, n:] == -1).all() and (tokens[b, n:] == -1).all() and (out[b, n:] == -np.inf).all()
            assert (done_out[b, n:] == 1).all()
            if n == 0:
                continue
            k = parents[b, :n] - b * self.K
            assert ((k >= 0) & (k < self.K) & (tokens[b, :n] >= 0) & (tokens[b, :n] < self.V)).all()
            flat = k.astype(np.int64) * self.V + tokens[b, :n]
            assert len(set(flat.tolist())) == n
            v, ve = t[flat], e[flat]
            assert (v > -np.inf).all()
            assert (np.abs(out[b, :n] - v) <= ve + 2.0 ** -24 * np.abs(v)).all()
            # in order, as far as two beams can be told apart by their lse
            order = v[:-1] - v[1:]
            assert (order >= -(ve[:-1] + ve[1:])).all()
            rest = np.setdiff1d(np.arange(t.size), flat, assume_unique=True)
            rest = rest[t[rest] > -np.inf]
            assert (t[rest] <= v[-1] + e[rest] + ve[-1]).all()
            # within a beam the order is that of the logits, equal ones by token: exactly
            for beam in set(k.tolist()):
                if self.done is not None and self.done[b, beam]:
                    continue
                mine = tokens[b, :n][k == beam]
                row = x[b, beam]
                want = np.lexsort((np.arange(self.V), -row))[:len(mine)]
                assert np.array_equal(mine, want)
            ended = (self.done[b, k] != 0) if self.done is not None else np.zeros(n, bool)
            assert np.array_equal(done_out[b, :n] != 0, ended | (tokens[b, :n] == self.eos))
            if self.history is not None:
                h, ho = self.history.cpu().numpy(), self.history_out.cpu().numpy()[b * self.N:(b + 1) * self.N]
                for i in range(n):
                    assert np.array_equal(ho[i, :self.length], h[parents[b, i], :self.length])
                    assert ho[i, self.length] == tokens[b, i] and (ho[i, self.length + 1:] == -9).all()
                assert (ho[n:] == -9).all()
        return self


def normal(seed, *shape, scale=2.5, half=False):
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)) * scale
    return x.to(torch.bfloat16) if half else x


def some_scores(seed, *shape):
    return -20 * np.random.default_rng(seed).random(shape)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V", [1, 2, 31, 257, 1000, 8185, 8192, 8193, 16384, 50001])
@pytest.mark.parametrize("K,N", [(1, 1), (4, 8), (3, 64)])
def test_sizes(B, V, K, N, half):
    Case(B, normal(V, 3, K, V, half=half), some_scores(K, 3, K), N).run().check()


@pytest.mark.parametrize("K,N,users", [(64, 64, 2), (16, 32, 20), (8, 16, 100), (2, 2, 700)])
def test_many_beams_and_users(B, K, N, users):
    Case(B, normal(K, users, K, 600), some_scores(N, users, K), N).run().check()


@pytest.mark.parametrize("half", [False, True])
def test_many_rows_of_many_steps(B, half):
    Case(B, normal(12, 80, 8, 9001, half=half), some_scores(12, 80, 8), 16).run().check()


def test_a_large_vocabulary(B):
    Case(B, normal(1, 2, 5, 300007, half=True), some_scores(1, 2, 5), 10).run().check()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("V,gap,offset", [(1000, 1, 0), (1003, 0, 1), (777, 6, 3), (9000, 7, 5), (64, 64, 2)])
def test_rows_anywhere(B, half, V, gap, offset):
    """Rows that begin at any element, with anything (NaN) before, between and behind them."""
    x = normal(V, 2, 3, V, half=half)
    store = torch.full((6 * (V + gap) + 16,), float("nan"), dtype=x.dtype, device="cuda")
    place = store[offset:offset + 6 * (V + gap)].view(6, V + gap)[:, :V]
    Case(B, x, some_scores(2, 2, 3), 12, place=place).run().check()


@pytest.mark.parametrize("V", [100, 8192, 20000])
def test_equal_logits_go_to_the_lower_beam_and_token(B, V):
    x = torch.zeros(2, 3, V)
    c = Case(B, x, np.array([[-1.0, -1.0, -1.0], [-2.0, -1.0, -3.0]]), 20).run().check()
    # the beams have the same lse, so equal scores are equal: beam 0's first tokens; and those of the best beam
    assert c.parents[0].tolist() == [0] * 20 and c.tokens[0].tolist() == list(range(20)) and c.parents[1].tolist() == [4] * 20
    step = torch.from_numpy((np.random.default_rng(3).integers(0, 4, (2, 3, V)) * 0.5).astype(np.float32))
    Case(B, step, some_scores(3, 2, 3), 33).run().check()
    few = torch.zeros(1, 2, V)
    few[0, :, V - 3:] = 1.0  # fewer above than places: the rest from the start
    c = Case(B, few, np.zeros((1, 2)), 10).run().check()
    assert c.tokens[0].tolist() == [V - 3, V - 2, V - 1] * 2 + [0, 1, 2, 3]


def test_zeros_of_both_signs_are_equal(B):
    x = torch.full((1, 1, 300), -5.0)
    x[0, 0, 7], x[0, 0, 9], x[0, 0, 30], x[0, 0, 200] = -0.0, 0.0, 0.0, -0.0
    assert Case(B, x, np.zeros((1, 1)), 4).run().check().tokens[0].tolist() == [7, 9, 30, 200]


@pytest.mark.parametrize("N", [2, 64])
def test_more_equal_scores_than_the_list_holds(B, N):
    c = Case(B, torch.ones(2, 64, 9000), np.full((2, 64), -3.0), N).run().check()
    for b in range(2):
        assert c.parents[b].tolist() == [64 * b] * N and c.tokens[b].tolist() == list(range(N))
    near = torch.ones(1, 64, 40000) + torch.arange(40000) * 2.0 ** -23  # (in steps of fp32's grain: far below 64-bit scores' upper halves)
    Case(B, near, np.full((1, 64), -3.0), N).run().check()


@pytest.mark.parametrize("half", [False, True])
def test_plateaus_in_long_rows(B, half):
    """Rows of many steps to a block: more values above the bound than there is room for, and a value shared by many."""
    users, K, V = 160, 4, 70001
    x = torch.zeros(1, K, V)
    x[0, 0, ::3] = 2.0                      # a third of the row is the maximum
    x[0, 1] = torch.arange(V) % 4096 / 64   # rises again and again
    x[0, 2, ::256] = 5.0                    # one thread's
    x[0, 2, 1::256] = torch.arange(len(x[0, 2, 1::256])) / 128.0
    x[0, 3, 60000:] = 1.0
    x = x.to(torch.bfloat16) if half else x
    c = Case(B, x.expand(users, K, V), np.tile(some_scores(11, 1, K) / 10, (users, 1)), 24)
    c.run()
    for out in (c.parents - torch.arange(users, device="cuda", dtype=torch.int32)[:, None] * K, c.tokens, c.out, c.lse):
        assert (out == out[:1]).all()
    one = Case(B, x, c.scores[:1], 24)
    one.run().check()
    c.logits, c.scores, c.B = c.logits[:1], c.scores[:1], 1
    c.parents, c.tokens, c.out, c.lse, c.done_out = (t[:1] for t in (c.parents, c.tokens, c.out, c.lse, c.done_out))
    c.check()


@pytest.mark.parametrize("half", [False, True])
def test_rising_and_falling_rows(B, half):
    up = torch.arange(20000, dtype=torch.float32).view(1, 1, -1) / 1000
    x = torch.cat([up, -up, up.flip(2)], 1)
    Case(B, x.to(torch.bfloat16) if half else x, np.zeros((1, 3)), 64).run().check()


@pytest.mark.parametrize("keep", [0, 1, 5, 40])
def test_masks_that_leave_few(B, keep):
    """Masked by -infinity or by the type's lowest value."""
    r = np.random.default_rng(keep)
    for low in (-np.inf, float(torch.finfo(torch.float32).min)):
        x = normal(4, 2, 3, 17000)
        m = torch.ones(2, 3, 17000, dtype=torch.bool)
        for b in range(2):
            for k in range(3):
                m[b, k, r.choice(17000, keep, replace=False)] = False
        Case(B, x.masked_fill(m, low), some_scores(4, 2, 3), 16).run().check()


def test_rows_that_offer_nothing(B):
    x = normal(5, 4, 4, 9000)
    x[0, 1, 8500], x[0, 2, 3], x[0, 3] = float("nan"), float("inf"), -float("inf")
    x[1, 0, 5], x[1, 0, 6] = float("inf"), float("nan")
    x[1, 1, 8999] = -float("nan")
    x[2] = -float("inf")
    scores = some_scores(5, 4, 4)
    scores[1, 2], scores[1, 3] = -np.inf, np.nan
    scores[3] = [np.inf, -np.inf, np.nan, -np.inf]
    c = Case(B, x, scores, 6).run().check()
    assert (c.parents[0] == 0).all() and (c.parents[1:] == -1).all()


def test_ended_beams(B):
    x = normal(6, 5, 4, 9000)
    done = np.zeros((5, 4), bool)
    done[0, 1] = done[1, 0] = done[1, 3] = done[2] = done[3, 2] = True
    x[1, 0] = float("nan")  # not looked at
    scores = some_scores(6, 5, 4)
    scores[0, 1], scores[3, 2], scores[2, 1] = 0.0, -1e4, -np.inf
    h = np.random.default_rng(6).integers(0, 9000, (20, 12)).astype(np.int32)
    c = Case(B, x, scores, 6, done=done, eos=77, history=h, length=7).run().check()
    assert c.parents[0, 0] == 1 and c.tokens[0, 0] == 77
    c = Case(B, x, scores, 6, eos=77, history=h, length=0).run().check()


def test_a_token_that_ends_a_beam(B):
    x = normal(7, 2, 3, 500)
    x[:, 1, 42] = 30.0
    c = Case(B, x, np.zeros((2, 3)), 4, eos=42).run().check()
    assert c.tokens[0, 0] == 42 and c.done_out[0, 0] == 1


def test_great_and_tiny_numbers(B):
    for scale in (1e30, 1e-30, 1e4):
        Case(B, normal(8, 2, 3, 9000, scale=scale), some_scores(8, 2, 3), 9).run().check()
    Case(B, normal(8, 2, 3, 900), some_scores(8, 2, 3) * 1e6, 9).run().check()


def test_same_bits_again_on_a_stream_and_in_a_graph(B):
    c = Case(B, normal(9, 6, 4, 30000), some_scores(9, 6, 4), 8).run().check()
    first = [x.clone() for x in (c.parents, c.tokens, c.out, c.lse)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (c.parents, c.tokens, c.out, c.lse)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for _ in range(3):
        for x in (c.parents, c.tokens, c.out, c.lse):
            x.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (c.parents, c.tokens, c.out, c.lse)))


def test_one_workspace_for_many_sizes(B):
    cases = [Case(B, normal(i, b, k, v), some_scores(i, b, k), n) for i, (b, k, v, n) in
             enumerate([(1, 4, 20000, 8), (50, 3, 300, 2), (3, 64, 9000, 64), (700, 1, 50, 1)])]
    ws = max((c.ws for c in cases), key=lambda w: w.numel()).clone()
    for c in cases + cases[::-1]:
        c.ws = ws
        c.run().check()


def test_offsets_past_32_bits(B):
    V, rows = 1 << 24, 140
    x = torch.full((rows, V), -9.0, dtype=torch.bfloat16, device="cuda")
    x[rows - 1, V - 5], x[rows - 1, 3] = 4.0, 3.0
    i32 = lambda: torch.empty(rows, 2, dtype=torch.int32, device="cuda")
    parents, tokens, out = i32(), i32(), torch.empty(rows, 2, device="cuda")
    ws = torch.zeros(B.tl_beam_select_workspace_size(rows, 1, 2, V), dtype=torch.uint8, device="cuda")
    B.tl_beam_select(x, torch.zeros(rows, 1, device="cuda"), parents, tokens, out, ws)
    assert parents[rows - 1].tolist() == [rows - 1] * 2 and tokens[rows - 1].tolist() == [V - 5, 3]
    assert tokens[0].tolist() == [0, 1]


def test_binding_refuses(B):
    x = normal(10, 2, 3, 100)
    c = Case(B, x, np.zeros((2, 3)), 4).run().check()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    good = dict(logits=c.d, scores=c.ds, parents=c.parents, tokens=c.tokens, scores_out=c.out, workspace=c.ws)
    for bad in (dict(logits=c.d.half()), dict(logits=c.d.cpu()), dict(logits=c.d[:5]), dict(logits=c.d.t().contiguous().t()),
                dict(scores=c.ds.double()), dict(tokens=c.tokens[:1]), dict(scores_out=c.out.half()), dict(parents=c.parents.long()),
                dict(done=torch.zeros(2, 3, device="cuda"), eos=1), dict(history=i32(6, 9)),
                dict(history=i32(6, 9), history_out=i32(6, 9)), dict(lse=c.lse[:1])):
        with pytest.raises(ValueError):
            B.tl_beam_select(**{**good, **bad})
    h = i32(6, 9)
    for bad in (dict(workspace=c.ws[:64]), dict(eos=100), dict(done=torch.zeros(2, 3, dtype=torch.uint8, device="cuda")),
                dict(history=h, history_out=i32(8, 9), length=9), dict(history=h, history_out=i32(8, 9), length=-1),
                dict(parents=i32(2, 65), tokens=i32(2, 65), scores_out=torch.zeros(2, 65, device="cuda"))):
        with pytest.raises(B.TLError):
            B.tl_beam_select(**{**good, **bad})
