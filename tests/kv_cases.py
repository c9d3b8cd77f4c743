"""Ragged batches over the 8-bit paged cache, shared by its tests: device tensors on one
side, float64 arrays for the oracle on the other, from one seed."""
import numpy as np
import torch

from oracle import kv_cache as ora


class Batch:
    """q[s] new tokens and len[s] tokens in all of each sequence; the pool's pages dealt out in random order."""

    def __init__(self, q, lens, *, H, Hkv, D, ps, seed=0, spare=1, order="hnd", extra_columns=0):
        self.rng = np.random.default_rng(seed)
        self.q, self.lens, self.H, self.Hkv, self.D, self.ps = list(q), list(lens), H, Hkv, D, ps
        need = [-(-n // ps) for n in lens]
        self.pages = sum(need) + spare
        deal = self.rng.permutation(self.pages)
        self.cols = max(need + [1]) + extra_columns
        self.table = np.full((len(q), self.cols), -1, np.int32)  # unused entries are never read
        at = 0
        for s, k in enumerate(need):
            self.table[s, :k] = deal[at:at + k]
            at += k
        self.cu = np.concatenate([[0], np.cumsum(self.q)]).astype(np.int32)
        self.n = int(self.cu[-1])
        self.order = order

    def pool(self, codes):
        """Codes [pages, H_kv, ps, D] as a device tensor of that shape, in the batch's memory order."""
        t = torch.from_numpy(codes)
        if self.order == "nhd":   # the tokens of a page outside, heads inside
            return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        return t.cuda()

    def both(self, kc, vc):
        """The two pools; order "kv" puts them in one buffer, page by page."""
        if self.order == "kv":
            t = torch.from_numpy(np.stack([kc, vc], 1)).cuda()
            return t[:, 0], t[:, 1]
        return self.pool(kc), self.pool(vc)

    def random_codes(self, spread=3):
        """Codes without NaN and scale bytes within 2^+-spread of 2^-6."""
        c = self.rng.integers(0, 127, (self.pages, self.Hkv, self.ps, self.D)).astype(np.uint8)
        # magnitudes like a normal variable's: mostly in the upper half of the exponents
        c = np.where(self.rng.random(c.shape) < 0.9, c % 56 + 64, c).astype(np.uint8)
        c |= (self.rng.integers(0, 2, c.shape) << 7).astype(np.uint8)
        return c, self.rng.integers(121 - spread, 122 + spread, (self.pages, self.Hkv)).astype(np.uint8)

    def bf16(self, *shape, scale=1.0):
        return (torch.from_numpy(self.rng.standard_normal(shape).astype(np.float32)) * scale).to(torch.bfloat16)

    def device(self):
        return (torch.from_numpy(self.cu).cuda(), torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                torch.from_numpy(self.table).cuda())


def tables(positions, rot, theta=10000.0):
    f = theta ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(positions)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def f64(t):
    return t.detach().cpu().double().numpy()


def expected_attention(b, q, kc, ks, vc, vs, causal, scale):
    """(O [n, H, D], lse [H, n], and the bounds' two magnitudes) of the whole batch in float64."""
    out, lse = np.zeros((b.n, b.H, b.D)), np.full((b.H, b.n), -np.inf)
    vmax, smax = np.zeros((b.n, b.H, 1)), np.zeros((b.n, b.H, 1))
    for s in range(len(b.q)):
        if b.q[s] == 0:
            continue
        rows = slice(b.cu[s], b.cu[s + 1])
        k = ora.values(kc, ks, b.table[s], b.lens[s])
        v = ora.values(vc, vs, b.table[s], b.lens[s])
        out[rows], lse[:, rows] = ora.attention(q[rows], k, v, causal, scale)
        if b.lens[s]:
            group = b.H // b.Hkv
            kk, vv = np.abs(np.nan_to_num(k)).repeat(group, 1), np.abs(np.nan_to_num(v)).repeat(group, 1)
            vmax[rows] = vv.max((0, 2))[None, :, None]
            smax[rows] = scale * np.einsum("thd,jhd->thj", np.abs(q[rows]), kk).max(2)[:, :, None]
    return out, lse, vmax, smax


def check_attention(got, lse_got, want, lse_want, vmax, smax):
    """Bounds counted from the roundings.

    A score is a sum of up to 128 products in fp32, taken sixteen at a time by the tensor cores, scaled and
    reduced by the maximum: at most 12 roundings of up to a whole step, 2^-23, of smax = scale * sum |q_d k_d|.
    The exponential adds 2^-21 of its result.  So a weight is off by w = 12 * 2^-23 * smax + 2^-20 of itself,
    and by 2^-11 more where P is rounded to fp16 for the second product.  O is a weighted mean of values of
    magnitude at most vmax, numerator and denominator off by as much: 2 (2^-11 + w) vmax, and its last rounding
    to bf16 by 2^-8 of it (a whole step, for results that fall on the other side of a border).  lse is off by w
    and by the fp32 roundings of its own magnitude.
    """
    got, lse_got = np.asarray(got), np.asarray(lse_got)
    assert got.shape == want.shape and lse_got.shape == lse_want.shape
    w = 12 * 2.0 ** -23 * smax + 2.0 ** -20
    tol = 2.0 ** -8 * np.abs(want) + 2 * (2.0 ** -11 + w) * vmax
    bad = ~(np.abs(got - want) <= tol) & ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), got[bad][:5], want[bad][:5])
    inf = np.isinf(lse_want)
    assert np.array_equal(inf, np.isinf(lse_got)) and np.all(lse_got[inf] == lse_want[inf])
    nan = np.isnan(lse_want)
    assert np.array_equal(nan, np.isnan(lse_got))
    fine = ~inf & ~nan
    d = np.abs(lse_got[fine] - lse_want[fine])
    assert (d <= w[..., 0].T[fine] + 2.0 ** -22 * np.abs(lse_want[fine])).all(), d.max()
