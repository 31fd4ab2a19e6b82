"""The decode's definition in 64 bits on the GPU, for batches and lengths too large for
kv_cache_utils.decode64, with bounds that follow the kernels' own depth of sums."""

import math

import torch

from kv_cache_utils import EPS32, cap64
from split_model import decode_ctas, pieces


class Want:
    """o, lse, the weights' additions; per (sequence, head) the sum of P |v| that o's
    roundings are relative to; per sequence the error of t and the largest |t|."""

    def __init__(self, q, cache, lens, ap, temp=None, tokens=200_000):
        B, Hq, D = q.shape
        Hkv, page = cache.Hkv, cache.page_size
        f8 = dict(dtype=torch.float64, device="cuda")
        self.o, self.size = torch.zeros(B, Hq, D, **f8), torch.zeros(B, Hq, D, **f8)
        self.lse = torch.full((B, Hq), -math.inf, **f8)
        self.add = torch.zeros(B, Hkv, cache.max_len, **f8)
        self.et, self.top = torch.zeros(B, **f8), torch.zeros(B, **f8)
        order = sorted((b for b in range(B) if lens[b]), key=lambda b: -lens[b])
        at = 0
        while at < len(order):
            n = lens[order[at]]
            b = torch.tensor(order[at:at + max(1, tokens // n)], device="cuda")
            at += len(b)
            self._some(q, cache, b, n, lens, ap, temp, page, Hkv, D)

    def _some(self, q, cache, b, n, lens, ap, temp, page, Hkv, D):
        m = len(b)
        table = cache.table[b, :-(-n // page)].clamp(min=0).long()
        rows = lambda x: torch.nan_to_num(x[table].transpose(1, 2).reshape(m, Hkv, -1, D)[:, :, :n].double())  # noqa: E731
        k, v = rows(cache.k), rows(cache.v)
        qb = q[b].double().reshape(m, Hkv, -1, D)
        length = torch.tensor([lens[int(x)] for x in b], device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        live = j < length
        if ap.window_len > 0:
            live &= j >= length - ap.window_len
        live = live[:, None, None]
        s = torch.matmul(qb, k.transpose(-1, -2)) * ap.sm_scale
        s = torch.where(live, s, 0.0)
        tb = torch.ones(m, 1, 1, 1, device="cuda", dtype=torch.float64) if temp is None else temp[b].double()[:, None, None, None]
        t = cap64(s, ap.cap_method, ap.cap, ap.alpha, ap.beta) * tb
        dots = torch.where(live, torch.matmul(qb.abs(), k.abs().transpose(-1, -2)), 0.0).amax((1, 2, 3))
        self.et[b] = tb.abs().flatten() * EPS32 * 1.5 * ((D + 8) * abs(ap.sm_scale) * dots + 16 * s.abs().amax((1, 2, 3)))
        self.top[b] = t.abs().amax((1, 2, 3))
        t = t.masked_fill(~live, -math.inf)
        norm = torch.logsumexp(t, -1)
        p = torch.exp(t - norm[..., None])
        self.o[b] = torch.matmul(p, v).reshape(m, -1, D)
        self.size[b] = torch.matmul(p, v.abs()).reshape(m, -1, D)
        self.lse[b] = norm.reshape(m, -1)
        self.add[b, :, :n] = p.sum(2)


def check(got, want, q, cache, lens, window, weights=None):
    """t is off by at most et; each exponential by 1.5 half steps of its argument (at
    most twice the largest |t|, and 8), twice (its own and the rescalings, whose
    arguments add up to no more), and 8 steps of its own.  A sum's depth is that of its
    longest piece (fp32: a tile of 32 keys adds 32 products and one rescaling; bf16: a
    warp's 16 keys of a tile in the tensor cores, counted as 8 half steps each of the two
    halves of P) and of the join.  bf16: 2^-16 of P is lost in its two halves."""
    (o, lse), dtype = got, got[0].dtype
    e = dtype.itemsize
    Hq, D = q.shape[1:]
    ps = pieces(lens, Hq, cache.Hkv, D, e, cache.max_len, window)
    tiles = max(p[4] for p in ps)
    split = {}
    for p in ps:
        split[p[1:3]] = split.get(p[1:3], 0) + 1
    join = max(split.values()) / 4 + 3 + 3 + 4
    groups = decode_ctas(lens, Hq, cache.Hkv, D, e, cache.max_len)[0] // 64  # of 16 keys a warp and tile (bf16)
    depth_l = 2 * tiles * max(1, groups) + 8 + join
    depth_o = (33 * tiles if e == 4 else 16 * tiles * groups) + join
    exps = (2 * 1.5 * (2 * want.top + 8) + 8) * EPS32
    half = torch.finfo(dtype).eps / 2
    p_err = 2 * want.et + 2 * exps + (depth_l + depth_o + 4) * EPS32 + (2.0 ** -16 if e == 2 else 0)
    assert torch.isfinite(o).all()
    off = (o.double() - want.o).abs()
    bound = 1.0001 * half * want.o.abs() + want.size * p_err[:, None, None]
    assert (off <= bound).all(), float((off / bound.clamp(min=1e-300)).max())
    empty = torch.isneginf(want.lse)
    assert torch.equal(torch.isneginf(lse), empty)
    # (a sequence without keys adds nothing: its lse enters no bound)
    lse_err = (want.et + exps + (depth_l + 4) * EPS32)[:, None] + 4 * EPS32 * torch.where(empty, 0.0, want.lse).abs()
    assert ((lse.double() - want.lse).abs() <= lse_err)[~empty].all()
    if weights is not None:
        before, after = weights
        total = before.double() + want.add
        part = (lse_err.amax(1) + want.et + exps)[:, None, None] + (Hq // cache.Hkv + 4) * EPS32
        assert ((after.double() - total).abs() <= want.add * part + 4 * EPS32 * total).all()
