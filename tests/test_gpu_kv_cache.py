"""GPU tests of the paged cache against plain 64-bit forms on the CPU."""

import math

import numpy as np
import pytest
import torch

from kv_cache_utils import CAPS, EPS32, Pool, decode64, evict_row, key_weights64, live_mask, method_of
from parity_utils import Guarded
from soft_capped_attention_gb300 import capattn as ca

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def kv():
    from soft_capped_attention_gb300 import kv_cache
    return kv_cache


def params(cap, D, window=0, scale=None):
    c, a, b = CAPS[cap]
    return ca.AttnParams(sm_scale=scale or 1 / math.sqrt(D), cap_method=method_of(cap), cap=c, alpha=a, beta=b, causal=True,
                         window_len=window)


def check_decode(got, want, et, vmax, dtype, n_max, weights=None):
    """Bounds: t is off by at most et, so each P by 2 et relative (its own t and the
    sum's) plus a few roundings of exp; the outputs add n products (each step of an
    fp32 sum rounds by EPS32 of it) and one rounding to the output's type; P enters
    the tensor cores as two bf16 halves (2^-16 of it is lost)."""
    (o, lse), (o64, lse64, add64) = got, want
    half = torch.finfo(dtype).eps / 2
    o, lse = o.double().cpu(), lse.double().cpu()
    p_err = (2 * et + 16 * EPS32 + n_max * EPS32 + (2.0 ** -16 if dtype == BF16 else 0))[:, None, None]
    assert torch.isfinite(o).all()
    assert ((o - o64).abs() <= 1.0001 * half * o64.abs() + vmax * p_err).all(), float((o - o64).abs().max())
    empty = torch.isneginf(lse64)
    assert torch.equal(torch.isneginf(lse), empty)
    lse_err = et[:, None] + (8 + n_max) * EPS32 + 4 * EPS32 * lse64.abs()
    assert ((lse - lse64).abs()[~empty] <= lse_err.expand_as(lse)[~empty]).all()
    if weights is not None:
        before, after = weights
        n = add64.shape[2]
        sum64 = before[:, :, :n].double() + add64
        err = add64 * (2 * et[:, None, None] + (32 + n_max) * EPS32) + 4 * EPS32 * sum64
        assert ((after[:, :, :n].double() - sum64).abs() <= err).all()
        assert torch.equal(after[:, :, n:], before[:, :, n:])


DECODE = [
    # lens, Hq, Hkv, D, page, dtype, cap, window, temp, pos
    ([1], 1, 1, 128, 16, BF16, "none", 0, False, False),
    ([5, 0, 17], 2, 2, 64, 8, BF16, "tanh", 0, True, False),
    ([64, 63, 65, 128], 4, 2, 128, 16, BF16, "alsc", 0, False, False),
    ([300, 1, 777], 8, 2, 128, 32, BF16, "soft_sign", 0, True, False),
    ([1000, 33, 250], 6, 2, 128, 64, BF16, "tanh", 100, False, False),
    ([513, 511], 5, 1, 64, 128, BF16, "alsc", 64, True, False),
    ([700, 90], 16, 2, 128, 1024, BF16, "tanh", 0, False, False),
    ([400, 129], 32, 2, 128, 16, BF16, "none", 0, False, False),
    ([130, 257], 40, 2, 64, 32, BF16, "alsc", 0, True, False),
    ([600, 70, 0], 17, 1, 128, 16, BF16, "soft_sign", 1, False, False),
    ([3000, 10], 4, 4, 128, 64, BF16, "tanh", 0, True, True),
    ([900, 321], 8, 2, 64, 16, BF16, "alsc", 200, False, True),
    ([5000], 16, 1, 128, 16, BF16, "tanh", 0, False, False),
    ([20000], 4, 1, 128, 64, BF16, "alsc", 0, False, False),
    ([40] * 70, 8, 2, 64, 16, BF16, "none", 0, False, False),
    ([250, 0, 256, 3], 4, 2, 128, 16, BF16, "tanh", 0, True, False),      # whole groups
    ([500, 130] * 40, 4, 2, 128, 32, BF16, "soft_sign", 0, False, False),  # whole groups, many
    ([520, 130] * 40, 4, 2, 128, 32, BF16, "soft_sign", 0, False, False),  # the same, split
    ([800, 90], 8, 2, 128, 16, BF16, "tanh50", 0, True, False),
    ([800, 90], 24, 2, 64, 16, BF16, "tanh15", 0, False, False),
    ([800, 90], 4, 4, 128, 16, BF16, "alsc90", 0, False, False),
    ([800, 90], 16, 1, 64, 32, BF16, "alsc30", 300, True, False),
    ([1], 1, 1, 64, 8, FP32, "tanh", 0, False, False),
    ([100, 0, 33], 4, 2, 64, 16, FP32, "alsc", 0, True, False),
    ([1000, 31], 5, 1, 128, 32, FP32, "tanh", 100, False, False),
    ([500, 77], 40, 2, 64, 16, FP32, "soft_sign", 0, True, True),
    ([700, 300], 16, 2, 128, 64, FP32, "none", 77, False, True),
    ([9000], 2, 2, 64, 16, FP32, "tanh", 0, False, False),
]


# batches whose split takes several groups of sequences (and runs of groups)
LARGE = [(300, 70, 4, 2, 128, BF16), (9000, 20, 2, 1, 64, BF16), (700, 40, 3, 1, 64, FP32)]


@pytest.mark.parametrize("B,longest,Hq,Hkv,D,dtype", LARGE, ids=str)
def test_decode_of_large_batches(B, longest, Hq, Hkv, D, dtype):
    """Against fp32 on the GPU, every sequence: o within the types' roundings and the
    terms of check_decode for at most 70 keys (t below 40)."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    pool = Pool(lens, Hkv, D, 16, dtype, B)
    q = torch.randn(B, Hq, D, generator=g).to(dtype)
    ap = params("tanh", D)
    cache = pool.cuda()
    o, lse = kv().cache_decode(q.cuda(), cache, ap)
    n = pool.max_pages * 16
    gather = lambda x: torch.nan_to_num(x[cache.table.clamp(min=0).long()].transpose(1, 2).reshape(B, Hkv, n, D).double())  # noqa: E731
    s = torch.einsum("bhgd,bhnd->bhgn", q.cuda().double().reshape(B, Hkv, -1, D), gather(cache.k)) * ap.sm_scale
    t = ap.cap * torch.tanh(s / ap.cap)
    live = torch.arange(n, device="cuda") < cache.lens[:, None]
    t = t.masked_fill(~live[:, None, None], -math.inf)
    want = torch.einsum("bhgn,bhnd->bhgd", torch.nan_to_num(torch.softmax(t, -1)), gather(cache.v)).reshape(B, Hq, D)
    half = torch.finfo(dtype).eps / 2
    assert ((o.double() - want).abs() <= 1.0001 * half * want.abs() + 5 * 2.0 ** -13).all()
    assert torch.equal(torch.isneginf(lse), torch.isneginf(torch.logsumexp(t, -1).reshape(B, Hq)))
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("acc", [False, True], ids=["plain", "weights"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(str(x)[:24] for x in c))
def test_decode(case, acc):
    lens, Hq, Hkv, D, page, dtype, cap, window, with_temp, with_pos = case
    B, seed = len(lens), sum(lens) + Hq
    pool = Pool(lens, Hkv, D, page, dtype, seed)
    g = pool.gen
    q = (3 * torch.randn(B, Hq, D, generator=g)).to(dtype)
    temp = 1.5 * torch.rand(B, generator=g) - 0.25 if with_temp else None
    max_len = pool.max_pages * page
    pos = qpos = None
    if with_pos:  # distinct positions in no order; some heads' window is empty
        pos = torch.stack([torch.stack([torch.randperm(max_len, generator=g) for _ in range(Hkv)]) for _ in range(B)]).to(torch.int32)
        qpos = torch.full((B,), max_len + (window if B == 1 else 3), dtype=torch.int32)
    weights = torch.rand(B, Hkv, max_len, generator=g)
    ap = params(cap, D, window)
    o64, lse64, add64, et = decode64(q, pool.k, pool.v, pool.table, lens, ap, temp, pos, qpos)
    cache = pool.cuda(weights=weights, pos=pos, qpos=qpos)
    tt = temp.cuda() if temp is not None else None
    go, gl = Guarded((B, Hq, D), dtype), Guarded((B, Hq), FP32)
    o, lse = kv().cache_decode(q.cuda(), cache, ap, temp=tt, accumulate=acc, out=(go.tensor, gl.tensor))
    torch.cuda.synchronize()
    assert cache.status() == (0, 0)
    assert go.intact() and gl.intact()
    vmax = float(torch.nan_to_num(pool.v.float()).abs().max())
    w = (weights, cache.weights.cpu()) if acc else None
    check_decode((o, lse), (o64, lse64, add64), et, vmax, dtype, max(lens), w)
    # the same bits again, whatever ran before
    if acc:
        cache.weights.copy_(weights)
    o2, lse2 = kv().cache_decode(q.cuda(), cache, ap, temp=tt, accumulate=acc)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if acc:
        assert torch.equal(cache.weights.cpu(), w[1])


def test_decode_reads_shared_pages_and_strided_queries():
    """Three candidates behind one history: the tables share the history's pages."""
    pool = Pool([256 + 5, 256 + 9, 256 + 1], 2, 128, 64, BF16, 3)
    pool.table[1:, :4] = pool.table[0, :4]
    fused = torch.randn(3, 8 * 128 + 512).to(BF16)
    q = fused[:, :1024].unflatten(1, (8, 128))
    ap = params("alsc", 128)
    o64, lse64, add64, et = decode64(q, pool.k, pool.v, pool.table, pool.lens, ap)
    cache = pool.cuda()
    o, lse = kv().cache_decode(fused.cuda()[:, :1024].unflatten(1, (8, 128)), cache, ap)
    check_decode((o, lse), (o64, lse64, add64), et, 5.0, BF16, 300)


def test_decode_reads_pages_past_32_bit_offsets():
    """Pages that start 4.3e9 elements into the cache."""
    big = torch.empty(((1 << 32) // (2 * 64 * 128) + 9, 2, 64, 128), dtype=BF16, device="cuda")
    vig = torch.empty_like(big)
    pool = Pool([200], 2, 128, 64, BF16, 5, spare=0)
    last = big.shape[0] - 4 + torch.arange(4)
    big[last], vig[last] = pool.k[pool.table[0].long()].cuda(), pool.v[pool.table[0].long()].cuda()
    table = last.to(torch.int32)[None].cuda()
    cache = kv().KVCache(big, vig, table, torch.tensor([201], dtype=torch.int32, device="cuda"))
    new = torch.randn(2, 1, 2, 128).to(BF16)
    kv().cache_append(cache, new[0].cuda(), new[1].cuda())
    page, slot = int(pool.table[0, 3]), 200 % 64
    pool.k[page, :, slot], pool.v[page, :, slot] = new[0, 0], new[1, 0]
    q = torch.randn(1, 4, 128).to(BF16)
    ap = params("tanh", 128)
    o64, lse64, add64, et = decode64(q, pool.k, pool.v, pool.table, [201], ap)
    o, lse = kv().cache_decode(q.cuda(), cache, ap)
    check_decode((o, lse), (o64, lse64, add64), et, 5.0, BF16, 201)
    w = torch.rand(1, 2, 256)
    cache.weights = w.cuda()
    before = big[last].cpu()  # the sequence's four pages
    src = kv().cache_evict(cache, 90, 2, 20).cpu()
    after = big[last].cpu()
    for h in range(2):
        want = evict_row(w[0, h].tolist(), None, 200, 201, 90, 2, 20)
        assert src[0, h].tolist() == want
        for dst, old in enumerate(want):
            assert torch.equal(after[dst // 64, h, dst % 64], before[old // 64, h, old % 64])
    assert cache.status() == (0, 0)


def test_nan_in_masked_slots_stays_out_and_in_live_ones_comes_through():
    pool = Pool([150], 1, 128, 16, BF16, 9)
    q = torch.randn(1, 4, 128).to(BF16).cuda()
    page = pool.table[0].tolist()
    for x in (pool.k, pool.v):  # slots 0..9 lie before the window
        x[page[0], :, :10] = math.nan
    cache, ap = pool.cuda(), params("tanh", 128, window=140)
    o, lse = kv().cache_decode(q, cache, ap)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    pos = torch.arange(160, dtype=torch.int32).expand(1, 1, -1).contiguous()
    cache = pool.cuda(pos=pos, qpos=torch.tensor([149], dtype=torch.int32))
    o2, lse2 = kv().cache_decode(q, cache, ap)
    assert torch.isfinite(o2).all() and torch.allclose(lse, lse2, rtol=0, atol=1e-5)
    o3, lse3 = kv().cache_decode(q, cache, params("tanh", 128, window=141))
    assert torch.isnan(o3).all() and torch.isnan(lse3).all()


APPEND = [
    # lens after, new rows, Hkv, D, page, dtype, stride padding, trailing rows
    ([7], [1], 1, 64, 8, BF16, 0, 0),
    ([900, 33, 1], [1, 1, 1], 8, 128, 16, BF16, 256, 0),
    ([100, 64, 0, 17], [37, 64, 0, 1], 2, 128, 32, BF16, 0, 5),
    ([2000, 5], [1999, 5], 3, 64, 64, FP32, 64, 2),
    ([130], [129], 16, 128, 128, FP32, 0, 0),
    ([5000, 1, 4000], [5000, 1, 3999], 4, 128, 1024, BF16, 0, 1),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x)[:24] for x in c))
def test_append(case):
    lens, new, Hkv, D, page, dtype, pad, trailing = case
    B, N = len(lens), sum(new) + trailing
    pool = Pool(lens, Hkv, D, page, dtype, N + page)
    g = pool.gen
    fused = [torch.randn(N, Hkv * D + pad, generator=g).to(dtype) for _ in range(2)]
    rows = [x[:, :Hkv * D].unflatten(1, (Hkv, D)) for x in fused]
    max_len = pool.max_pages * page
    weights = torch.rand(B, Hkv, max_len, generator=g)
    pos = torch.full((B, Hkv, max_len), -7, dtype=torch.int32)
    qpos = torch.randint(10000, 20000, (B,), generator=g).to(torch.int32)
    cu = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32)
    cache = pool.cuda(weights=weights, pos=pos, qpos=qpos)
    one = new == [1] * B and not trailing
    dev = [x.cuda()[:, :Hkv * D].unflatten(1, (Hkv, D)) for x in fused]
    kv().cache_append(cache, dev[0], dev[1], cu_new=None if one else cu.cuda())
    torch.cuda.synchronize()
    assert cache.status() == (0, 0)
    for b in range(B):
        for r in range(new[b]):
            slot = lens[b] - new[b] + r
            at = int(pool.table[b, slot // page])
            pool.k[at, :, slot % page] = rows[0][cu[b] + r]
            pool.v[at, :, slot % page] = rows[1][cu[b] + r]
        weights[b, :, lens[b] - new[b]:lens[b]] = 0
        pos[b, :, lens[b] - new[b]:lens[b]] = qpos[b] - new[b] + 1 + torch.arange(new[b])
    bits = lambda x: x.view(torch.int16 if x.dtype == BF16 else torch.int32)  # noqa: E731  (NaN and all)
    assert torch.equal(bits(cache.k.cpu()), bits(pool.k)) and torch.equal(bits(cache.v.cpu()), bits(pool.v))
    assert torch.equal(cache.weights.cpu(), weights) and torch.equal(cache.pos.cpu(), pos)


EVICT = [
    # lens, Hkv, D, page, dtype, budget, first, last, pos, kind of weights
    ([5], 1, 64, 8, BF16, 1, 0, 0, False, "random"),
    ([100, 3, 0, 64], 2, 128, 16, BF16, 64, 4, 10, False, "random"),
    ([65, 64, 63], 3, 64, 32, FP32, 64, 0, 64, False, "zeros"),
    ([1000, 777], 2, 128, 64, BF16, 500, 4, 100, True, "ties"),
    ([5000], 2, 64, 128, BF16, 4990, 0, 0, True, "random"),
    ([4097, 2049], 1, 128, 16, FP32, 33, 8, 25, False, "ties"),
    ([40000], 1, 64, 64, BF16, 5000, 4, 64, True, "random"),
    ([300, 300], 2, 64, 16, BF16, 100, 1, 1, False, "odd"),
]


@pytest.mark.parametrize("in_place", [False, True], ids=["out", "in_place"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "-".join(str(x)[:24] for x in c))
def test_evict(case, in_place):
    lens, Hkv, D, page, dtype, budget, first, last, with_pos, kind = case
    B = len(lens)
    pool = Pool(lens, Hkv, D, page, dtype, budget, max_len=max(max(lens), budget))
    g = pool.gen
    max_len = pool.max_pages * page
    w = torch.exp(2 * torch.randn(B, Hkv, max_len, generator=g))
    if kind == "zeros":
        w.zero_()
    elif kind == "ties":
        w = (w * 2).floor() / 8
    elif kind == "odd":  # signed zeros, infinities, NaN, negative numbers
        some = torch.randint(0, 8, w.shape, generator=g)
        for i, x in enumerate((-0.0, 0.0, math.inf, math.nan, -math.inf, -1.0)):
            w = torch.where(some == i, torch.tensor(x), w)
    pos = qpos = None
    if with_pos:
        pos = torch.stack([torch.stack([torch.randperm(2 * max_len, generator=g)[:max_len] for _ in range(Hkv)])
                           for _ in range(B)]).to(torch.int32)
        qpos = torch.full((B,), 2 * max_len - 1, dtype=torch.int32)
    cache = pool.cuda(weights=w, pos=pos, qpos=qpos)
    outs = [Guarded((B,), torch.int32), Guarded(w.shape, FP32), Guarded(w.shape, torch.int32)]
    out = None
    if not in_place:
        out = (outs[0].tensor, outs[1].tensor, outs[2].tensor if with_pos else None)
    src = kv().cache_evict(cache, budget, first, last, out=out)
    torch.cuda.synchronize()
    assert cache.status() == (0, 0)
    lens_out, w_out, pos_out = (cache.lens, cache.weights, cache.pos) if in_place else out
    assert in_place or all(x.intact() for x in outs)
    assert lens_out.tolist() == [min(n, budget) for n in lens]
    src, w_out = src.cpu(), w_out.cpu()
    want_k, want_v = pool.k.clone(), pool.v.clone()
    for b, n in enumerate(lens):
        for h in range(Hkv):
            newest = int(qpos[b]) if with_pos else n - 1
            want = evict_row(w[b, h].tolist(), pos[b, h].tolist() if with_pos else None, newest, n, budget, first, last)
            m = len(want)
            assert src[b, h, :m].tolist() == want and (src[b, h, m:] == -1).all()
            assert torch.equal(w_out[b, h, :m].view(torch.int32), w[b, h][want].view(torch.int32))
            if with_pos:
                assert torch.equal(pos_out[b, h, :m].cpu(), pos[b, h][want])
            for dst, old in enumerate(want):
                if dst != old:
                    to, fro = int(pool.table[b, dst // page]), int(pool.table[b, old // page])
                    want_k[to, h, dst % page] = pool.k[fro, h, old % page]
                    want_v[to, h, dst % page] = pool.v[fro, h, old % page]
    bits = lambda x: x.view(torch.int16 if x.dtype == BF16 else torch.int32)  # noqa: E731
    assert torch.equal(bits(cache.k.cpu()), bits(want_k)) and torch.equal(bits(cache.v.cpu()), bits(want_v))


def test_evict_past_the_keys_that_fit_shared_memory():
    """400,000 slots, of which a cluster's shared memory holds fewer; in place."""
    n, page, budget = 399_990, 1024, 150_001
    pool = Pool([n], 1, 64, page, BF16, 8)
    w = (torch.randn(1, 1, pool.max_pages * page, generator=pool.gen) * 3).round()  # many ties
    cache = pool.cuda(weights=w)
    before = cache.k.clone()
    src = kv().cache_evict(cache, budget, 3, 1000).cpu()[0, 0]
    want = torch.tensor(evict_row(w[0, 0].tolist(), None, n - 1, n, budget, 3, 1000), dtype=torch.int32)
    assert torch.equal(src, want)
    assert cache.lens.tolist() == [budget]
    assert torch.equal(cache.weights[0, 0, :budget].cpu(), w[0, 0][want.long()])
    table = cache.table[0].long()
    at = lambda j: (table[j // page], j % page)  # noqa: E731
    new, old = torch.arange(budget, device="cuda"), want.long().cuda()
    (p0, s0), (p1, s1) = at(new), at(old)
    assert torch.equal(cache.k[p0, 0, s0].view(torch.int16), before[p1, 0, s1].view(torch.int16))
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("n, heads, budget, first, last", [
    (700, 2, 203, 0, 0), (2048, 80, 2047, 3, 3), (4095, 80, 1026, 5, 2), (9000, 2, 4097, 0, 17), (70_001, 1, 33_335, 2, 1),
    (400_000, 1, 7, 3, 4), (400_000, 1, 399_999, 0, 0),
])
@pytest.mark.parametrize("kind", ["equal", "zeros", "nan", "lowest", "close", "two"])
def test_evict_of_keys_alike(n, heads, budget, first, last, kind):
    """Weights whose leading digits are the same for few, many or all slots, budgets off
    whole vectors, one to eight CTAs a row with and without the keys in shared memory."""
    page = 1024 if n > 10_000 else 64
    pool = Pool([n], heads, 64, page, BF16, n + budget)
    shape = (1, heads, pool.max_pages * page)
    if kind == "close":  # within 2^-13 of one another, most of them different
        w = 1 + torch.randint(0, 1000, shape, generator=pool.gen) * 2.0**-23
    elif kind == "two":  # 1 in 20 of another value
        w = torch.where(torch.randint(0, 20, shape, generator=pool.gen) == 0, 0.75, 0.5)
    else:
        w = torch.full(shape, {"equal": 0.3, "zeros": 0.0, "nan": math.nan, "lowest": -math.inf}[kind])
    w = w.float()
    cache = pool.cuda(weights=w)
    before = cache.k.clone()
    src = kv().cache_evict(cache, budget, first, last).cpu()
    assert cache.status() == (0, 0) and cache.lens.tolist() == [budget]
    table = cache.table[0].long()
    new = torch.arange(budget, device="cuda")
    for h in range(heads):
        want = torch.tensor(evict_row(w[0, h].tolist(), None, n - 1, n, budget, first, last), dtype=torch.int32)
        assert torch.equal(src[0, h], want)
        assert torch.equal(cache.weights[0, h, :budget].cpu().view(torch.int32), w[0, h][want.long()].view(torch.int32))
        old = want.long().cuda()
        assert torch.equal(cache.k[table[new // page], h, new % page].view(torch.int16),
                           before[table[old // page], h, old % page].view(torch.int16))


WEIGHTS = [
    # B, L, Lk, Hq, Hkv, D, dtype, cap, causal, window, temp, mask, rows
    (1, 1, 1, 1, 1, 128, BF16, "none", True, 0, False, None, None),
    (2, 130, 130, 4, 2, 128, BF16, "tanh", True, 0, False, None, [[0, 130], [5, 77]]),
    (1, 300, 300, 8, 2, 64, BF16, "alsc", True, 50, True, None, [[236, 300]]),
    (2, 257, 257, 3, 3, 128, BF16, "soft_sign", False, 0, True, "seg", [[0, 0], [0, 257]]),
    (2, 200, 200, 5, 1, 64, BF16, "tanh", False, 0, False, "ranker", None),
    (1, 100, 333, 4, 4, 128, BF16, "alsc", False, 0, False, None, None),
    (1, 333, 100, 4, 2, 128, BF16, "none", True, 30, False, None, None),
    (1, 700, 700, 2, 1, 128, BF16, "tanh", True, 0, True, "seg", None),
    (1, 2500, 2500, 4, 2, 64, BF16, "alsc", True, 0, False, None, [[100, 2400]]),
    (3, 640, 640, 6, 3, 128, BF16, "none", True, 200, True, None, [[0, 640], [639, 640], [128, 512]]),
    (2, 400, 400, 4, 2, 128, BF16, "tanh50", True, 0, True, None, None),
    (1, 400, 400, 4, 4, 64, BF16, "tanh15", True, 90, False, None, None),
    (1, 400, 400, 4, 2, 128, BF16, "alsc30", True, 0, True, None, None),
    (1, 400, 400, 2, 2, 64, BF16, "alsc90", False, 0, False, "ranker", None),
    (2, 150, 150, 4, 2, 64, FP32, "tanh", True, 0, True, None, [[1, 2], [0, 150]]),
    (1, 129, 129, 2, 2, 128, FP32, "alsc", False, 0, False, "ranker", None),
    (1, 65, 200, 2, 2, 64, FP32, "soft_sign", False, 9, False, None, None),
]


@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: "-".join(str(x)[:24] for x in c))
def test_key_weights(case):
    B, L, Lk, Hq, Hkv, D, dtype, cap, causal, window, with_temp, mask, rows = case
    g = torch.Generator().manual_seed(L + Hq)
    q, k = ((2 * torch.randn(B, n, h, D, generator=g)).to(dtype) for n, h in ((L, Hq), (Lk, Hkv)))
    temp = 1.5 * torch.rand(B, L, generator=g) - 0.25 if with_temp else None
    seg = bounds = None
    if mask == "seg":
        seg = torch.cumsum((torch.rand(B, L, generator=g) < 0.02).int(), 1).to(torch.int32)
    elif mask == "ranker":
        bounds = torch.tensor([[3 * b, 60 + b, 60 + b, 90 + b] for b in range(B)], dtype=torch.int32)
    c, a, be = CAPS[cap]
    ap = ca.AttnParams(sm_scale=1 / math.sqrt(D), cap_method=method_of(cap), cap=c, alpha=a, beta=be, causal=causal,
                         window_len=window)
    live = live_mask(B, L, Lk, causal, window, seg, bounds)
    d = lambda x: None if x is None else x.cuda()  # noqa: E731
    _, lse, _, _ = ca.capattn_fwd(q.cuda(), k.cuda(), k.cuda().clone(), ap, d(temp), d(seg), d(bounds))
    rt = torch.tensor(rows, dtype=torch.int32) if rows is not None else None
    w64, et = key_weights64(q, k, lse.cpu(), ap, live, temp, rt)
    guard = Guarded((B, Hkv, Lk + 5), FP32)
    guard.tensor.fill_(-3.0)
    w = kv().key_weights(q.cuda(), k.cuda(), lse, ap, d(temp), d(seg), d(bounds), rows=d(rt), out=guard.tensor).cpu()
    assert guard.intact() and (w[..., Lk:] == -3.0).all()
    # each P is off by et (its t; the lse is an input) and a few roundings of exp and
    # of t - lse; a key's sum has at most L * G terms, in fp32
    t_max = float(lse[torch.isfinite(lse)].abs().max()) + 40
    err = w64 * (et + 2 * EPS32 * t_max + (16 + L * Hq // Hkv) * EPS32) + 1e-30
    assert ((w[..., :Lk].double() - w64).abs() <= err).all(), float(((w[..., :Lk].double() - w64).abs() / (w64 + 1e-30)).max())
    again = kv().key_weights(q.cuda(), k.cuda(), lse, ap, d(temp), d(seg), d(bounds), rows=d(rt))
    assert torch.equal(again.cpu(), w[..., :Lk])


def test_bad_device_data_is_flagged_and_harmless():
    ap = params("tanh", 128)
    q = torch.randn(2, 4, 128).to(BF16).cuda()
    for what, bit in (("long", 32), ("negative", 32), ("page", 64)):
        pool = Pool([100, 50], 2, 128, 16, BF16, 1)
        if what == "page":
            pool.table[1, 2] = pool.k.shape[0]
        w = torch.rand(2, 2, pool.max_pages * 16)
        cache = pool.cuda(weights=w)
        if what != "page":
            cache.lens[1] = 10 ** 6 if what == "long" else -5
        good = kv().cache_decode(q, pool.cuda(), ap)[0][0]
        bits = lambda: cache.status()[1]  # noqa: E731
        o, _ = kv().cache_decode(q, cache, ap)
        assert torch.equal(o[0], good)  # the other sequence is untouched
        assert bits() & bit
        new = torch.zeros(2, 2, 128, dtype=BF16, device="cuda")
        if what != "page":
            kv().cache_append(cache, new, new)
            assert bits() == bit
        kv().cache_evict(cache, 20, out=(torch.zeros_like(cache.lens), torch.zeros_like(cache.weights), None))
        assert bits() & bit
        assert cache.status() == (0, 0)


def test_append_flags_bad_rows():
    pool = Pool([10, 20], 1, 64, 16, BF16, 2)
    new = torch.ones(40, 1, 64, dtype=BF16, device="cuda")
    for cu in ([0, 11, 12], [0, 30, 10]):
        cache = pool.cuda()
        kv().cache_append(cache, new, new, cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert cache.status() == (6, 128)
    cache = pool.cuda()
    kv().cache_append(cache, new[:2], new[:2])
    bad = pool.cuda()
    bad.table.fill_(99)
    kv().cache_append(bad, new[:2], new[:2])
    assert bad.status() == (6, 64)
    assert torch.equal(bad.k.cpu().view(torch.int16), pool.k.view(torch.int16))


def test_key_weights_flags_bad_rows():
    q = torch.randn(1, 100, 2, 64).to(BF16).cuda()
    ap = params("none", 64)
    _, lse, _, _ = ca.capattn_fwd(q, q, q, ap)
    ws = kv().new_key_weights_workspace(q, q, ap)
    w = kv().key_weights(q, q, lse, ap, rows=torch.tensor([[-4, 200]], dtype=torch.int32, device="cuda"), workspace=ws)
    assert ca.capattn_device_status(ws) == (6, 256)
    assert torch.equal(w, kv().key_weights(q, q, lse, ap, workspace=ws))
    assert ca.capattn_device_status(ws) == (0, 0)


def test_refusals_of_the_binding():
    pool = Pool([100, 50], 2, 128, 16, BF16, 1)
    cache, ap = pool.cuda(), params("tanh", 128)
    q = torch.randn(2, 4, 128).to(BF16).cuda()
    new = torch.zeros(2, 2, 128, dtype=BF16, device="cuda")
    for call, match in [
        (lambda: kv().cache_decode(q[:1], cache, ap), "q: want"),
        (lambda: kv().cache_decode(q.float(), cache, ap), "q: want"),
        (lambda: kv().cache_decode(q.cpu(), cache, ap), "q: want"),
        (lambda: kv().cache_decode(q.transpose(0, 1).contiguous().transpose(0, 1), cache, ap), "contiguous"),
        (lambda: kv().cache_decode(q, cache, ap, accumulate=True), "weights"),
        (lambda: kv().cache_decode(q, cache, ap, temp=torch.ones(3, device="cuda")), "temp: want"),
        (lambda: kv().cache_append(cache, new[:1], new[:1]), "one new row"),
        (lambda: kv().cache_append(cache, new, new.float()), "v_new: want"),
        (lambda: kv().cache_append(cache, new, new, cu_new=torch.zeros(2, dtype=torch.int32, device="cuda")), "cu_new"),
        (lambda: kv().cache_evict(cache, 20), "weights"),
        (lambda: kv().KVCache(cache.k, cache.v, cache.table, cache.lens, pos=torch.zeros(2, 2, 112, dtype=torch.int32, device="cuda")), "qpos"),
        (lambda: kv().KVCache(cache.k, cache.v, cache.table.long(), cache.lens), "table"),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
    good, cache.lens = cache.lens, cache.lens.long()  # a replaced tensor is checked too
    with pytest.raises(ValueError, match="lens: want"):
        kv().cache_decode(q, cache, ap)
    cache.lens, cache.k = good, cache.k[:-1]
    with pytest.raises(ValueError, match="k and v"):
        kv().cache_append(cache, new, new)
    cache.k = cache.v.clone()
    with pytest.raises(ca.CapattnError, match="invalid argument"):
        kv().cache_decode(torch.zeros(2, 5, 128, dtype=BF16, device="cuda"), cache, ap)
    cache = pool.cuda(weights=torch.zeros(2, 2, 112))
    with pytest.raises(ValueError, match="budget"):
        kv().cache_evict(cache, 113)
    with pytest.raises(ValueError, match="budget"):
        kv().cache_evict(cache, 10, 6, 5)


def test_a_served_sequence_from_prompt_to_eviction_and_on():
    """Prompt (capattn_fwd), append, key_weights, decoding steps under one captured
    graph on a side stream, eviction, more steps: every step against a cache kept
    as plain per-head lists."""
    B, Hq, Hkv, D, page, max_pages, budget = 2, 4, 2, 64, 16, 12, 40
    prompt = [70, 45]
    g = torch.Generator().manual_seed(11)
    ap = params("alsc", D, window=60)
    L = max(prompt)
    q, k, v = ((torch.randn(B, L, h, D, generator=g)).to(BF16) for h in (Hq, Hkv, Hkv))
    max_len = page * max_pages
    pool = torch.full((B * max_pages, Hkv, page, D), math.nan, dtype=BF16, device="cuda")
    table = torch.randperm(B * max_pages, generator=g).to(torch.int32).reshape(B, max_pages).cuda()
    zeros = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    cache = kv().KVCache(pool, pool.clone(), table, torch.tensor(prompt, dtype=torch.int32).cuda(),
                         weights=zeros(B, Hkv, max_len, t=FP32), pos=zeros(B, Hkv, max_len),
                         qpos=torch.tensor(prompt, dtype=torch.int32).cuda() - 1)
    o, lse, _, _ = ca.capattn_fwd(q.cuda(), k.cuda(), v.cuda(), ap)
    packed = [torch.cat([x[b, :n] for b, n in enumerate(prompt)]).cuda() for x in (k, v)]
    cu = torch.tensor([0, prompt[0], sum(prompt)], dtype=torch.int32).cuda()
    kv().cache_append(cache, *packed, cu_new=cu)
    rows = torch.tensor([[0, n] for n in prompt], dtype=torch.int32).cuda()
    kv().key_weights(q.cuda(), k.cuda(), lse, ap, rows=rows, out=cache.weights)
    live = live_mask(B, L, L, True, 60)
    w64, _ = key_weights64(q, k, lse.cpu(), ap, live, rows=rows.cpu())
    # the plain cache: per (b, head) lists of (key, value, weight, position)
    plain = [[[[k[b, j, h], v[b, j, h], float(w64[b, h, j]), j] for j in range(n)] for h in range(Hkv)] for b, n in enumerate(prompt)]

    qs, ks, vs = zeros(B, Hq, D, t=BF16), zeros(B, Hkv, D, t=BF16), zeros(B, Hkv, D, t=BF16)
    os, ls = zeros(B, Hq, D, t=BF16), zeros(B, Hq, t=FP32)

    def step():
        cache.lens.add_(1)
        cache.qpos.add_(1)
        kv().cache_append(cache, ks, vs)
        kv().cache_decode(qs, cache, ap, accumulate=True, out=(os, ls))

    side = torch.cuda.Stream()
    saved = [x.clone() for x in (cache.lens, cache.qpos, cache.weights, cache.pos)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # the workspace grows here, before the capture
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((cache.lens, cache.qpos, cache.weights, cache.pos), saved):
        x.copy_(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    def check_step():
        new = [torch.randn(B, h, D, generator=g).to(BF16) for h in (Hq, Hkv, Hkv)]
        for dst, x in zip((qs, ks, vs), new):
            dst.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        newest = cache.qpos.tolist()
        for b in range(B):
            for h in range(Hkv):
                plain[b][h].append([new[1][b, h], new[2][b, h], 0.0, newest[b]])
                cells = plain[b][h]
                kk, vv = (torch.stack([c[i] for c in cells]).double() for i in (0, 1))
                s = new[0][b, 2 * h:2 * h + 2].double() @ kk.T * ap.sm_scale
                from kv_cache_utils import cap64
                t = cap64(s, ap.cap_method, ap.cap, ap.alpha, ap.beta)
                at = torch.tensor([c[3] for c in cells])
                t = t.masked_fill(at <= newest[b] - ap.window_len, -math.inf)
                p = torch.softmax(t, -1)
                # bf16 outputs: half a step of the value, the rest as in check_decode (t below 40)
                assert ((os[b, 2 * h:2 * h + 2].double().cpu() - p @ vv).abs() <= 2 ** -8 * (p @ vv).abs() + 5 * 1e-4).all()
                assert ((ls[b, 2 * h:2 * h + 2].double().cpu() - torch.logsumexp(t, -1)).abs() <= 1e-4).all()
                for c, x in zip(cells, p.sum(0).tolist()):
                    c[2] += x
                n = len(cells)
                got = cache.weights[b, h, :n].double().cpu()
                want = torch.tensor([c[2] for c in cells], dtype=torch.float64)
                assert ((got - want).abs() <= 1e-4 * want + 1e-6).all()
                assert cache.pos[b, h, :n].tolist() == [c[3] for c in cells]

    for _ in range(5):
        check_step()
    for _ in range(2):
        weights = cache.weights.cpu()  # the kernel's own weights decide near ties
        lens, newest = cache.lens.tolist(), cache.qpos.tolist()
        src = kv().cache_evict(cache, budget, keep_first=2, keep_last=8).cpu()
        for b in range(B):
            for h in range(Hkv):
                want = evict_row(weights[b, h].tolist(), [c[3] for c in plain[b][h]], newest[b], lens[b], budget, 2, 8)
                assert src[b, h, :len(want)].tolist() == want
                plain[b][h] = [plain[b][h][j] for j in want]
        assert cache.lens.tolist() == [min(n, budget) for n in lens]
        for _ in range(4):
            check_step()
    assert cache.status() == (0, 0)


def test_calls_on_a_given_stream():
    """Everything on a side stream while the default one is busy elsewhere."""
    pool = Pool([333, 120], 2, 128, 16, BF16, 4)
    ap = params("tanh", 128)
    q = torch.randn(2, 8, 128).to(BF16).cuda()
    want = kv().cache_decode(q, pool.cuda(), ap)
    cache, side = pool.cuda(), torch.cuda.Stream()
    torch.cuda.synchronize()
    o, lse = kv().cache_decode(q, cache, ap, stream=side)
    side.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert cache.status(stream=side) == (0, 0)


def test_two_caches_over_the_same_tensors_on_two_streams():
    """Calls that overlap need a KVCache each; the tensors may be the same."""
    pool = Pool([5000, 3100], 2, 128, 16, BF16, 21)
    ap = params("tanh", 128)
    q = [torch.randn(2, 8, 128).to(BF16).cuda() for _ in range(2)]
    one = pool.cuda()
    two = kv().KVCache(one.k, one.v, one.table, one.lens)
    want = [kv().cache_decode(x, one, ap) for x in q]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, cache in enumerate((one, two)):
            got[i].append(kv().cache_decode(q[i], cache, ap, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]) for o, lse in got[i])


def test_a_graph_outlives_a_larger_workspace():
    """A graph captured before the cache's workspace grew still replays, and a growth
    during a capture is refused."""
    pool = Pool([900, 333], 2, 128, 16, BF16, 22)
    ap = params("alsc", 128)
    q = torch.randn(2, 4, 128).to(BF16).cuda()
    cache = pool.cuda(weights=torch.zeros(2, 2, pool.max_pages * 16))
    want, _ = kv().cache_decode(q, cache, ap)
    out = (torch.zeros_like(want), torch.zeros(2, 4, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv().cache_decode(q, cache, ap, out=out)
    with pytest.raises(RuntimeError, match="grow"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            kv().cache_decode(q, cache, ap, accumulate=True, out=out)
    torch.cuda.synchronize()
    kv().cache_decode(q, cache, ap, accumulate=True)
    filler = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    out[0].zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want) and len(filler) == 64
    total = cache.weights[0, 0, :900].sum().item()  # two query heads a group, one step
    assert abs(total - 2.0) < 1e-4 and cache.status() == (0, 0)


def test_empty_batch_of_rows_appends_nothing():
    pool = Pool([10], 1, 64, 16, BF16, 6)
    cache = pool.cuda()
    none = torch.zeros(0, 1, 64, dtype=BF16, device="cuda")
    kv().cache_append(cache, none, none, cu_new=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert np.array_equal(cache.k.cpu().view(torch.int16).numpy(), pool.k.view(torch.int16).numpy())
