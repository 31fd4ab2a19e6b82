"""GPU tests of attention over the paged cache under caps so wide, or temperatures so large, that
the scores lie far inside their bound."""

import math

import pytest
import torch

from kv_cache_utils import Pool
from paged_cases import MANY_PIECES
from paged_ref import Attend, check
from soft_capped_attention_gb300 import capattn as ca
from test_gpu_kv_cache import BF16, FP32
from test_gpu_paged import a_tree, i32, paged, run, sums

pytestmark = pytest.mark.gpu

# bounds of x in log2 units: 115, 121 (either side of the rule), 216, 433, 1443; 577; 130, 411, 137 (below 0: 1150)
WIDE = [("tanh", 80.0, 0, 0), ("tanh", 84.0, 0, 0), ("tanh", 150.0, 0, 0), ("tanh", 300.0, 0, 0), ("tanh", 1000.0, 0, 0),
        ("soft_sign", 400.0, 0, 0), ("alsc", 66.0, 2.0, 0.5), ("alsc", 209.0, 2.0, 0.5), ("alsc", 84.0, 2.0, 1.06)]


def ap_of(cap, D, window=0, scale=None):
    method, c, a, b = cap
    return ca.AttnParams(sm_scale=scale or 1 / math.sqrt(D), cap_method=method, cap=c, alpha=a, beta=b, causal=True, window_len=window)


@pytest.mark.parametrize("tree", [False, True], ids=["prompt", "tree"])
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (FP32, 64)], ids=str)
@pytest.mark.parametrize("scale", [1.0, 20.0])
@pytest.mark.parametrize("cap", WIDE, ids=str)
def test_wide_caps(cap, scale, dtype, D, tree):
    pool = Pool([700, 40, 130], 2, D, 16, dtype, 3)
    got, want = run(pool, [150, 40, 7], 4, ap_of(cap, D), dtype, tree, seed=9, scale=scale, first=1, tail=2)
    check(got, want, dtype)


@pytest.mark.parametrize("name", MANY_PIECES)
@pytest.mark.parametrize("cap", [("tanh", 300.0, 0, 0), ("soft_sign", 400.0, 0, 0), ("alsc", 209.0, 2.0, 0.5)], ids=lambda c: c[0])
def test_many_pieces_under_wide_caps(cap, name):
    lens, new, Hq, Hkv, page, window, tree, _ = MANY_PIECES[name]
    D = 64 if cap[0] == "tanh" else 128
    pool = Pool(lens, Hkv, D, page, BF16, 4)
    q = torch.randn(sum(new), Hq, D, generator=pool.gen).bfloat16()
    up = a_tree(new, pool.gen) if tree else None
    ap, cache = ap_of(cap, D, window), pool.cuda()
    given = q.cuda(), cache, ap, i32(sums(new)), None if up is None else up.cuda()
    one = paged().cache_attend(*given)
    check(one, Attend(q, pool.k, pool.v, pool.table, lens, sums(new), ap, up), BF16)
    for _ in range(30):
        two = paged().cache_attend(*given)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("name", MANY_PIECES)
@pytest.mark.parametrize("cap", [("tanh", 50.0, 0, 0), ("soft_sign", 60.0, 0, 0), ("alsc", 30.0, 2.0, 0.5)], ids=lambda c: c[0])
def test_temperatures_that_widen_some_rows(cap, name):
    """Of 0.5 and 4 in runs of 40 rows, and batches whose CTAs get many pieces: the bound is wide in
    some of them, for some of a tile's rows."""
    lens, new, Hq, Hkv, page, window, tree, _ = MANY_PIECES[name]
    D = 64 if cap[0] == "tanh" else 128
    pool = Pool(lens, Hkv, D, page, BF16, 4)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(sum(new), Hq, D, generator=g).bfloat16()
    up = a_tree(new, g) if tree else None
    temp = torch.where(torch.arange(sum(new)) // 40 % 2 == 0, 0.5, 4.0)
    ap, cache = ap_of(cap, D, window), pool.cuda()
    given = q.cuda(), cache, ap, i32(sums(new)), None if up is None else up.cuda(), temp.cuda()
    one = paged().cache_attend(*given)
    check(one, Attend(q, pool.k, pool.v, pool.table, lens, sums(new), ap, up, temp), BF16)
    for _ in range(10):
        two = paged().cache_attend(*given)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert cache.status() == (0, 0)


def test_a_single_slot_gives_its_value_under_a_wide_cap():
    pool = Pool([300], 2, 128, 16, BF16, 3)
    q = torch.randn(300, 4, 128, generator=pool.gen).bfloat16().cuda()
    v = torch.stack([pool.v[pool.table[0][t // 16], :, t % 16] for t in range(300)]).repeat_interleave(2, 1).cuda()
    for cap in WIDE:
        o, _ = paged().cache_attend(q, pool.cuda(), ap_of(cap, 128, 1), i32([0, 300]))
        assert torch.equal(o, v), cap


def test_scores_at_both_ends_of_a_wide_cap():
    """The first keys' scores at one end of it, the later ones' at the other."""
    for sign in (1.0, -1.0):
        pool = Pool([900], 1, 128, 16, BF16, 4)
        for at, page in enumerate(pool.table[0, :57].long().tolist()):
            x = pool.k[page, :, :, 0]
            pool.k[page, :, :, 0] = torch.where(torch.isnan(x.float()), math.nan, sign * (-300.0 if at < 20 else 300.0)).to(BF16)
        for c in (150.0, 1000.0):
            got, want = run(pool, [130], 2, ap_of(("tanh", c, 0, 0), 128, scale=1.0), BF16, seed=2)
            check(got, want, BF16)


@pytest.mark.parametrize("cap,temp", [(150.0, 1.0), (300.0, 1.0), (1000.0, 1.0), (50.0, 4.0)])
def test_a_wide_cap_takes_no_longer(cap, temp):
    """A prompt of 2048 tokens: less than twice the time of a usual cap (nearer is measured
    elsewhere; row by row it would be far more)."""
    n, Hq, Hkv, D = 2048, 16, 4, 128
    pool = Pool([n], Hkv, D, 64, BF16, 3)
    q = torch.randn(n, Hq, D, generator=pool.gen).bfloat16().cuda()
    cache, cu, t = pool.cuda(), i32([0, n]), torch.full((n,), temp, device="cuda")

    def best(ap, temp):
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(200_000)  # the host runs ahead
            a.record()
            paged().cache_attend(q, cache, ap, cu, temp=temp)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    usual = best(ap_of(("tanh", 50.0, 0, 0), D), torch.ones_like(t))
    assert best(ap_of(("tanh", cap, 0, 0), D), t) < 2 * usual
    assert cache.status() == (0, 0)
