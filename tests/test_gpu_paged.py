"""GPU tests of attention of many new tokens over the paged cache: prompts, chunks of
prompts and trees of drafted tokens, against plain 64-bit forms."""

import itertools
import math

import pytest
import torch

from kv_cache_utils import CAPS, Pool, method_of
from paged_ref import Attend, check
from soft_capped_attention_gb300 import capattn as ca
from test_gpu_kv_cache import BF16, FP32, params

pytestmark = pytest.mark.gpu


def paged():
    from soft_capped_attention_gb300 import paged
    return paged


def sums(new, first=0):
    return [first] + [first + x for x in itertools.accumulate(new)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def a_tree(new, gen, bushy=0.5):
    """Parents of packed rows: each continues an earlier row of its sequence, or (some) none."""
    up = []
    for n in new:
        for i in range(n):
            u = float(torch.rand((), generator=gen))
            up.append(-1 if i == 0 or u < 0.05 else int(i * (bushy + (1 - bushy) * u)) if u < 0.9 else i - 1)
            up[-1] = min(up[-1], i - 1)
    return torch.tensor(up, dtype=torch.int32)


def positions(pool, Hkv, gen, newest=None):
    """Positions of a cache whose tokens were moved about by evictions, the new ones last in order."""
    B, n = len(pool.lens), pool.max_pages * pool.page
    pos = torch.zeros(B, Hkv, n, dtype=torch.int32)
    qpos = []
    for b, L in enumerate(pool.lens):
        far = L + 50 if newest is None else newest
        for h in range(Hkv):
            pos[b, h, :L] = torch.sort(torch.randperm(far, generator=gen)[:L]).values.to(torch.int32)
            pos[b, h, :L] = pos[b, h, :L][torch.randperm(L, generator=gen)]
        qpos.append(far + 10)
    return pos, torch.tensor(qpos, dtype=torch.int32)


def run(pool, new, Hq, ap, dtype, tree=False, temp=False, pos=False, seed=0, first=0, tail=0, scale=1.0):
    """The call and its definition; `first` and `tail` rows belong to nobody."""
    g = torch.Generator().manual_seed(seed)
    Hkv, D = pool.k.shape[1], pool.k.shape[3]
    cu = sums(new, first)
    N = cu[-1] + tail
    q = (scale * torch.randn(N, Hq, D, generator=g)).to(dtype)
    t = 0.5 + torch.rand(N, generator=g) if temp else None
    up = torch.full((N,), 77, dtype=torch.int32) if tree else None
    if tree:
        up[first:cu[-1]] = a_tree(new, g)
    kw, ps, qp = {}, None, None
    if pos:
        ps, qp = positions(pool, Hkv, g)
        for b, n in enumerate(new):  # the new tokens' own, as append writes them
            ps[b, :, pool.lens[b] - n:pool.lens[b]] = qp[b] - n + 1 + torch.arange(n, dtype=torch.int32)
        kw = dict(pos=ps, qpos=qp)
    cache = pool.cuda(**kw)
    d = lambda x: None if x is None else x.cuda()  # noqa: E731
    o, lse = torch.full((N, Hq, D), 7.0, dtype=dtype, device="cuda"), torch.full((N, Hq), 7.0, device="cuda")
    paged().cache_attend(q.cuda(), cache, ap, i32(cu), parents=d(up), temp=d(t), out=(o, lse))
    assert cache.status() == (0, 0)
    want = Attend(q, pool.k, pool.v, pool.table, pool.lens, cu, ap, up, t, ps if ap.window_len else None, qp)
    for x in (o, lse):  # rows of nobody
        assert (x[:first] == 7).all() and (x[cu[-1]:] == 7).all()
    return (o, lse), want


CASES = [
    # lens, new, Hq, Hkv, D, page, dtype, cap, window, temp, pos
    ([1], [1], 1, 1, 128, 16, BF16, "none", 0, False, False),
    ([5, 3, 17], [2, 0, 17], 2, 2, 64, 8, BF16, "tanh", 0, True, False),
    ([128, 127, 129, 256], [128, 127, 1, 2], 4, 2, 128, 16, BF16, "alsc", 0, False, False),
    ([300, 1, 777], [300, 1, 77], 8, 2, 128, 32, BF16, "soft_sign", 0, True, False),
    ([1000, 33, 250], [90, 33, 129], 6, 2, 128, 64, BF16, "tanh", 100, False, False),
    ([513, 511], [513, 100], 5, 1, 64, 128, BF16, "alsc", 64, True, False),
    ([700, 90], [33, 90], 16, 2, 128, 1024, BF16, "tanh", 0, False, False),
    ([400, 129], [65, 64], 32, 2, 128, 16, BF16, "none", 0, True, False),
    ([130, 257], [4, 5], 40, 2, 64, 32, BF16, "alsc", 0, True, False),
    ([60, 7], [9, 2], 130, 1, 64, 16, BF16, "tanh50", 0, False, False),
    ([60, 7], [9, 2], 129, 1, 128, 16, BF16, "tanh50", 0, False, False),   # two unequal parts of a group
    ([600, 70, 9], [100, 70, 9], 17, 1, 128, 16, BF16, "soft_sign", 1, False, False),
    ([2000, 100], [40, 9], 4, 4, 128, 64, BF16, "tanh", 300, True, True),
    ([900, 321], [30, 100], 8, 2, 64, 16, BF16, "alsc", 200, False, True),
    ([5000], [70], 4, 1, 128, 16, BF16, "tanh50", 0, False, False),
    ([9000], [9], 4, 1, 128, 64, BF16, "alsc30", 0, False, False),
    ([40] * 70, [3, 0] * 35, 8, 2, 64, 16, BF16, "none", 0, False, False),
    ([800, 90], [200, 5], 24, 2, 64, 16, BF16, "tanh15", 0, False, False),
    ([800, 90], [200, 5], 4, 4, 128, 16, BF16, "alsc90", 0, False, False),
    ([800, 90], [130, 60], 16, 1, 64, 32, BF16, "alsc30", 300, True, False),
    ([700, 650], [700, 650], 3, 3, 128, 16, BF16, "none", 31, False, False),
    ([1], [1], 1, 1, 64, 8, FP32, "tanh", 0, False, False),
    ([100, 4, 33], [100, 0, 2], 4, 2, 64, 16, FP32, "alsc", 0, True, False),
    ([1000, 31], [64, 31], 5, 1, 128, 32, FP32, "tanh", 100, False, False),
    ([500, 77], [65, 3], 40, 2, 64, 16, FP32, "soft_sign", 90, True, True),
    ([700, 300], [17, 300], 16, 2, 128, 64, FP32, "none", 77, False, True),
    ([4000], [9], 2, 2, 64, 16, FP32, "tanh15", 0, False, False),
    ([60, 7], [9, 2], 70, 1, 128, 16, FP32, "alsc90", 0, False, False),
    ([60, 7], [9, 2], 65, 1, 64, 16, FP32, "tanh15", 0, True, False),
]


@pytest.mark.parametrize("tree", [False, True], ids=["prompt", "tree"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x)[:24] for x in c))
def test_attend(case, tree):
    lens, new, Hq, Hkv, D, page, dtype, cap, window, temp, pos = case
    pool = Pool(lens, Hkv, D, page, dtype, sum(lens) + Hq)
    got, want = run(pool, new, Hq, params(cap, D, window), dtype, tree, temp, pos, seed=sum(new), first=len(lens) % 3,
                    tail=sum(lens) % 4)
    check(got, want, dtype)


@pytest.mark.parametrize("cap,scale", [(20.0, 1.0), (20.0, 3.0), (4.0, 0.3)])
def test_soft_sign_near_zero(cap, scale):
    """Scores inside its polynomial's range, across it, and far below the cap."""
    pool = Pool([700, 90], 2, 128, 16, BF16, 5)
    ap = ca.AttnParams(sm_scale=1 / math.sqrt(128), cap_method="soft_sign", cap=cap, causal=True)
    got, want = run(pool, [200, 30], 4, ap, BF16, False, True, seed=3, scale=scale)
    check(got, want, BF16)


@pytest.mark.parametrize("tree", [False, True], ids=["prompt", "tree"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_many_sequences(dtype, tree):
    """More sequences than threads of a CTA, most of them without new tokens."""
    B = 1500
    lens = [(7 * b) % 50 + 1 for b in range(B)]
    new = [min(lens[b], b % 11) if b % 5 == 0 or b > 1480 else 0 for b in range(B)]
    pool = Pool(lens, 2, 64, 16, dtype, 5)
    got, want = run(pool, new, 4, params("tanh", 64), dtype, tree, True, first=2, tail=3)
    check(got, want, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cap,scale", [("none", 40.0), ("tanh", 40.0), ("alsc30", 60.0), ("soft_sign", 60.0)])
@pytest.mark.parametrize("tree", [False, True], ids=["prompt", "tree"])
def test_large_scores(dtype, cap, scale, tree):
    """Scores of hundreds, negative for every key of some rows; temperatures too."""
    pool = Pool([700, 40], 2, 128, 16, dtype, 3)
    pool.k[:, :, :, 0] = pool.k[:, :, :, 0].abs() + 1  # (NaN where no token is stays NaN)
    got, want = run(pool, [150, 40], 4, params(cap, 128), dtype, tree, True, seed=9, scale=scale)
    check(got, want, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cap", ["none", "tanh", "alsc30", "soft_sign"])
def test_temperatures_of_any_sign_and_size(dtype, cap):
    """0 (the plain mean), negative ones, tiny and large ones side by side in a tile."""
    pool = Pool([700, 40], 2, 128, 16, dtype, 3)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(190, 4, 128, generator=g).to(dtype)
    temp = torch.tensor([0.0, -1.0, 1e-3, 1.0, -0.3, 30.0, -20.0, 1e-30])[torch.randint(0, 8, (190,), generator=g)]
    ap, cu = params(cap, 128), [0, 150, 190]
    cache = pool.cuda()
    got = paged().cache_attend(q.cuda(), cache, ap, i32(cu), temp=temp.cuda())
    check(got, Attend(q, pool.k, pool.v, pool.table, pool.lens, cu, ap, temp=temp), dtype)
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 1 << 30, 900])
@pytest.mark.parametrize("pos", [False, True], ids=["slots", "pos"])
def test_windows_wider_than_the_cache(dtype, window, pos):
    pool = Pool([700, 40], 2, 64, 16, dtype, 3)
    for tree in (False, True):
        got, want = run(pool, [150, 40], 4, params("tanh15", 64, window), dtype, tree, pos=pos, seed=4)
        check(got, want, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("scale", [0.0, -0.1])
@pytest.mark.parametrize("cap", ["none", "tanh50", "alsc30", "soft_sign"])
def test_scales_of_any_sign(dtype, scale, cap):
    pool = Pool([300, 40], 2, 128, 16, dtype, 3)
    c, a, b = CAPS[cap]
    ap = ca.AttnParams(sm_scale=scale, cap_method=method_of(cap), cap=c, alpha=a, beta=b, causal=True)
    got, want = run(pool, [50, 40], 4, ap, dtype, False, True, seed=4)
    check(got, want, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_a_long_chain_of_drafts(dtype):
    """A tree that is one chain is a prompt, however long."""
    pool = Pool([700, 650], 2, 64, 16, dtype, 9)
    new = [600, 650]
    q = torch.randn(sum(new), 2, 64, generator=pool.gen).to(dtype).cuda()
    chain = torch.cat([torch.arange(-1, n - 1, dtype=torch.int32) for n in new]).cuda()
    cache, ap = pool.cuda(), params("tanh", 64, 77)
    one = paged().cache_attend(q, cache, ap, i32(sums(new)))
    two = paged().cache_attend(q, cache, ap, i32(sums(new)), parents=chain)
    want = Attend(q.cpu(), pool.k, pool.v, pool.table, pool.lens, sums(new), ap)
    check(one, want, dtype)
    check(two, want, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", ["none", "tanh", "alsc", "soft_sign"])
def test_a_single_slot_gives_its_value(dtype, D, cap):
    """First tokens, windows of one, drafts that continue nothing: o is v, to the bit."""
    new = [500, 1, 130]
    pool = Pool(new, 2, D, 16, dtype, 3)
    q = torch.randn(sum(new), 4, D, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()
    cache, cu = pool.cuda(), i32(sums(new))
    v = torch.cat([torch.cat([pool.v[pool.table[b][t // 16], :, t % 16][None] for t in range(n)]) for b, n in enumerate(new)])
    v = v.repeat_interleave(2, 1).cuda()
    roots = torch.full((sum(new),), -1, dtype=torch.int32).cuda()
    chain = torch.cat([torch.arange(-1, n - 1, dtype=torch.int32) for n in new]).cuda()
    for window, up in ((1, None), (1, chain), (0, roots), (40, roots)):
        o, lse = paged().cache_attend(q, cache, params(cap, D, window), cu, parents=up)
        assert torch.equal(o, v), (window, up is None)
    for up in (None, chain):
        o, lse = paged().cache_attend(q, cache, params(cap, D), cu, parents=up)
        first = [0, 500, 501]
        assert torch.equal(o[first], v[first])
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("dtype,step", [(BF16, 2.0 ** -8), (FP32, 2.0 ** -20)], ids=["bf16", "fp32"])
def test_the_longest_tree(dtype, step):
    """8192 tokens, a chain, which is a prompt: outputs within max |v| times half a step of P and half
    of o for either call, fp32's sums of 8192 terms within the usual few steps; a longer one is
    flagged and gives nothing."""
    n = 8192
    pool = Pool([n + 1], 1, 64, 16, dtype, 9)
    q = torch.randn(n + 1, 1, 64, generator=pool.gen).to(dtype).cuda()
    chain = torch.arange(-1, n, dtype=torch.int32).cuda()
    cache, ap = pool.cuda(), params("tanh", 64)
    one = paged().cache_attend(q[:n], cache, ap, i32([0, n]))
    two = paged().cache_attend(q[:n], cache, ap, i32([0, n]), parents=chain[:n])
    assert (one[0].double() - two[0].double()).abs().max() <= 4 * step * pool.v.double().nan_to_num(0).abs().max()
    assert (one[1] - two[1]).abs().max() <= 2 ** -18
    assert cache.status() == (0, 0)
    out = torch.full_like(q, 3), torch.full_like(q[:, :, 0], 3, dtype=torch.float32)
    paged().cache_attend(q, cache, ap, i32([0, n + 1]), parents=chain, out=out)
    assert all((x == 3).all() for x in out) and cache.status() == (6, 512)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_two_caches_on_two_streams(dtype):
    """Calls at once, each cache with a workspace of its own."""
    pools = [Pool([900, 40, 333], 2, 128, 16, dtype, s) for s in (1, 2)]
    caches, streams = [p.cuda() for p in pools], [torch.cuda.Stream() for _ in pools]
    q = torch.randn(300, 8, 128, generator=pools[0].gen).to(dtype).cuda()
    cu, ap = i32([0, 160, 190, 300]), params("alsc30", 128)
    want = [paged().cache_attend(q, c, ap, cu) for c in caches]
    torch.cuda.synchronize()
    got = [[paged().cache_attend(q, c, ap, cu, stream=s) for c, s in zip(caches, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for row in got:
        for x, y in zip(row, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,scale", [("none", 1), ("tanh", 1), ("alsc", 1), ("soft_sign", 1), ("tanh15", 1), ("tanh15", 0.02),
                                       ("tanh50", 3), ("alsc30", 0.01), ("alsc90", 1), ("soft_sign", 0.01)])
def test_what_lies_in_free_slots_changes_no_bit(dtype, D, cap, scale):
    """Slots behind a sequence's last token, of its page and of pages it has not, hold anything."""
    pool = Pool([300, 40, 7], 2, D, 64, dtype, 3)
    q = (scale * torch.randn(77, 4, D, generator=torch.Generator().manual_seed(6))).to(dtype).cuda()
    used = torch.zeros(pool.k.shape[0], pool.page, dtype=torch.bool)
    for b, L in enumerate(pool.lens):
        for t in range(L):
            used[pool.table[b][t // pool.page], t % pool.page] = True
    cu, up, kept = i32([0, 30, 70, 77]), a_tree([30, 40, 7], torch.Generator().manual_seed(1)).cuda(), []
    for junk in (0.0, 5.0, 1e4, -3e38, math.inf, math.nan):
        free = ~used[:, None, :, None].expand_as(pool.k)
        pool.k[free] = torch.tensor(junk).to(dtype)
        pool.v[free] = torch.tensor(-junk).to(dtype)
        cache = pool.cuda()
        for parents in (None, up):
            kept.append(paged().cache_attend(q, cache, params(cap, D), cu, parents=parents))
    for first in range(2):
        for o, lse in kept[first::2]:
            assert torch.equal(o, kept[first][0]) and torch.equal(lse, kept[first][1])


def test_a_first_tile_far_below_the_rest():
    """Without a cap: the first keys' scores say nothing of the later ones'."""
    for sign in (1.0, -1.0):
        pool = Pool([900], 1, 128, 16, BF16, 4)
        pages = pool.table[0, :57].long()
        for at, page in enumerate(pages.tolist()):
            pool.k[page, :, :, 0] = torch.where(torch.isnan(pool.k[page, :, :, 0].float()), math.nan, sign * (-300.0 if at < 20 else 300.0)).to(BF16)
        got, want = run(pool, [130], 2, params("none", 128, scale=1.0), BF16, seed=2)
        check(got, want, BF16)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("tree,window", [(False, 0), (True, 0), (False, 40), (True, 30)])
def test_what_is_not_live_stays_out(dtype, what, tree, window):
    """NaN or infinities in keys and values of new tokens, of window-expired ones and behind
    the lengths: rows that do not see them give what finite values there would."""
    lens, new = [300, 90], [70, 50]
    pool = Pool(lens, 2, 128, 16, dtype, 8)
    g = torch.Generator().manual_seed(1)
    up = a_tree(new, g) if tree else None
    cu = sums(new)
    q = torch.randn(cu[-1], 4, 128, generator=g).to(dtype)
    ap = params("tanh15", 128, window)
    bad = [(0, 300 - 70 + 33), (1, 90 - 50 + 20), (0, 3)] if window else [(0, 300 - 70 + 33), (1, 90 - 50 + 20)]
    want = Attend(q, pool.k, pool.v, pool.table, lens, cu, ap, up)
    sees = torch.zeros(cu[-1], dtype=torch.bool)
    from paged_ref import live_of
    for b, slot in bad:
        r = slice(cu[b], cu[b + 1])
        sees[r] |= live_of(new[b], lens[b], window, None if up is None else up[r].tolist())[0][:, slot]
        page = int(pool.table[b, slot // 16])
        pool.k[page, :, slot % 16, 5] = what
        pool.v[page, :, slot % 16] = what
    assert sees.any() and not sees.all()
    cache = pool.cuda()
    o, lse = paged().cache_attend(q.cuda(), cache, ap, i32(cu), parents=None if up is None else up.cuda())
    want.rows &= ~sees
    check((o, lse), want, dtype)
    if math.isnan(what):
        assert torch.isnan(lse.cpu()[sees]).all() and torch.isnan(o.cpu()[sees]).all()
    assert cache.status() == (0, 0)
    again = paged().cache_attend(q.cuda(), cache, ap, i32(cu), parents=None if up is None else up.cuda())
    assert torch.equal(again[0].view(torch.uint8), o.view(torch.uint8)) and torch.equal(again[1].view(torch.uint8), lse.view(torch.uint8))


def test_rows_without_live_slots():
    """Positions of a cache may say that a window reaches nothing, not even the row itself."""
    for dtype in (BF16, FP32):
        pool = Pool([200, 30], 2, 64, 16, dtype, 2)
        pos = torch.zeros(2, 2, pool.max_pages * 16, dtype=torch.int32)
        cache = pool.cuda(pos=pos, qpos=torch.tensor([500, 600], dtype=torch.int32))
        q = torch.randn(60, 4, 64, generator=pool.gen).to(dtype).cuda()
        o, lse = paged().cache_attend(q, cache, params("tanh", 64, 100), i32([0, 40, 60]))
        assert (o == 0).all() and torch.isneginf(lse).all() and cache.status() == (0, 0)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_rows_of_a_fused_projection(dtype):
    pool = Pool([300, 90], 2, 128, 16, dtype, 6)
    fused = torch.randn(100, 8 * 128 + 64, generator=pool.gen).to(dtype)
    q = fused[:, 64:64 + 4 * 128].unflatten(1, (4, 128))
    cache, ap = pool.cuda(), params("tanh", 128)
    got = paged().cache_attend(fused.cuda()[:, 64:64 + 4 * 128].unflatten(1, (4, 128)), cache, ap, i32([0, 70, 100]))
    check(got, Attend(q, pool.k, pool.v, pool.table, pool.lens, [0, 70, 100], ap), dtype)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tree", [False, True], ids=["prompt", "tree"])
def test_same_bits_and_replays(dtype, tree):
    """Runs in a row, and a captured one replayed with other inputs, lengths and trees."""
    pool = Pool([3000, 500, 64], 2, 128, 16, dtype, 7)
    g = pool.gen
    new = [40, 100, 64]
    cu, N = i32(sums(new)), sum(new)
    q = torch.randn(N, 8, 128, generator=g).to(dtype).cuda()
    up = a_tree(new, g).cuda() if tree else None
    cache, ap = pool.cuda(), params("alsc", 128)
    one = paged().cache_attend(q, cache, ap, cu, parents=up)
    for _ in range(3):
        two = paged().cache_attend(q, cache, ap, cu, parents=up)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    graph, out = torch.cuda.CUDAGraph(), (torch.zeros_like(one[0]), torch.zeros_like(one[1]))
    with torch.cuda.graph(graph):
        paged().cache_attend(q, cache, ap, cu, parents=up, out=out)
    graph.replay()
    assert torch.equal(one[0], out[0]) and torch.equal(one[1], out[1])
    other = [10, 0, 20]
    cache.lens.copy_(i32([2500, 333, 20]))
    cu.copy_(i32(sums(other)))
    q.copy_(torch.randn(N, 8, 128, generator=g).to(dtype))
    if tree:
        up[:30] = a_tree(other, g).cuda()
    graph.replay()
    want = Attend(q.cpu(), pool.k, pool.v, pool.table, [2500, 333, 20], sums(other), ap, None if up is None else up.cpu())
    check(out, want, dtype)
    assert torch.equal(out[0][30:], one[0][30:])
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("tree", [False, True], ids=["prompt", "tree"])
def test_on_a_given_stream(tree):
    from test_gpu_kv_cache_streams import late
    pool = Pool([333, 120], 2, 128, 16, BF16, 4)
    g = torch.Generator().manual_seed(2)
    new = [50, 20]
    q, temp = torch.randn(70, 8, 128, generator=g).bfloat16().cuda(), (0.5 + torch.rand(70, generator=g)).cuda()
    up, cu, ap = a_tree(new, g).cuda() if tree else None, i32(sums(new)), params("tanh", 128)
    cache, side = pool.cuda(), torch.cuda.Stream()
    want = paged().cache_attend(q, cache, ap, cu, parents=up, temp=temp)
    pairs = [(torch.zeros_like(x), x) for x in (q, temp, cu) + ((up,) if tree else ())]
    torch.cuda.synchronize()
    late(side, pairs)
    got = paged().cache_attend(pairs[0][0], cache, ap, pairs[2][0], parents=pairs[3][0] if tree else None, temp=pairs[1][0],
                               stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and cache.status(stream=side) == (0, 0)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_offsets_past_32_bits(dtype):
    """Pages more than 2^32 bytes into the cache."""
    n = (5 << 30) // (4 * 64 * 128 * dtype.itemsize)
    pool = Pool([200, 90], 4, 128, 64, dtype, 12)
    far = torch.zeros(n, 4, 64, 128, dtype=dtype, device="cuda"), torch.zeros(n, 4, 64, 128, dtype=dtype, device="cuda")
    used = pool.table[pool.table >= 0].long()
    for x, y in zip(far, (pool.k, pool.v)):
        x[n - 1 - used] = y[used].cuda()
    from soft_capped_attention_gb300 import kv_cache as kv
    table = torch.where(pool.table >= 0, n - 1 - pool.table, -1).to(torch.int32).cuda()
    cache = kv.KVCache(*far, table, i32(pool.lens))
    q = torch.randn(100, 8, 128, generator=pool.gen).to(dtype)
    ap = params("tanh", 128)
    got = paged().cache_attend(q.cuda(), cache, ap, i32([0, 60, 100]))
    check(got, Attend(q, pool.k, pool.v, pool.table, pool.lens, [0, 60, 100], ap), dtype)


BAD = [  # lens, cu_new, parents, table: what is wrong, and its bit
    (dict(lens=[300, 5000]), 32), (dict(lens=[300, -1]), 32), (dict(lens=[300, 29]), 128), (dict(cu=[0, 40, 30]), 128),
    (dict(cu=[0, 40, 71]), 128), (dict(up=(55, 15)), 512), (dict(up=(55, -2)), 512), (dict(up=(55, 2 ** 31 - 1)), 512),
    (dict(table=-1), 64), (dict(table=10 ** 6), 64),
]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("bad,bit", BAD, ids=str)
def test_bad_device_data(dtype, bad, bit):
    """The second sequence's data are wrong: its bit, and the first one's results as ever (to the
    order of their sums: the split follows all lengths)."""
    pool = Pool([300, 90], 2, 128, 16, dtype, 3)
    g = pool.gen
    q = torch.randn(70, 4, 128, generator=g).to(dtype).cuda()
    up = a_tree([40, 30], g)
    ap = params("tanh", 128)
    cache = pool.cuda()
    if "lens" in bad:
        cache.lens.copy_(i32(bad["lens"]))
    if "table" in bad:
        cache.table[1, 2] = bad["table"]
    if "up" in bad:
        up[bad["up"][0]] = bad["up"][1]
    got = paged().cache_attend(q, cache, ap, i32(bad.get("cu", [0, 40, 70])), parents=up.cuda() if "up" in bad else None)
    assert cache.status() == (6, bit)
    first = None if "up" not in bad else up[:40]
    check((got[0][:40], got[1][:40]), Attend(q[:40].cpu(), pool.k, pool.v, pool.table, [300], [0, 40], ap, first), dtype)
    good = pool.cuda()
    again = paged().cache_attend(q, good, ap, i32([0, 40, 70]), parents=a_tree([40, 30], g).cuda() if "up" in bad else None)
    assert torch.isfinite(again[1]).all() and good.status() == (0, 0)


def test_no_rows():
    pool = Pool([30], 2, 64, 16, BF16, 1)
    cache = pool.cuda()
    o, lse = paged().cache_attend(torch.zeros(0, 4, 64, dtype=BF16, device="cuda"), cache, params("tanh", 64), i32([0, 0]))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    o, lse = paged().cache_attend(torch.zeros(5, 4, 64, dtype=BF16, device="cuda"), cache, params("tanh", 64), i32([0, 0]),
                                  out=(torch.ones(5, 4, 64, dtype=BF16, device="cuda"), torch.ones(5, 4, device="cuda")))
    assert (o == 1).all() and (lse == 1).all() and cache.status() == (0, 0)
