"""GPU tests of a step's plan and of accepted paths, and of whole steps together."""

import math
import random

import pytest
import torch

from kv_cache_utils import Pool
from paged_ref import Attend, check, plan, walk
from test_gpu_kv_cache import BF16, FP32, kv, params
from test_gpu_paged import a_tree, i32, paged, sums

pytestmark = pytest.mark.gpu


def a_state(B, page, max_pages, seed, spare=40):
    """Sequences of odd lengths, some of which hold more pages than they need."""
    r = random.Random(seed)
    lens = [r.choice([0, 1, page, page + 1, r.randint(0, page * max_pages // 2)]) for _ in range(B)]
    held = [min(max_pages, -(-n // page) + r.choice([0, 0, 1, 3])) for n in lens]
    order = list(range(sum(held) + spare))
    r.shuffle(order)
    table, at = [], 0
    for h in held:
        table.append(order[at:at + h] + [-1] * (max_pages - h))
        at += h
    free = order[at:] + [-1] * (len(order) - spare)
    return lens, held, table, free, spare


def a_cache(table, lens, num_pages, page, qpos=None):
    k = torch.zeros(num_pages, 1, page, 64, dtype=BF16, device="cuda")
    kw = {}
    if qpos is not None:
        kw = dict(pos=torch.zeros(len(lens), 1, len(table[0]) * page, dtype=torch.int32, device="cuda"), qpos=i32(qpos))
    return kv().KVCache(k, k.clone(), i32(table), i32(lens), **kw)


PLANS = [(1, 16, 8, 1), (2, 8, 3, 1), (5, 64, 4, 9), (64, 16, 20, 1), (64, 16, 20, 40), (700, 32, 6, 50), (1100, 16, 4, 3),
         (6000, 8, 4, 2), (3, 16, 700, 5000), (9000, 8, 3, 2)]


@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "out"])
@pytest.mark.parametrize("with_pos", [False, True], ids=["slots", "pos"])
@pytest.mark.parametrize("B,page,max_pages,most", PLANS, ids=str)
def test_plan(B, page, max_pages, most, with_pos, in_place):
    r = random.Random(B + most)
    need = B * (most // page + 2)
    lens, held, table, free, n_free = a_state(B, page, max_pages, B, spare=need)
    n_new = [r.choice([-1, 0, 1, r.randint(0, most)]) for _ in range(B)]
    n_new = [min(n, max_pages * page - x) for n, x in zip(n_new, lens)]
    qpos = [x + 5 * b - 1 for b, x in enumerate(lens)] if with_pos else None
    rows = max(1, sum(max(n, 0) for n in n_new)) + r.randint(0, 5)
    cache = a_cache(table, lens, len(free), page, qpos)
    pool = paged().PagePool(i32(free), i32([n_free]), i32(held))
    out = None if in_place else (i32([9] * B), i32([9] * B) if with_pos else None, i32([9] * B), i32([9]))
    want = plan(table, lens, held, free, n_free, n_new, page, rows, qpos)
    for _ in range(1 if in_place else 2):  # the same inputs give the same again
        cu, slots, positions = paged().cache_plan(cache, pool, i32(n_new), rows, out=out)
        got = (cache.lens, cache.qpos, pool.held, pool.n_free) if in_place else out
        assert cu.tolist() == want["cu"] and slots.tolist() == want["slots"] and positions.tolist() == want["positions"]
        assert got[0].tolist() == want["lens"] and got[2].tolist() == want["held"] and got[3].tolist() == [want["n_free"]]
        assert not with_pos or got[1].tolist() == want["qpos"]
        assert cache.table.tolist() == want["table"]
        assert pool.free.tolist()[:want["n_free"]] == want["free"][:want["n_free"]]
    assert cache.status() == (0, 0)


BAD_PLANS = [dict(n_new=[40, 3, 60]), dict(n_new=[3, 4, 70]), dict(n_new=[2, 400, 0]), dict(held=[1, -1, 2]), dict(held=[1, 99, 2]),
             dict(n_free=-1), dict(n_free=90), dict(lens=[1, -5, 3]), dict(lens=[1, 9999, 3])]


@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "out"])
@pytest.mark.parametrize("bad", BAD_PLANS, ids=str)
def test_a_plan_that_does_not_fit_changes_nothing(bad, in_place):
    d = dict(n_new=[1, 2, 3], lens=[10, 0, 30], held=[1, 0, 2], n_free=4)
    d.update(bad)
    table = [[5, -1, -1, -1, -1], [-1] * 5, [7, 2, -1, -1, -1]]
    free = [0, 1, 3, 4, -1, -1, -1, -1]
    cache = a_cache(table, d["lens"], 8, 16)
    pool = paged().PagePool(i32(free), i32([d["n_free"]]), i32(d["held"]))
    out = None if in_place else (i32([9] * 3), None, i32([9] * 3), i32([9]))
    cu, slots, positions = paged().cache_plan(cache, pool, i32(d["n_new"]), 64, out=out)
    got = (cache.lens, None, pool.held, pool.n_free) if in_place else out
    assert cache.status() == (6, 1024)
    assert cu.tolist() == [0] * 4 and (slots == -1).all() and (positions == -1).all()
    assert got[0].tolist() == d["lens"] and got[2].tolist() == d["held"] and got[3].tolist() == [d["n_free"]]
    assert cache.table.tolist() == table and pool.free.tolist() == free


ACCEPTS = [  # new, Hkv, D, page, dtype, width
    ([1], 1, 64, 16, BF16, 1), ([9, 0, 33], 2, 128, 16, BF16, 6), ([64, 5], 8, 128, 64, BF16, 64), ([40, 7, 1, 20], 3, 64, 8, FP32, 5),
    ([300, 2], 2, 128, 16, FP32, 200), ([1500, 90], 1, 64, 32, BF16, 700), ([25] * 40, 4, 128, 16, BF16, 9),
]


def a_walk(new, up, gen, vocab=3):
    """Few tokens, so that walks go deep and siblings may agree."""
    N = sum(new)
    return (torch.randint(0, vocab, (N,), generator=gen, dtype=torch.int32), torch.randint(0, vocab, (N,), generator=gen, dtype=torch.int32))


@pytest.mark.parametrize("given", [False, True], ids=["verify", "accept"])
@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "out"])
@pytest.mark.parametrize("extras", [False, True], ids=["plain", "weights_and_pos"])
@pytest.mark.parametrize("case", ACCEPTS, ids=lambda c: "-".join(str(x)[:20] for x in c))
def test_accept(case, extras, in_place, given):
    new, Hkv, D, page, dtype, width = case
    lens = [n + 3 + 7 * b for b, n in enumerate(new)]
    pool = Pool(lens, Hkv, D, page, dtype, sum(new))
    g = pool.gen
    up = a_tree(new, g, bushy=0.8)
    tokens, says = a_walk(new, up, g)
    cu, B = sums(new), len(new)
    paths = []
    for b in range(B):
        r = slice(cu[b], cu[b + 1])
        paths.append(walk(up[r].tolist(), tokens[r].tolist(), says[r].tolist(), width))
    kw = {}
    if extras:
        kw = dict(weights=torch.rand(B, Hkv, pool.max_pages * page, generator=g),
                  pos=torch.randint(0, 9999, (B, Hkv, pool.max_pages * page), generator=g, dtype=torch.int32),
                  qpos=torch.tensor([n + 100 for n in lens], dtype=torch.int32))
    cache = pool.cuda(**kw)
    out = None if in_place else (i32([9] * B), i32([9] * B) if extras else None)
    if given:
        path = torch.full((B, width), 10 ** 6, dtype=torch.int32)
        for b, (p, _) in enumerate(paths):
            path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        paged().cache_accept(cache, i32(cu), path.cuda(), i32([len(p) for p, _ in paths]), out=out)
    else:
        path, count, nxt = paged().cache_verify(cache, i32(cu), tokens.cuda(), says.cuda(), up.cuda(), width, out=out)
        assert [p + [-1] * (width - len(p)) for p, _ in paths] == path.tolist()
        assert count.tolist() == [len(p) for p, _ in paths] and nxt.tolist() == [t for _, t in paths]
    lens_out, qpos_out = (cache.lens, cache.qpos) if in_place else out
    assert lens_out.tolist() == [L - n + len(p) for L, n, (p, _) in zip(lens, new, paths)]
    k, v = pool.k.clone(), pool.v.clone()
    for b, (p, _) in enumerate(paths):
        base = lens[b] - new[b]
        for i, x in enumerate(p):
            to, fro = int(pool.table[b, (base + i) // page]), int(pool.table[b, (base + x) // page])
            k[to, :, (base + i) % page], v[to, :, (base + i) % page] = pool.k[fro, :, (base + x) % page], pool.v[fro, :, (base + x) % page]
            if extras:
                assert torch.equal(cache.weights[b, :, base + i].cpu(), kw["weights"][b, :, base + x])
                assert (cache.pos[b, :, base + i] == lens[b] + 100 - new[b] + 1 + i).all()
        if extras:
            assert torch.equal(cache.weights[b, :, :base].cpu(), kw["weights"][b, :, :base])
            assert torch.equal(cache.pos[b, :, :base].cpu(), kw["pos"][b, :, :base])
            assert int(qpos_out[b]) == lens[b] + 100 - new[b] + len(p)
    bits = torch.int16 if dtype == BF16 else torch.int32
    assert torch.equal(cache.k.cpu().view(bits), k.view(bits)) and torch.equal(cache.v.cpu().view(bits), v.view(bits))
    assert cache.status() == (0, 0)


BAD_PATHS = [([[0, 0]], [2], 2048), ([[0, 3]], [2], 2048), ([[1, 0]], [2], 2048), ([[-1, 2]], [2], 2048), ([[0, 1]], [3], 2048),
             ([[0, 1]], [-1], 2048)]


@pytest.mark.parametrize("path,count,bit", BAD_PATHS, ids=str)
def test_a_bad_path_moves_nothing(path, count, bit):
    pool = Pool([20, 30], 2, 64, 16, BF16, 3)
    cache = pool.cuda()
    paged().cache_accept(cache, i32([0, 3, 8]), i32(path + [[0, 4]]), i32(count + [2]))
    assert cache.status() == (6, bit) and cache.lens.tolist() == [20, 27]
    first = pool.table[0, :2].long()
    assert torch.equal(cache.k.cpu()[first].view(torch.int16), pool.k[first].view(torch.int16))


@pytest.mark.parametrize("lens,cu,bit", [([20, 999], [0, 3, 8], 32), ([20, 4], [0, 3, 8], 128), ([20, 30], [0, 3, 2], 128)], ids=str)
def test_accept_of_bad_device_data(lens, cu, bit):
    pool = Pool([20, 30], 2, 64, 16, BF16, 3)
    cache = pool.cuda()
    cache.lens.copy_(i32(lens))
    up, t = i32([-1, 0, 1, -1, 0, 1, 2, 3]), i32([5] * 8)
    path, count, nxt = paged().cache_verify(cache, i32(cu), t, t, up, 4)
    assert cache.status() == (6, bit)
    assert cache.lens.tolist() == [20, lens[1]] and count.tolist() == [3, 0] and path.tolist() == [[0, 1, 2, -1], [-1] * 4]
    assert nxt.tolist() == [5, -1]


def test_verify_without_rows():
    cache = Pool([20, 30], 2, 64, 16, BF16, 3).cuda()
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    path, count, nxt = paged().cache_verify(cache, i32([0, 0, 0]), none, none, none, 3)
    assert (path == -1).all() and count.tolist() == [0, 0] and nxt.tolist() == [-1, -1]
    assert cache.lens.tolist() == [20, 30] and cache.status() == (0, 0)


@pytest.mark.parametrize("shape", [(), (5, 1)], ids=str)
def test_tokens_of_another_shape_are_refused(shape):
    cache = Pool([20], 2, 64, 16, BF16, 3).cuda()
    x = torch.zeros(shape, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="tokens"):
        paged().cache_verify(cache, i32([0, 0]), x, x, x, 3)


@pytest.mark.parametrize("what", ["plan", "longer_plan", "verify", "accept"])
def test_steps_on_a_given_stream(what):
    """What the call reads arrives on that stream, late.  (The longer plan needs slots 112 .. 119,
    which the table has no place for.)"""
    from test_gpu_kv_cache_streams import late
    side = torch.cuda.Stream()

    def a_call(stream, work):
        cache = Pool([100, 50], 2, 64, 16, BF16, 3).cuda()
        pool = paged().PagePool(torch.arange(cache.num_pages, dtype=torch.int32, device="cuda"), i32([3]), i32([7, 4]))
        if "plan" in what:
            given = [i32([12 if what == "plan" else 20, -1])]
        elif what == "verify":
            given = [i32([0, 30, 50])] + [x.cuda() for x in (*a_walk([50], None, torch.Generator().manual_seed(3), vocab=2),
                                                              a_tree([30, 20], torch.Generator().manual_seed(4)))]
        else:
            given = [i32([0, 30, 50]), i32([[0, 4, 9], [3, 19, -1]]), i32([3, 2])]
        late_ones = [torch.zeros_like(x) for x in given]
        torch.cuda.synchronize()
        work(list(zip(late_ones, given)))
        if "plan" in what:
            got = paged().cache_plan(cache, pool, late_ones[0], 40, stream=stream)
        elif what == "verify":
            got = paged().cache_verify(cache, *late_ones, 4, stream=stream)
        else:
            paged().cache_accept(cache, *late_ones, stream=stream)
            got = ()
        if stream is not None:
            stream.synchronize()
        return [*got, cache.k, cache.v, cache.lens, cache.table, pool.held, pool.n_free, pool.free], cache.status(stream=stream)

    def now(pairs):
        for a, b in pairs:
            a.copy_(b)

    want, status = a_call(None, now)
    got, status2 = a_call(side, lambda pairs: late(side, pairs))
    assert status == status2 == ((6, 1024) if what == "longer_plan" else (0, 0))
    assert all(torch.equal(a.nan_to_num(7.0) if a.is_floating_point() else a, b.nan_to_num(7.0) if b.is_floating_point() else b)
               for a, b in zip(got, want))


class Dense:
    """A sequence kept as plain rows, for what a whole run has to give."""

    def __init__(self):
        self.k, self.v = [], []


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("window", [0, 50])
def test_steps_together(dtype, window):
    """Prompts in two chunks, then drafted steps, while sequences end and new ones begin: plan,
    append, attend, verify.  Every row's output against the definition over the rows that the
    sequence has kept."""
    B, Hq, Hkv, D, page, max_pages, pages, width = 4, 4, 2, 128, 16, 24, 60, 5
    g = torch.Generator().manual_seed(5)
    r = random.Random(6)
    k = torch.full((pages, Hkv, page, D), math.nan, dtype=dtype, device="cuda")
    cache = kv().KVCache(k, k.clone(), i32([[-1] * max_pages] * B), i32([0] * B))
    pool = paged().PagePool.full(cache)
    ap = params("tanh15", D, window)
    held = [Dense() for _ in range(B)]
    rows = 256

    def step(n_new, tree):
        cu, slots, positions = paged().cache_plan(cache, pool, i32(n_new), rows)
        new = [max(n, 0) for n in n_new]
        assert cu.tolist() == sums(new)
        N = sum(new)
        q, kn, vn = (torch.randn(rows, h, D, generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
        kv().cache_append(cache, kn.cuda(), vn.cuda(), cu_new=cu)
        assert positions[:N].tolist() == [len(held[b].k) * (n_new[b] >= 0) + i for b in range(B) for i in range(new[b])]
        at = slots[:N].cpu()  # the slot map names the rows that append wrote
        assert torch.equal(cache.k.cpu()[at // page, :, at % page], kn[:N])
        up = torch.full((rows,), -1, dtype=torch.int32)
        up[:N] = a_tree(new, g) if tree else 0
        o, lse = paged().cache_attend(q.cuda(), cache, ap, cu, parents=up.cuda() if tree else None)
        for b in range(B):
            if n_new[b] < 0:
                held[b] = Dense()
            for i in range(sums(new)[b], sums(new)[b + 1]):
                held[b].k.append(kn[i])
                held[b].v.append(vn[i])
        lens = [len(x.k) for x in held]
        most = -(-max(lens) // page)
        table = torch.arange(B * most, dtype=torch.int32).reshape(B, most)
        kd, vd = torch.zeros(B * most, Hkv, page, D, dtype=dtype), torch.zeros(B * most, Hkv, page, D, dtype=dtype)
        for b in range(B):
            for x, rows_ in ((kd, held[b].k), (vd, held[b].v)):
                for j, row in enumerate(rows_):
                    x[b * most + j // page, :, j % page] = row
        check((o, lse), Attend(q, kd, vd, table, lens, sums(new) , ap, up if tree else None), dtype)
        if tree:
            tokens, says = a_walk([rows], None, g, vocab=2)
            path, count, _ = paged().cache_verify(cache, cu, tokens.cuda(), says.cuda(), up.cuda(), width)
            for b in range(B):
                a, e = sums(new)[b], sums(new)[b + 1]
                p, _ = walk(up[a:e].tolist(), tokens[a:e].tolist(), says[a:e].tolist(), width)
                assert path[b, :int(count[b])].tolist() == p
                for x in (held[b].k, held[b].v):
                    first = len(x) - new[b]
                    x[first:] = [x[first + i] for i in p]
        assert cache.lens.tolist() == [len(x.k) for x in held]
        assert int(pool.n_free) + sum(pool.held.tolist()) == pages
        owned = [int(x) for b in range(B) for x in cache.table[b, :int(pool.held[b])]] + pool.free[:int(pool.n_free)].tolist()
        assert sorted(owned) == list(range(pages))

    step([70, 1, 0, 33], False)
    step([50, 90, 7, 1], False)
    for i in range(6):
        step([r.randint(1, 20) for _ in range(B)], True)
        if i == 2:
            step([-1, 1, -1, 1], False)
            step([40, 1, 17, 0], False)
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_a_captured_step(dtype):
    """Plan, append, attend, verify in one graph: replays give what the same calls give one by one."""
    B, Hq, Hkv, D, page, max_pages, pages, rows, width = 3, 4, 2, 64, 16, 12, 40, 64, 4
    g = torch.Generator().manual_seed(8)

    def state():
        k = torch.zeros(pages, Hkv, page, D, dtype=dtype, device="cuda")
        cache = kv().KVCache(k, k.clone(), i32([[-1] * max_pages] * B), i32([0] * B), weights=torch.ones(B, Hkv, max_pages * page, device="cuda"))
        return cache, paged().PagePool.full(cache)

    ap = params("alsc", D)
    inputs = [[torch.randn(rows, h, D, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv)] +
              [torch.randint(0, 2, (rows,), generator=g, dtype=torch.int32).cuda() for _ in range(2)] for _ in range(5)]
    news = [[20, 1, 30], [9, 20, 30], [-1, 0, 7], [33, 5, 1], [1, 1, 1]]
    trees = [a_tree([max(n, 0) for n in new], g) for new in news]
    trees = [torch.cat([t, torch.full((rows - len(t),), -1, dtype=torch.int32)]).cuda() for t in trees]

    def step(cache, pool, q, k, v, tokens, says, n_new, up):
        cu, _, _ = paged().cache_plan(cache, pool, n_new, rows)
        kv().cache_append(cache, k, v, cu_new=cu)
        o, lse = paged().cache_attend(q, cache, ap, cu, parents=up, out=(out_o, out_lse))
        return paged().cache_verify(cache, cu, tokens, says, up, width)

    out_o, out_lse = torch.zeros(rows, Hq, D, dtype=dtype, device="cuda"), torch.zeros(rows, Hq, device="cuda")
    held = [x.clone() for x in inputs[0]] + [i32(news[0]), trees[0].clone()]
    one, two = state(), state()
    warm = state()  # (its workspace is not the others': make theirs before the capture)
    for x in (two, warm):
        step(*x, *held)
    for a, b in zip((two[0].k, two[0].v, two[0].table, two[0].lens, two[0].weights, two[1].free, two[1].n_free, two[1].held),
                    (one[0].k, one[0].v, one[0].table, one[0].lens, one[0].weights, one[1].free, one[1].n_free, one[1].held)):
        a.copy_(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*two, *held)
    for x, new, up in zip(inputs, news, trees):
        out_o.zero_()
        out_lse.zero_()
        want = step(*one, *x, i32(new), up)
        kept = [out_o.clone(), out_lse.clone()]
        out_o.zero_()
        out_lse.zero_()
        for a, b in zip(held, x + [i32(new), up]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out_o, kept[0]) and torch.equal(out_lse, kept[1])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(one[0].k, two[0].k) and torch.equal(one[0].lens, two[0].lens) and torch.equal(one[1].held, two[1].held)
    assert one[0].status() == (0, 0) and two[0].status() == (0, 0)
