"""GPU tests of accepted paths whose rows lie on, or go to, pages that the table names wrongly."""

import pytest
import torch

from kv_cache_utils import Pool
from test_gpu_kv_cache import BF16, FP32
from test_gpu_paged import i32, paged

pytestmark = pytest.mark.gpu

NEW = 40  # drafts of a sequence, slots 20 .. 59 in pages of 16


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("bad", [-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("given", [False, True], ids=["verify", "accept"])
@pytest.mark.parametrize("entry", [1, 2, 3])
def test_a_bad_page_moves_nothing(entry, given, bad, dtype):
    """Rows 0, 5, 14, 30, 39 of the second sequence: from entries 1, 1, 2, 3, 3 to entry 1.  Keys,
    values, weights, positions and lengths stay; the first sequence's path is taken."""
    path = [0, 5, 14, 30, 39]
    pool = Pool([60, 60], 2, 64, 16, dtype, 3)
    n = pool.max_pages * 16
    kw = dict(weights=torch.rand(2, 2, n, generator=pool.gen), pos=torch.randint(0, 999, (2, 2, n), generator=pool.gen, dtype=torch.int32),
              qpos=torch.tensor([80, 90], dtype=torch.int32))
    cache = pool.cuda(**kw)
    cache.table[1, entry] = bad
    cu = i32([0, NEW, 2 * NEW])
    if given:
        paged().cache_accept(cache, cu, i32([path, path]), i32([5, 5]))
    else:
        up, tokens, says = [-1] * NEW, [1] * NEW, [2] * NEW
        for a, b in zip(path, path[1:]):
            up[b], tokens[b], says[a] = a, 7, 7
        got, count, nxt = paged().cache_verify(cache, cu, i32(tokens * 2), i32(says * 2), i32(up * 2), 6)
        assert got.tolist() == [path + [-1], [-1] * 6] and count.tolist() == [5, 0] and nxt.tolist() == [2, -1]
    assert cache.status() == (6, 64)
    assert cache.lens.tolist() == [25, 60] and cache.qpos.tolist() == [45, 90]
    second = pool.table[1, :4].long()
    bits = torch.int16 if dtype == BF16 else torch.int32
    for x, y in ((cache.k, pool.k), (cache.v, pool.v)):
        assert torch.equal(x.cpu()[second].view(bits), y[second].view(bits))
    assert torch.equal(cache.weights[1].cpu(), kw["weights"][1]) and torch.equal(cache.pos[1].cpu(), kw["pos"][1])
    first = pool.table[0].long()
    for i, x in enumerate(path):
        to, fro = divmod(20 + i, 16), divmod(20 + x, 16)
        assert torch.equal(cache.k[int(first[to[0]]), :, to[1]].cpu(), pool.k[int(first[fro[0]]), :, fro[1]])


def test_pages_of_rows_that_stay_or_go_are_not_looked_at():
    """Entries that name no page, of drafts that the path leaves out or that are where they go."""
    pool = Pool([60], 2, 64, 16, BF16, 3)
    for path, entry in (([0, 5, 7], 3), ([0, 1, 2, 3], 1)):
        cache = pool.cuda()
        cache.table[0, entry] = -1
        paged().cache_accept(cache, i32([0, NEW]), i32([path]), i32([len(path)]))
        assert cache.status() == (0, 0) and cache.lens.tolist() == [20 + len(path)]


@pytest.mark.parametrize("entry", [0, 30, 60, 90])
def test_a_bad_page_far_along_a_long_path(entry):
    """More rows than a CTA stages: 1500 drafts, every row but the first moves by one."""
    pool = Pool([1502], 1, 64, 16, BF16, 3)
    cache = pool.cuda()
    cache.table[0, entry] = -1
    path = [[i + 1 for i in range(1500)]]
    paged().cache_accept(cache, i32([0, 1502]), i32(path), i32([1500]))
    assert cache.status() == (6, 64) and cache.lens.tolist() == [1502]
    pages = pool.table[0].long()
    assert torch.equal(cache.k.cpu()[pages].view(torch.int16), pool.k[pages].view(torch.int16))
    good = pool.cuda()
    paged().cache_accept(good, i32([0, 1502]), i32(path), i32([1500]))
    assert good.status() == (0, 0) and good.lens.tolist() == [1500]
    rows = pool.k[pages].transpose(0, 1).reshape(1, -1, 64)
    assert torch.equal(good.k.cpu()[pages].transpose(0, 1).reshape(1, -1, 64)[:, :1500], rows[:, 1:1501])
