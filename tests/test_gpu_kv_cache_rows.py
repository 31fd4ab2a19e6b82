"""GPU tests of cu_new, the rows of an append: what it may say and what is flagged."""

import pytest
import torch

from kv_cache_utils import Pool
from test_gpu_kv_cache import kv

pytestmark = pytest.mark.gpu


def append(lens, cu, rows):
    pool = Pool(lens, 1, 64, 16, torch.bfloat16, 2)
    new = torch.ones(rows, 1, 64, dtype=torch.bfloat16, device="cuda")
    cache = pool.cuda()
    kv().cache_append(cache, new, new, cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    return pool, cache


@pytest.mark.parametrize("lens, cu, rows", [
    ([10, 20], [0, 8, 5], 8),          # decreases, within every length
    ([10, 20], [0, 8, 5], 40),
    ([10, 20], [3, 0, 5], 8),
    ([10, 20], [0, 4, 9], 8),          # more rows than there are
    ([10, 20], [0, 9, 9], 8),
    ([10, 20], [-1, 4, 8], 8),         # before the first row
    ([5] * 900, [2 * min(b, 700) for b in range(900)] + [1399], 1400),  # the last of many
], ids=lambda x: str(x)[:30])
def test_bad_rows_are_flagged(lens, cu, rows):
    _, cache = append(lens, cu, rows)
    assert cache.status() == (6, 128)
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("lens, cu, rows", [
    ([10, 20], [0, 8, 8], 8), ([10, 20], [0, 0, 0], 3), ([10, 20], [0, 4, 7], 8), ([10, 20], [2, 4, 7], 7),
    ([5] * 900, list(range(901)), 900),
], ids=lambda x: str(x)[:30])
def test_good_rows_are_not(lens, cu, rows):
    pool, cache = append(lens, cu, rows)
    assert cache.status() == (0, 0)
    for b, n in enumerate(lens):
        for slot in range(n - (cu[b + 1] - cu[b]), n):
            pool.k[int(pool.table[b, slot // 16]), :, slot % 16] = 1
    assert torch.equal(cache.k.cpu().view(torch.int16), pool.k.view(torch.int16))
