"""GPU tests of wrong device data: what it may not touch."""

import pytest
import torch

from kv_cache_utils import Pool
from test_gpu_kv_cache import kv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, 113, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("with_pos", [False, True], ids=["slots", "pos"])
def test_eviction_of_a_bad_length_moves_nothing(bad, with_pos):
    """The table's entries behind a sequence's tokens are leftovers, here the pages of
    another one."""
    pool = Pool([100, 50], 2, 128, 16, torch.bfloat16, 1)
    pool.table[1, 4:] = pool.table[0, :3]
    w = torch.rand(2, 2, pool.max_pages * 16, generator=pool.gen)
    pos = torch.arange(pool.max_pages * 16, dtype=torch.int32).expand(2, 2, -1).contiguous() if with_pos else None
    extra = dict(pos=pos, qpos=torch.tensor([99, 49], dtype=torch.int32)) if with_pos else {}
    good, cache = pool.cuda(weights=w, **extra), pool.cuda(weights=w, **extra)
    good.lens[1] = 0
    cache.lens[1] = bad
    want = kv().cache_evict(good, 30, 2, 5)
    src = kv().cache_evict(cache, 30, 2, 5)
    assert cache.status() == (6, 32) and good.status() == (0, 0)
    for x, y in ((cache.k, good.k), (cache.v, good.v)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(src[0], want[0]) and torch.equal(cache.weights[0], good.weights[0])
    assert cache.lens[0] == 30 and 0 <= int(cache.lens[1]) <= 30
