"""GPU tests of plans for sequences that do not own the pages of all their tokens (a prefix that
several share): refused, so that no page of theirs is replaced or given away."""

import pytest

from paged_ref import plan
from test_gpu_paged import i32, paged
from test_gpu_paged_steps import a_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("held", [0, 1, 4])
@pytest.mark.parametrize("n_new", [0, 5, 30, -1])
@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "out"])
def test_a_shared_prefix_is_refused(held, n_new, in_place):
    """Two sequences of 70 tokens over the same four pages and one of their own each; the second
    counts none, its own one or the shared ones alone."""
    table = [[5, 1, 7, 2, 3, -1, -1], [5, 1, 7, 2, 0, -1, -1]]
    free = [4, 6, 8, 9, 10, 11] + [-1] * 6
    lens = [70, 70]
    cache = a_cache(table, lens, len(free), 16)
    pool = paged().PagePool(i32(free), i32([6]), i32([5, held]))
    out = None if in_place else (i32([9] * 2), None, i32([9] * 2), i32([9]))
    cu, slots, positions = paged().cache_plan(cache, pool, i32([3, n_new]), 64, out=out)
    got = (cache.lens, None, pool.held, pool.n_free) if in_place else out
    assert cache.status() == (6, 1024)
    assert cu.tolist() == [0] * 3 and (slots == -1).all() and (positions == -1).all()
    assert got[0].tolist() == lens and got[2].tolist() == [5, held] and got[3].tolist() == [6]
    assert cache.table.tolist() == table and pool.free.tolist() == free


@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 32])
def test_pages_that_just_reach_are_enough(length):
    held = -(-length // 16)
    table = [[5, 1, -1, -1]]
    free = [4, 6, 8, 0] + [-1] * 5
    cache = a_cache(table, [length], len(free), 16)
    pool = paged().PagePool(i32(free), i32([4]), i32([held]))
    want = plan(table, [length], [held], free, 4, [20], 16, 32)
    cu, slots, _ = paged().cache_plan(cache, pool, i32([20]), 32)
    assert cache.status() == (0, 0) and cu.tolist() == want["cu"] and slots.tolist() == want["slots"]
    assert cache.lens.tolist() == want["lens"] and pool.held.tolist() == want["held"] and cache.table.tolist() == want["table"]
