"""GPU tests of attention over the paged cache where every CTA gets many pieces of query tiles:
of one, two, three and mixed steps, whole and shared, with every cap and without."""

import pytest
import torch

from kv_cache_utils import Pool
from paged_cases import MANY_PIECES
from paged_ref import check
from test_gpu_kv_cache import BF16, FP32, params
from test_gpu_paged import a_tree, i32, paged, run, sums

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap,D", [("none", 64), ("none", 128), ("tanh", 128), ("alsc30", 64), ("soft_sign", 128)])
@pytest.mark.parametrize("name", MANY_PIECES)
def test_many_pieces(name, D, cap):
    lens, new, Hq, Hkv, page, window, tree, _ = MANY_PIECES[name]
    pool = Pool(lens, Hkv, D, page, BF16, D + len(cap))
    got, want = run(pool, new, Hq, params(cap, D, window), BF16, tree, cap == "soft_sign", seed=7, first=1, tail=2)
    check(got, want, BF16)


@pytest.mark.parametrize("name", MANY_PIECES)
def test_many_pieces_fp32(name):
    lens, new, Hq, Hkv, page, window, tree, _ = MANY_PIECES[name]
    pool = Pool(lens, Hkv, 64, page, FP32, 5)
    got, want = run(pool, new, Hq, params("none", 64, window), FP32, tree, True, seed=7, first=1, tail=2)
    check(got, want, FP32)


@pytest.mark.parametrize("cap", ["none", "tanh", "alsc30", "soft_sign"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", MANY_PIECES)
def test_many_pieces_again_and_again(name, D, cap):
    """The same bits however the warps of a CTA fall out."""
    lens, new, Hq, Hkv, page, window, tree, _ = MANY_PIECES[name]
    pool = Pool(lens, Hkv, D, page, BF16, 3)
    q = torch.randn(sum(new), Hq, D, generator=pool.gen).bfloat16().cuda()
    up = a_tree(new, torch.Generator().manual_seed(2)).cuda() if tree else None
    cache, cu, ap = pool.cuda(), i32(sums(new)), params(cap, D, window)
    one = paged().cache_attend(q, cache, ap, cu, parents=up)
    assert torch.isfinite(one[0].float()).all() and torch.isfinite(one[1]).all()
    for _ in range(30):
        two = paged().cache_attend(q, cache, ap, cu, parents=up)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert cache.status() == (0, 0)
