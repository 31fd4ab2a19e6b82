"""GPU tests of decodes whose split leaves pieces without tiles, against 64 bits."""

import pytest
import torch

from kv_cache_utils import Pool, decode64
from split_cases import FP32_CASES
from test_gpu_kv_cache import check_decode, kv, params

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", ["none", "alsc"])
@pytest.mark.parametrize("case", FP32_CASES, ids=lambda c: str(c)[:40])
def test_fp32_decode_of_pieces_without_tiles(case, cap):
    lens, Hq, Hkv, D, page = case
    pool = Pool(lens, Hkv, D, page, torch.float32, sum(lens))
    q = torch.randn(len(lens), Hq, D, generator=pool.gen)
    ap = params(cap, D)
    o64, lse64, add64, et = decode64(q, pool.k, pool.v, pool.table, lens, ap)
    cache, qd = pool.cuda(), q.cuda()
    got = kv().cache_decode(qd, cache, ap)
    vmax = float(torch.nan_to_num(pool.v).abs().max())
    check_decode(got, (o64, lse64, add64), et, vmax, torch.float32, max(lens))
    for _ in range(20):
        again = kv().cache_decode(qd, cache, ap)
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert cache.status() == (0, 0)
