"""GPU tests of long decodes and large batches against 64 bits, within the error that the
kernels' own depth of sums allows (not the length's)."""

import math
import random

import pytest
import torch

from kv_cache_ref import Want, check
from split_model import pieces
from test_gpu_kv_cache import kv, params

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


def cache_of(lens, Hkv, D, page, dtype, seed):
    """A cache on the GPU: shuffled pages, -1 in unused entries of the table."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    used = [-(-n // page) for n in lens]
    width = max(1, max(used))
    order = torch.randperm(sum(used), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    start = torch.tensor([0, *used]).cumsum(0)[:-1]
    col = torch.arange(width)
    inside = col < torch.tensor(used)[:, None]
    table = torch.where(inside, order[(start[:, None] + col).clamp(max=len(order) - 1)], torch.tensor(-1, dtype=torch.int32))
    k, v = (torch.randn(sum(used), Hkv, page, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    w = torch.rand(len(lens), Hkv, width * page, generator=g, device="cuda")
    return kv().KVCache(k, v, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), weights=w), g


def lengths(B, short, long, every, seed):
    """B lengths up to `short`, and one of about `long` every so many sequences."""
    r = random.Random(seed)
    return [r.randint(long // 2, long) if b % every == every // 2 else r.randint(0, short) for b in range(B)]


CASES = [
    # lens, Hq, Hkv, D, page, dtype, cap, window
    ([20_000], 4, 1, 128, 64, BF16, "alsc30", 0),
    ([130_977], 32, 8, 128, 64, BF16, "tanh50", 0),
    ([30_000, 1, 9_000], 12, 1, 64, 16, BF16, "soft_sign", 0),
    ([50_000, 777], 4, 2, 128, 32, BF16, "tanh50", 8_000),
    ([40_000], 1, 1, 64, 16, FP32, "tanh50", 0),
    ([20_000, 3], 16, 1, 128, 64, FP32, "none", 0),
    # more than 64 sequences, split: sums and searches over groups of 32 of them
    (lengths(300, 70, 2500, 50, 1), 4, 2, 128, 16, BF16, "tanh50", 0),
    (lengths(300, 70, 2500, 299, 2), 8, 1, 64, 16, BF16, "none", 0),
    (lengths(700, 40, 1200, 100, 3), 3, 1, 64, 16, FP32, "tanh50", 0),
    # and more than 8192: over runs of such groups
    (lengths(9_000, 20, 1800, 1000, 4), 2, 1, 64, 16, BF16, "alsc30", 0),
    (lengths(17_000, 9, 900, 3000, 5), 1, 1, 64, 16, FP32, "none", 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1]}-{c[2]}-{c[3]}-{c[5]}-{c[6]}-{c[7]}")
@pytest.mark.parametrize("acc", [False, True], ids=["plain", "weights"])
def test_long_and_many(case, acc):
    lens, Hq, Hkv, D, page, dtype, cap, window = case
    cache, g = cache_of(lens, Hkv, D, page, dtype, len(lens) + Hq)
    assert not all(p[5] for p in pieces(lens, Hq, Hkv, D, dtype.itemsize, cache.max_len, window))  # some are split
    q = torch.randn(len(lens), Hq, D, generator=g, device="cuda").to(dtype)
    temp = 0.5 + torch.rand(len(lens), generator=g, device="cuda")
    ap = params(cap, D, window)
    before = cache.weights.clone()
    got = kv().cache_decode(q, cache, ap, temp=temp, accumulate=acc)
    assert cache.status() == (0, 0)
    want = Want(q, cache, lens, ap, temp)
    check(got, want, q, cache, lens, window, (before, cache.weights) if acc else None)
    if not acc:
        assert torch.equal(before, cache.weights)
    again = kv().cache_decode(q, cache, ap, temp=temp)
    assert all(torch.equal(x, y) for x, y in zip(again, got))
