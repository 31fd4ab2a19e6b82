"""GPU tests of the cache's calls on a given stream: their inputs arrive there, late."""

import math

import pytest
import torch

from kv_cache_utils import Pool
from soft_capped_attention_gb300 import capattn as ca
from test_gpu_kv_cache import kv, params

pytestmark = pytest.mark.gpu

LENS, HKV, HQ, D = [333, 120], 2, 8, 128


def late(side, pairs):
    """On `side`: some milliseconds of nothing, then every buffer gets its value.  What
    was launched on another stream reads what the buffers held before."""
    with torch.cuda.stream(side):
        torch.cuda._sleep(30_000_000)
        for buffer, value in pairs:
            buffer.copy_(value)


def bits(x):
    return x.view(torch.int16 if x.dtype is torch.bfloat16 else torch.int32)


def same(got, want):
    assert all(torch.equal(bits(x), bits(y)) for x, y in zip(got, want))


def cache_of(pool):
    w = torch.rand(2, HKV, pool.max_pages * 16, generator=torch.Generator().manual_seed(1))
    return pool.cuda(weights=w)


def test_decode_on_a_given_stream():
    pool, ap = Pool(LENS, HKV, D, 16, torch.bfloat16, 4), params("tanh", D)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(2, HQ, D, generator=g).bfloat16().cuda()
    temp = (0.5 + torch.rand(2, generator=g)).cuda()
    ref, cache, side = cache_of(pool), cache_of(pool), torch.cuda.Stream()
    want = [*kv().cache_decode(q, ref, ap, temp=temp, accumulate=True), ref.weights]
    kv().cache_decode(q, cache, ap, temp=temp, accumulate=True)  # the workspace is there
    start = cache_of(pool).weights
    qs, ts = torch.zeros_like(q), torch.zeros_like(temp)
    cache.weights.fill_(7.0)
    torch.cuda.synchronize()
    late(side, [(qs, q), (ts, temp), (cache.weights, start)])
    o, lse = kv().cache_decode(qs, cache, ap, temp=ts, accumulate=True, stream=side)
    side.synchronize()
    same([o, lse, cache.weights], want)
    outs = torch.zeros_like(o), torch.zeros_like(lse)
    qs.zero_()
    torch.cuda.synchronize()
    late(side, [(qs, q)])
    kv().cache_decode(qs, cache, ap, temp=ts, out=outs, stream=side)
    side.synchronize()
    same(outs, want)
    assert cache.status(stream=side) == (0, 0)


@pytest.mark.parametrize("packed", [False, True], ids=["step", "packed"])
def test_append_on_a_given_stream(packed):
    pool = Pool(LENS, HKV, D, 16, torch.bfloat16, 5)
    g = torch.Generator().manual_seed(3)
    n = [40, 7] if packed else [1, 1]
    new = [torch.randn(sum(n), HKV, D, generator=g).bfloat16().cuda() for _ in range(2)]
    cu = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda") if packed else None
    ref, cache, side = cache_of(pool), cache_of(pool), torch.cuda.Stream()
    kv().cache_append(ref, *new, cu_new=cu)
    buffers = [torch.zeros_like(x) for x in new]
    held = None if cu is None else torch.zeros_like(cu)
    torch.cuda.synchronize()
    late(side, list(zip(buffers, new)) + ([] if cu is None else [(held, cu)]))
    kv().cache_append(cache, *buffers, cu_new=held, stream=side)
    side.synchronize()
    same([cache.k, cache.v, cache.weights], [ref.k, ref.v, ref.weights])
    assert cache.status(stream=side) == (0, 0)


@pytest.mark.parametrize("form", ["in_place", "out", "no_src"])
def test_evict_on_a_given_stream(form):
    pool = Pool(LENS, HKV, D, 16, torch.bfloat16, 6)
    ref, cache, side = cache_of(pool), cache_of(pool), torch.cuda.Stream()
    w = ref.weights.clone()
    want_src = kv().cache_evict(ref, 50, 3, 9)
    out = (torch.zeros_like(cache.lens), torch.zeros_like(w), None) if form == "out" else None
    cache.weights.zero_()
    torch.cuda.synchronize()
    late(side, [(cache.weights, w)])
    src = kv().cache_evict(cache, 50, 3, 9, out=out, want_src=form != "no_src", stream=side)
    side.synchronize()
    lens, weights, _ = out if out else (cache.lens, cache.weights, None)
    assert (src is None) == (form == "no_src")
    same([cache.k, cache.v, weights[..., :50], lens] + ([] if src is None else [src]),
         [ref.k, ref.v, ref.weights[..., :50], ref.lens] + ([] if src is None else [want_src]))
    assert cache.status(stream=side) == (0, 0)


@pytest.mark.parametrize("own_workspace", [False, True])
def test_key_weights_on_a_given_stream(own_workspace):
    g = torch.Generator().manual_seed(4)
    q, k = (torch.randn(2, 300, h, D, generator=g).bfloat16().cuda() for h in (HQ, HKV))
    temp = (0.5 + torch.rand(2, 300, generator=g)).cuda()
    seg = torch.zeros(2, 300, dtype=torch.int32, device="cuda")
    seg[:, 200:] = 1
    rows = torch.tensor([[0, 300], [20, 250]], dtype=torch.int32, device="cuda")
    ap = ca.AttnParams(sm_scale=1 / math.sqrt(D), cap_method="tanh", cap=20.0, causal=True)
    _, lse, _, _ = ca.capattn_fwd(q, k, k.clone(), ap, temp, seg)
    want = kv().key_weights(q, k, lse, ap, temp, seg, rows=rows)
    side = torch.cuda.Stream()
    held = [torch.zeros_like(x) for x in (q, k, lse, temp, seg, rows)]
    out = torch.zeros_like(want) if own_workspace else None
    ws = kv().new_key_weights_workspace(q, k, ap) if own_workspace else None
    torch.cuda.synchronize()
    late(side, list(zip(held, (q, k, lse, temp, seg, rows))))
    got = kv().key_weights(*held[:3], ap, held[3], held[4], rows=held[5], out=out, workspace=ws, stream=side)
    side.synchronize()
    same([got], [want])
