"""The joins of a split decode on given partial results: the kernels' own code, built
around tests/join_check.cu, against the formula in 64 bits."""

import ctypes
import math
import os
import subprocess

import pytest
import torch

from kv_cache_utils import EPS32
from soft_capped_attention_gb300 import capattn as ca

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
SLOTS, HEADS = 2 * 608, 16  # partial results a workspace holds


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from soft_capped_attention_gb300 import build
    so = str(tmp_path_factory.mktemp("join") / "join_check.so")
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-shared", os.path.join(HERE, "join_check.cu"), "-o", so],
                   check=True)
    h = ctypes.CDLL(so)
    h.join_check.argtypes = [ctypes.c_int] * 4 + [ctypes.c_void_p] * 7 + [ctypes.c_int, ctypes.c_void_p]
    return h


class Parts:
    """Partial results of `groups` groups: heavy and light pieces, empty ones and heads without any."""

    def __init__(self, D, groups, pieces, heads, seed):
        g = torch.Generator().manual_seed(seed)
        self.shape = D, groups, pieces, heads
        m = 4 * torch.randn(SLOTS, HEADS, generator=g)
        l = torch.rand(SLOTS, HEADS, generator=g) * 50 + 1
        o = l[..., None] * torch.randn(SLOTS, HEADS, D, generator=g)
        empty = torch.rand(SLOTS, HEADS, generator=g) < 0.1
        empty[:, 0] = False
        if heads > 1:
            empty[:, 1] = True
        m[empty], l[empty], o[empty] = -math.inf, 0.0, 0.0
        self.m, self.l, self.o = m, l, o
        self.ml = torch.stack([m, l], -1).contiguous().cuda()
        self.parts = o.cuda()
        self.part_ml, self.part_o = torch.zeros_like(self.ml), torch.zeros_like(self.parts)
        self.counters = torch.zeros(608, dtype=torch.int32, device="cuda")

    def run(self, lib, form):
        D, groups, pieces, heads = self.shape
        if form:
            self.part_ml.copy_(self.ml)
            self.part_o.copy_(self.parts)
        else:
            self.part_ml.fill_(1e30)
            self.part_o.fill_(1e30)
        o = torch.full((groups, heads, D), math.nan, device="cuda")
        lse = torch.full((groups, heads), math.nan, device="cuda")
        ptrs = [x.data_ptr() for x in (self.ml, self.parts, self.part_ml, self.part_o, self.counters, o, lse)]
        assert lib.join_check(D, groups, pieces, heads, *ptrs, form, torch.cuda.current_stream().cuda_stream) == 0
        return o, lse

    def want(self):
        """o and lse of every group in 64 bits, and the sum of |terms| that o's roundings are relative to."""
        D, groups, pieces, heads = self.shape
        o, lse = torch.zeros(groups, heads, D, dtype=torch.float64), torch.zeros(groups, heads, dtype=torch.float64)
        size = torch.zeros_like(o)
        for g in range(groups):
            slots = [2 * c + ((g & 1) if c == g * pieces else 0) for c in range(g * pieces, (g + 1) * pieces)]
            m, l, part = (x[slots, :heads].double() for x in (self.m, self.l, self.o))
            top = m.amax(0)
            w = torch.exp(m - torch.where(torch.isinf(top), 0.0, top))
            total = (l * w).sum(0)
            some = total > 0
            o[g] = torch.where(some[:, None], (part * w[..., None]).sum(0) / total.clamp(min=1e-300)[:, None], 0.0)
            size[g] = torch.where(some[:, None], (part.abs() * w[..., None]).sum(0) / total.clamp(min=1e-300)[:, None], 0.0)
            lse[g] = torch.where(some, top + torch.log(total.clamp(min=1e-300)), -math.inf)
        return o, lse, size


SHAPES = [(128, 3, 1, 5), (128, 5, 2, 16), (64, 4, 3, 4), (128, 2, 4, 8), (128, 9, 5, 4), (64, 7, 7, 16), (128, 6, 16, 3),
          (128, 5, 17, 8), (64, 3, 33, 5), (128, 8, 38, 4), (128, 15, 40, 16), (128, 2, 304, 4)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("form", [0, 1, 4], ids=["left", "one_warp", "four_warps"])
def test_a_join_adds_its_pieces(lib, shape, form):
    """Every term is scaled by at most two exponentials and as many products for each
    piece of its chain (exp's argument below 40, so 2^-24 * 40 of it, and 2 steps of
    its own), and added once."""
    p = Parts(*shape, seed=sum(shape))
    o, lse = p.run(lib, form)
    o64, lse64, size = p.want()
    err = (3 * 45 + 4 * shape[2] + 8) * EPS32
    assert torch.equal(torch.isneginf(lse.cpu()), torch.isneginf(lse64))
    assert ((o.cpu().double() - o64).abs() <= 2 * err * size).all()
    live = ~torch.isneginf(lse64)
    assert ((lse.cpu().double() - lse64).abs()[live] <= err + 4 * EPS32 * lse64.abs()[live]).all()
    assert not p.counters.any()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_pieces_left_by_other_ctas_are_all_read(lib, shape):
    """What a warp a piece leaves, counts in and joins is what a warp joins afterwards."""
    p = Parts(*shape, seed=sum(shape) + 1)
    want = p.run(lib, 1)
    for _ in range(30):
        got = p.run(lib, 0)
        assert torch.equal(got[0].view(torch.int32), want[0].view(torch.int32))
        assert torch.equal(got[1], want[1])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_join_has_the_same_bits_whoever_makes_it(lib, shape):
    """One warp (a group's last CTA, which has more to do) or four (the others)."""
    for seed in range(5):
        p = Parts(*shape, seed=1000 * seed + sum(shape))
        one, four = p.run(lib, 1), p.run(lib, 4)
        assert torch.equal(one[0].view(torch.int32), four[0].view(torch.int32))
        assert torch.equal(one[1], four[1])


@pytest.mark.parametrize("lens, Hq, Hkv, D, page, window", [
    ([2050 + 409 * i for i in range(16)], 32, 8, 128, 64, 0),
    ([130_977], 32, 8, 128, 64, 0),
    ([9000, 300, 20_000], 5, 1, 64, 32, 6000),
], ids=["batch", "long", "window"])
def test_split_decodes_repeat_their_bits_while_other_work_runs(lens, Hq, Hkv, D, page, window):
    """Another stream's kernels hold some of the SMs for some of the time, so that now one
    CTA comes last to a group and now another."""
    from soft_capped_attention_gb300 import kv_cache as kv
    g = torch.Generator(device="cuda").manual_seed(Hq)
    used = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32)
    order, at = torch.randperm(sum(used)).to(torch.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    k, v = (torch.randn(sum(used), Hkv, page, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    start = torch.rand(len(lens), Hkv, max(used) * page, generator=g, device="cuda")
    cache = kv.KVCache(k, v, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), weights=start.clone())
    q = torch.randn(len(lens), Hq, D, generator=g, device="cuda").bfloat16()
    ap = ca.AttnParams(sm_scale=1 / math.sqrt(D), cap_method="soft_sign", cap=20.0, causal=True, window_len=window)
    want = [x.clone() for x in kv.cache_decode(q, cache, ap, accumulate=True)] + [cache.weights.clone()]
    side, x = torch.cuda.Stream(), torch.randn(700, 700, device="cuda")
    torch.cuda.synchronize()
    for i in range(60):
        with torch.cuda.stream(side):
            for _ in range(i % 7):
                torch.mm(x, x)
        cache.weights.copy_(start)
        o, lse = kv.cache_decode(q, cache, ap, accumulate=True)
        assert torch.equal(o.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])
        assert torch.equal(cache.weights, want[2])
    assert cache.status() == (0, 0)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_pieces_with_nan_and_infinity_join_alike(lib, shape):
    """A piece of NaN scores only has no maximum but a NaN sum; one with an infinite score
    an infinite maximum and NaN; an output may be a negative zero."""
    D, groups, pieces, heads = shape
    p = Parts(*shape, seed=7 + sum(shape))
    g = torch.Generator().manual_seed(3)
    kind = torch.rand(SLOTS, HEADS, generator=g)
    m, l, o = p.m.clone(), p.l.clone(), p.o.clone()
    no_max, top, zero = kind < 0.02, (kind >= 0.02) & (kind < 0.04), (kind >= 0.04) & (kind < 0.3)
    m[no_max], l[no_max], o[no_max] = -math.inf, math.nan, math.nan
    m[top], l[top], o[top] = math.inf, math.nan, math.nan
    o[zero] = -0.0
    p.ml.copy_(torch.stack([m, l], -1))
    p.parts.copy_(o)
    one, left, four = p.run(lib, 1), p.run(lib, 0), p.run(lib, 4)
    for x, y, z in zip(one, left, four):
        assert torch.equal(x.view(torch.int32), z.view(torch.int32)) and torch.equal(y.view(torch.int32), z.view(torch.int32))
    for i in range(groups):
        slots = [2 * c + ((i & 1) if c == i * pieces else 0) for c in range(i * pieces, (i + 1) * pieces)]
        bad = (no_max | top)[slots, :heads].any(0)
        assert torch.equal(torch.isnan(four[1][i]).cpu(), bad) and torch.equal(torch.isnan(four[0][i]).all(-1).cpu(), bad)
