"""GPU tests of key_weights beyond its formula: refusals and what stays out of its sums."""

import math

import pytest
import torch

from kv_cache_utils import EPS32
from test_gpu_kv_cache import kv, params
from soft_capped_attention_gb300 import capattn as ca

pytestmark = pytest.mark.gpu


def test_workspaces_that_are_none_are_refused():
    """On the host, before anything is launched."""
    q = torch.randn(1, 100, 2, 64, device="cuda").bfloat16()
    ap = params("none", 64)
    lse = torch.zeros(1, 2, 100, device="cuda")
    good = kv().new_key_weights_workspace(q, q, ap)
    for bad in (good.cpu(), torch.zeros(good.numel(), device="cuda"), torch.zeros(2 * good.numel(), dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace: want"):
            kv().key_weights(q, q, lse, ap, workspace=bad)
    with pytest.raises(ca.CapattnError, match="workspace"):
        kv().key_weights(q, q, lse, ap, workspace=good[:-256])
    assert torch.isfinite(kv().key_weights(q, q, lse, ap, workspace=good)).all()
    assert ca.capattn_device_status(good) == (0, 0)


@pytest.mark.parametrize("dtype, L, Lk", [(torch.bfloat16, 262_144, 152 * 128), (torch.float32, 131_072, 64)], ids=["bf16", "fp32"])
@pytest.mark.parametrize("norm", [9.1, 9.77, 10.3, 10.9])
def test_sums_of_long_prompts_are_compensated(dtype, L, Lk, norm):
    """Every pair counts alike (q is zero), so that a running sum would round the same way
    at each of its 2048 steps, 1e-6 to 3e-5 in all.  The call over all rows against the
    sum, in 64 bits, of calls over 16 ranges of them, whose exponentials and sums of a
    tile are the same: a compensated sum is off by 2 half steps, and some 16 parts and 4
    pieces are added behind it; either side, so twice that."""
    q = torch.zeros(1, L, 1, 64, dtype=dtype, device="cuda")
    k = torch.randn(1, Lk, 1, 64, device="cuda").to(dtype)
    lse = torch.full((1, 1, L), norm, device="cuda")
    ap = ca.AttnParams(sm_scale=0.125, cap_method="none", causal=False)
    ws = kv().new_key_weights_workspace(q, k, ap)
    w = kv().key_weights(q, k, lse, ap, workspace=ws).double()
    parts = torch.zeros_like(w)
    for i in range(16):
        rows = torch.tensor([[i * L // 16, (i + 1) * L // 16]], dtype=torch.int32, device="cuda")
        parts += kv().key_weights(q, k, lse, ap, rows=rows, workspace=ws).double()
    assert ca.capattn_device_status(ws) == (0, 0)
    assert ((w - parts).abs() <= 2 * (2 + 16 + 4) * EPS32 * parts).all()
    # an exponential: 8 half steps and 2 of its argument
    exact = L * math.exp(-float(torch.tensor(norm)))
    assert ((w - exact).abs() <= (8 + 2 * norm + 2 * 22 + 64) * EPS32 * exact).all()


@pytest.mark.parametrize("cap", ["none", "tanh", "tanh50", "soft_sign", "alsc30"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("junk", [math.nan, math.inf, 3e38])
def test_padding_may_hold_anything(dtype, cap, junk):
    """Rows that are not counted, and keys that only they see."""
    g = torch.Generator().manual_seed(5)
    L, D, used = 300, 64, [300, 170, 1, 0]
    B = len(used)
    q, k = (torch.randn(B, L, h, D, generator=g).to(dtype).cuda() for h in (4, 2))
    temp = (0.5 + torch.rand(B, L, generator=g)).cuda()
    ap = params(cap, D, window=90)
    _, lse, _, _ = ca.capattn_fwd(q, k, k.clone(), ap, temp)
    rows = torch.tensor([[0, n] for n in used], dtype=torch.int32, device="cuda")
    want = kv().key_weights(q, k, lse, ap, temp, rows=rows)
    for b, n in enumerate(used):
        q[b, n:], k[b, n:], temp[b, n:], lse[b, :, n:] = junk, junk, junk, -junk
    ws = kv().new_key_weights_workspace(q, k, ap)
    got = kv().key_weights(q, k, lse, ap, temp, rows=rows, workspace=ws)
    assert ca.capattn_device_status(ws) == (0, 0)
    for b, n in enumerate(used):
        assert (got[b, :, n:] == 0).all()
        # whether a chunk takes the short polynomial goes by all its scores, the junk's
        # among them, so what is kept may differ by the polynomials' 3e-8 and a few
        # roundings of a score of less than 8 after the temperature
        assert torch.allclose(got[b, :, :n], want[b, :, :n], rtol=8 * 16 * EPS32, atol=0)
