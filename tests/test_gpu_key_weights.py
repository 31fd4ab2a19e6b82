"""GPU tests of key_weights beyond its formula: refusals and what stays out of its sums."""

import math

import pytest
import torch

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
