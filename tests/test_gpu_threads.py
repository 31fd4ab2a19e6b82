"""GPU tests of calls from a host thread that has made no CUDA call of its own: the tensor
maps of the bf16 kernels need a context there."""

import threading

import pytest
import torch

from kv_cache_utils import Pool
from soft_capped_attention_gb300 import capattn as ca
from test_gpu_kv_cache import kv, params

pytestmark = pytest.mark.gpu


def in_a_thread(work):
    failed = []

    def body():
        try:
            work()
        except Exception as e:  # carried over to the test's thread
            failed.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def test_decode():
    cache, ap = Pool([100, 50], 2, 128, 16, torch.bfloat16, 1).cuda(), params("tanh", 128)
    q = torch.randn(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    want = kv().cache_decode(q, cache, ap)
    out = tuple(torch.zeros_like(x) for x in want)
    in_a_thread(lambda: kv().cache_decode(q, cache, ap, out=out))
    assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_forward_and_backward():
    ap = ca.AttnParams(sm_scale=0.1, cap_method="tanh", cap=20.0, causal=True)
    q, k, v, do = (torch.randn(1, 300, h, 128, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2, 4))
    ws = ca.new_workspace(ca._config(q, k, ap), q.device)
    fwd = ca.capattn_fwd(q, k, v, ap, workspace=ws)
    bwd = ca.capattn_bwd(q, k, v, fwd[0], fwd[1], do, ap, workspace=ws)
    out, grads = [x.clone().zero_() for x in fwd[:2]] + [None, None], [torch.zeros_like(x) for x in bwd]
    in_a_thread(lambda: (ca.capattn_fwd(q, k, v, ap, workspace=ws, out=out)))
    in_a_thread(lambda: (ca.capattn_bwd(q, k, v, fwd[0], fwd[1], do, ap, workspace=ws, out=grads)))
    assert all(torch.equal(x, y) for x, y in zip(out[:2] + grads, list(fwd[:2]) + list(bwd)))
