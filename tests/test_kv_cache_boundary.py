"""CPU tests of the paged cache's boundary: the library exports what
capattn_cache.h declares, and every call refuses bad arguments on the host
before it launches anything."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from soft_capped_attention_gb300 import capattn as ca
from soft_capped_attention_gb300 import kv_cache as kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ca.LIB_PATH):
        from soft_capped_attention_gb300 import build
        build.build()
    return kv.lib()


def cfg(**kw):
    d = dict(B=2, Hq=4, Hkv=2, D=128, dtype=torch.bfloat16, num_pages=10, page_size=16, max_pages=4)
    ap = ca.AttnParams(sm_scale=kw.pop("sm_scale", 0.1), cap_method=kw.pop("cap_method", "tanh"),
                       cap=kw.pop("cap", 5.0), window_len=kw.pop("window_len", 0))
    d.update(kw)
    return kv.make_cache_config(ap, **d)


P = ctypes.c_void_p(4096)     # an aligned address that no refused call touches
ODD = ctypes.c_void_p(4104)   # 8-byte aligned only
WS = 1 << 40


def test_header_and_library_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "capattn_cache.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(capattn_[a-z_]+)\s*\(", text))
    assert names == set(kv.EXPORTED_SYMBOLS)
    for n in names:
        assert hasattr(lib, n), n


def test_the_header_is_plain_c(tmp_path):
    gcc, cuda = shutil.which("gcc"), "/usr/local/cuda/include"
    if gcc is None or not os.path.exists(os.path.join(cuda, "cuda_runtime_api.h")):
        pytest.skip("gcc or the CUDA headers are not available")
    src = tmp_path / "c.c"
    src.write_text('#include "capattn_cache.h"\nint main(void) { capattn_cache_config c = {0};'
                   ' return (int)sizeof(c) - 60 + (int)capattn_cache_validate_config(0); }\n')
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                    "-isystem", cuda, str(src)], check=True)
    assert ctypes.sizeof(kv.CacheConfig) == 60


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"D": 64}, 0), ({"dtype": torch.float32}, 0), ({"page_size": 8}, 0), ({"page_size": 1024}, 0),
    ({"Hq": 3}, 1), ({"B": 0}, 1), ({"num_pages": 0}, 1), ({"max_pages": 0}, 1), ({"page_size": 0}, 1),
    ({"window_len": -1}, 1), ({"sm_scale": float("nan")}, 1), ({"cap": float("inf")}, 1),
    ({"D": 96}, 2), ({"page_size": 24}, 2), ({"page_size": 4}, 2), ({"page_size": 2048}, 2),
    ({"max_pages": 1 << 27}, 2), ({"num_pages": 1 << 27}, 2), ({"B": 1 << 20, "max_pages": 1 << 14}, 2),
], ids=str)
def test_config(lib, kw, status):
    c = cfg(**kw)
    assert lib.capattn_cache_validate_config(ctypes.byref(c)) == status
    sizes = [lib.capattn_cache_workspace_bytes(ctypes.byref(c), i) for i in range(-1, 5)]
    assert sizes[0] == sizes[5] == 0
    assert all((s > 0) == (status == 0) for s in sizes[1:5])


def test_config_struct_size(lib):
    c = cfg()
    c.struct_size -= 4
    assert lib.capattn_cache_validate_config(ctypes.byref(c)) == 1
    assert lib.capattn_cache_validate_config(None) == 1


def append_args(**kw):
    a = dict(cfg=cfg(), k_new=P, v_new=P, ks=256, vs=256, n=2, cu=None, k=P, v=P, table=P, lens=P, weights=None,
             pos=None, qpos=None, ws=P, wb=WS)
    a.update(kw)
    return [ctypes.byref(a["cfg"])] + [a[n] for n in list(a)[1:]] + [None]


@pytest.mark.parametrize("kw,status", [
    ({"k_new": None}, 1), ({"v_new": None}, 1), ({"k": None}, 1), ({"v": None}, 1), ({"table": None}, 1),
    ({"lens": None}, 1), ({"n": -1}, 1), ({"n": 3}, 1), ({"ks": 255}, 1), ({"ks": 128}, 1), ({"vs": 260}, 1),
    ({"pos": P}, 1), ({"k_new": ODD}, 1), ({"k": ODD}, 1), ({"weights": ODD}, 1), ({"ws": None}, 5), ({"ws": ODD}, 5),
    ({"wb": 4095}, 5), ({"cfg": cfg(D=96)}, 2), ({"n": 0, "cu": P, "k_new": None, "v_new": None}, 0),
], ids=str)
def test_append_refusals(lib, kw, status):
    assert lib.capattn_cache_append(*append_args(**kw)) == status


def decode_args(**kw):
    a = dict(cfg=cfg(), q=P, qs=512, k=P, v=P, table=P, lens=P, temp=None, pos=None, qpos=None, o=P, lse=P,
             weights=None, ws=P, wb=WS)
    a.update(kw)
    return [ctypes.byref(a["cfg"])] + [a[n] for n in list(a)[1:]] + [None]


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, 1), ({"k": None}, 1), ({"v": None}, 1), ({"table": None}, 1), ({"lens": None}, 1), ({"o": None}, 1),
    ({"lse": None}, 1), ({"pos": P}, 1), ({"qs": 511}, 1), ({"qs": 256}, 1), ({"q": ODD}, 1), ({"temp": ODD}, 1),
    ({"ws": None}, 5), ({"wb": 4096}, 5), ({"cfg": cfg(page_size=12)}, 2), ({"cfg": cfg(Hq=5)}, 1),
], ids=str)
def test_decode_refusals(lib, kw, status):
    assert lib.capattn_cache_decode(*decode_args(**kw)) == status


def test_decode_with_weights_needs_the_larger_workspace(lib):
    c = cfg()
    small = lib.capattn_cache_workspace_bytes(ctypes.byref(c), kv.CALL_DECODE)
    assert lib.capattn_cache_workspace_bytes(ctypes.byref(c), kv.CALL_DECODE_WEIGHTS) >= small + 2 * 4 * 64 * 4
    assert lib.capattn_cache_decode(*decode_args(weights=P, wb=small)) == 5


def evict_args(**kw):
    a = dict(cfg=cfg(), budget=8, first=1, last=2, k=P, v=P, table=P, lens=P, weights=P, pos=None, qpos=None, lens_out=P,
             weights_out=P, pos_out=None, src=None, ws=P, wb=WS)
    a.update(kw)
    return [ctypes.byref(a["cfg"])] + [a[n] for n in list(a)[1:]] + [None]


@pytest.mark.parametrize("kw,status", [
    ({"budget": 0}, 1), ({"budget": 65}, 1), ({"first": -1}, 1), ({"last": -1}, 1), ({"first": 5, "last": 4}, 1),
    ({"first": 2 ** 31 - 1, "last": 8}, 1), ({"weights": None}, 1), ({"weights_out": None}, 1), ({"lens_out": None}, 1),
    ({"pos": P, "pos_out": P}, 1), ({"pos": P, "qpos": P}, 1), ({"pos_out": P}, 1), ({"src": ODD}, 1), ({"k": None}, 1),
    ({"ws": ODD}, 5), ({"wb": 256}, 5),
], ids=str)
def test_evict_refusals(lib, kw, status):
    assert lib.capattn_cache_evict(*evict_args(**kw)) == status


def weights_args(**kw):
    c = ca.make_config(ca.AttnParams(sm_scale=0.1, causal=True), 1, 100, 4, 2, 128, torch.bfloat16, Lk=kw.pop("Lk", 0))
    a = dict(q=P, k=P, lse=P, temp=None, seg=None, bounds=None, rows=None, w=P, stride=100, ws=P, wb=WS)
    a.update(kw)
    return [ctypes.byref(c)] + list(a.values()) + [None]


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, 1), ({"k": None}, 1), ({"lse": None}, 1), ({"w": None}, 1), ({"stride": 99}, 1), ({"rows": ODD}, 1),
    ({"Lk": 120, "stride": 120, "seg": P}, 1), ({"Lk": 120}, 1), ({"ws": None}, 5), ({"wb": 100}, 5),
], ids=str)
def test_key_weights_refusals(lib, kw, status):
    assert lib.capattn_key_weights(*weights_args(**kw)) == status


def test_key_weights_workspace_holds_the_forwards(lib):
    for dtype in (torch.bfloat16, torch.float32):
        c = ca.make_config(ca.AttnParams(sm_scale=0.1), 3, 1000, 4, 2, 64, dtype)
        n = lib.capattn_key_weights_workspace_bytes(ctypes.byref(c))
        assert n > lib.capattn_workspace_bytes(ctypes.byref(c), ca.PASS_FWD)
        assert lib.capattn_key_weights(*weights_args(wb=lib.capattn_workspace_bytes(ctypes.byref(c), 0))) == 5
    c.D = 96
    assert lib.capattn_key_weights_workspace_bytes(ctypes.byref(c)) == 0


def test_python_refuses_a_cache_off_the_gpu():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        kv.KVCache(k, k.clone(), table, lens)
    with pytest.raises(ValueError, match="unsupported dtype"):
        kv.KVCache(k.half(), k.half(), table, lens)
    with pytest.raises(ValueError, match="num_pages"):
        kv.KVCache(k[0], k[0], table, lens)
