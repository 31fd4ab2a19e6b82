"""CPU tests of the boundary of the steps with many new tokens: the library exports what
capattn_paged.h declares, and every call refuses bad arguments on the host before it
launches anything."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from soft_capped_attention_gb300 import kv_cache as kv
from soft_capped_attention_gb300 import paged
from test_kv_cache_boundary import ODD, ROOT, WS, P, cfg, lib as _cache_lib  # noqa: F401


@pytest.fixture(scope="module")
def lib(_cache_lib):
    return paged.lib()


def test_header_and_library_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "capattn_paged.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(capattn_paged_[a-z_]+)\s*\(", text))
    assert names == set(paged.EXPORTED_SYMBOLS)
    for n in names:
        assert hasattr(lib, n), n


def test_the_header_is_plain_c(tmp_path):
    gcc, cuda = shutil.which("gcc"), "/usr/local/cuda/include"
    if gcc is None or not os.path.exists(os.path.join(cuda, "cuda_runtime_api.h")):
        pytest.skip("gcc or the CUDA headers are not available")
    src = tmp_path / "c.c"
    src.write_text('#include "capattn_paged.h"\nint main(void) { return (int)capattn_paged_workspace_bytes(0, CAPATTN_PAGED_PLAN); }\n')
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                    "-isystem", cuda, str(src)], check=True)


@pytest.mark.parametrize("kw,fine", [({}, True), ({"D": 64}, True), ({"dtype": torch.float32}, True), ({"D": 96}, False),
                                     ({"page_size": 12}, False), ({"Hq": 3}, False)], ids=str)
def test_workspace_bytes(lib, kw, fine):
    c = cfg(**kw)
    sizes = [lib.capattn_paged_workspace_bytes(ctypes.byref(c), i) for i in range(-1, 4)]
    assert sizes[0] == sizes[4] == 0 and all((s >= kv.HEADER_BYTES) == fine for s in sizes[1:4])
    assert lib.capattn_paged_workspace_bytes(None, 0) == 0


def args(defaults, kw):
    a = dict(defaults)
    a.update(kw)
    c = a.pop("cfg")
    return [ctypes.byref(c)] + list(a.values()) + [None]


ATTEND = dict(cfg=cfg(), q=P, qs=512, n=5, cu=P, up=None, k=P, v=P, table=P, lens=P, temp=None, pos=None, qpos=None, o=P, lse=P,
              ws=P, wb=WS)


@pytest.mark.parametrize("kw,status", [
    ({"q": None}, 1), ({"n": -1}, 1), ({"cu": None}, 1), ({"k": None}, 1), ({"v": None}, 1), ({"table": None}, 1),
    ({"lens": None}, 1), ({"o": None}, 1), ({"lse": None}, 1), ({"pos": P}, 1), ({"qs": 511}, 1), ({"qs": 256}, 1), ({"qs": -512}, 1),
    ({"q": ODD}, 1), ({"cu": ODD}, 1), ({"up": ODD}, 1), ({"temp": ODD}, 1), ({"o": ODD}, 1), ({"ws": None}, 5), ({"ws": ODD}, 5),
    ({"wb": 1 << 20}, 5), ({"cfg": cfg(D=96)}, 2), ({"cfg": cfg(Hq=5)}, 1), ({"n": 0, "q": None, "o": None, "lse": None}, 0),
], ids=str)
def test_attend_refusals(lib, kw, status):
    assert lib.capattn_paged_attend(*args(ATTEND, kw)) == status


@pytest.mark.parametrize("shift", [0, 16, 4 * 512 * 2 + 511 * 2 // 16 * 16, -(5 * 512 * 2 - 16)])
def test_outputs_over_the_queries_are_refused(lib, shift):
    """512 elements a row (bf16), five rows."""
    assert cfg().Hq * cfg().D == 512
    at = (P if isinstance(P, int) else P.value) + (1 << 20)
    assert lib.capattn_paged_attend(*args(ATTEND, dict(q=at, o=at + shift))) == 1


PLAN = dict(cfg=cfg(), n_new=P, table=P, lens=P, qpos=None, held=P, free=P, n_free=P, lens_out=P, qpos_out=None, held_out=P,
            n_free_out=P, rows=5, cu=P, slots=P, positions=P, ws=P, wb=WS)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, 1) for n in ("n_new", "table", "lens", "held", "free", "n_free", "lens_out", "held_out", "n_free_out", "cu")],
    *[({n: ODD}, 1) for n in ("n_new", "free", "slots", "positions", "cu", "lens_out")],
    ({"rows": -1}, 1), ({"qpos": P}, 1), ({"qpos_out": P}, 1), ({"ws": None}, 5), ({"wb": 4096}, 5), ({"cfg": cfg(B=0)}, 1),
], ids=str)
def test_plan_refusals(lib, kw, status):
    assert lib.capattn_paged_plan(*args(PLAN, kw)) == status


ACCEPT = dict(cfg=cfg(), cu=P, n=5, tokens=P, says=P, up=P, width=3, path=P, count=P, next=P, k=P, v=P, table=P, lens=P,
              weights=None, pos=None, qpos=None, lens_out=P, qpos_out=None, ws=P, wb=WS)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, 1) for n in ("cu", "path", "count", "k", "v", "table", "lens", "lens_out", "tokens", "says", "up")],
    *[({n: ODD}, 1) for n in ("cu", "path", "count", "next", "k", "tokens", "weights", "lens_out")],
    ({"n": -1}, 1), ({"width": 0}, 1), ({"pos": P}, 1), ({"qpos": P}, 1), ({"qpos_out": P}, 1),
    ({"tokens": None, "says": None, "up": None}, 1), ({"ws": None}, 5), ({"wb": 4095}, 5), ({"cfg": cfg(page_size=4)}, 2),
], ids=str)
def test_accept_refusals(lib, kw, status):
    assert lib.capattn_paged_accept(*args(ACCEPT, kw)) == status
