"""Python binding of the paged key-value cache (argument checks and marshalling only).

The calls mirror include/capattn_cache.h: ``cache_append`` writes new keys and
values into their sequences' pages, ``cache_decode`` is attention of one new
token per sequence over its cached tokens with the caps of ``AttnParams``,
``cache_evict`` keeps the heaviest tokens of each head, and ``key_weights`` gives
the attention weight that each key of a prompt received, which starts a cache's
weights.  Lengths (and positions) are the caller's device tensors, taken as they
are after the new tokens, so that a decoding step is::

    cache.lens += 1
    cache_append(cache, k, v)
    o, lse = cache_decode(q, cache, ap)

and can be captured into a CUDA graph.  There is no fallback: if the shared
library is missing, every call raises.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import capattn as _ca
from .capattn import AttnParams, CAP_METHODS, DTYPES

HEADER_BYTES = 4096  # of a cache workspace, zero before its first use
CALL_APPEND, CALL_DECODE, CALL_DECODE_WEIGHTS, CALL_EVICT = 0, 1, 2, 3
EXPORTED_SYMBOLS = ("capattn_cache_validate_config", "capattn_cache_workspace_bytes", "capattn_cache_append",
                    "capattn_cache_decode", "capattn_cache_evict", "capattn_key_weights",
                    "capattn_key_weights_workspace_bytes")


class CacheConfig(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("cap_method", ctypes.c_int32),
                ("cap", ctypes.c_float), ("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("sm_scale", ctypes.c_float), ("window_len", ctypes.c_int32), ("B", ctypes.c_int32),
                ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


_lib_handle = None


def lib() -> ctypes.CDLL:
    """The loaded library with the cache's signatures; raises if it has not been built."""
    global _lib_handle
    if _lib_handle is None:
        h = _ca.lib()
        vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        cfgp = ctypes.POINTER(CacheConfig)
        h.capattn_cache_validate_config.restype = ctypes.c_int
        h.capattn_cache_validate_config.argtypes = [cfgp]
        h.capattn_cache_workspace_bytes.restype = sz
        h.capattn_cache_workspace_bytes.argtypes = [cfgp, ctypes.c_int]
        h.capattn_cache_append.restype = ctypes.c_int
        h.capattn_cache_append.argtypes = [cfgp, vp, vp, i64, i64, i32] + [vp] * 9 + [sz, vp]
        h.capattn_cache_decode.restype = ctypes.c_int
        h.capattn_cache_decode.argtypes = [cfgp, vp, i64] + [vp] * 11 + [sz, vp]
        h.capattn_cache_evict.restype = ctypes.c_int
        h.capattn_cache_evict.argtypes = [cfgp, i32, i32, i32] + [vp] * 12 + [sz, vp]
        h.capattn_key_weights_workspace_bytes.restype = sz
        h.capattn_key_weights_workspace_bytes.argtypes = [ctypes.POINTER(_ca.CapattnConfig)]
        h.capattn_key_weights.restype = ctypes.c_int
        h.capattn_key_weights.argtypes = [ctypes.POINTER(_ca.CapattnConfig)] + [vp] * 8 + [i64, vp, sz, vp]
        _lib_handle = h
    return _lib_handle


def make_cache_config(ap: AttnParams, B: int, Hq: int, Hkv: int, D: int, dtype: torch.dtype,
                      num_pages: int, page_size: int, max_pages: int) -> CacheConfig:
    if dtype not in DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    if ap.cap_method not in CAP_METHODS:
        raise ValueError(f"unknown cap method {ap.cap_method!r}")
    c = CacheConfig()
    c.struct_size = ctypes.sizeof(CacheConfig)
    c.cap_method = CAP_METHODS[ap.cap_method]
    c.cap, c.alpha, c.beta, c.sm_scale = ap.cap, ap.alpha, ap.beta, ap.sm_scale
    c.window_len = ap.window_len
    c.B, c.Hq, c.Hkv, c.D, c.dtype = B, Hq, Hkv, D, DTYPES[dtype]
    c.num_pages, c.page_size, c.max_pages = num_pages, page_size, max_pages
    return c


def cache_workspace_bytes(cfg: CacheConfig, call: int) -> int:
    return int(lib().capattn_cache_workspace_bytes(ctypes.byref(cfg), call))


def _fits(t, shape, dtype, device):
    return t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous()


def _want(t, what, shape, dtype, device):
    """A contiguous tensor of that shape, type and device, or None; gives its address."""
    if t is None:
        return None
    if not _fits(t, shape, dtype, device):
        raise ValueError(f"{what}: want a contiguous {dtype} tensor {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


def _rows(t, what, shape, dtype, device):
    """Rows of contiguous [heads, D] blocks; returns the row stride in elements."""
    n, heads, D = shape
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{what}: want a {dtype} tensor {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return heads * D
    stride = t.stride()
    if n and (stride[2] != 1 or (heads > 1 and stride[1] != D)):
        raise ValueError(f"{what}: the [heads, D] block of a row has to be contiguous, strides are {stride}")
    return stride[0] if n > 1 else heads * D


def _raw_stream(device, stream):
    """The handle of the current stream when the call needs no other device or
    stream than the current ones, else None."""
    if stream is None and torch._C._cuda_getDevice() == device.index:  # (CUDA is up: the tensors are there)
        return torch._C._cuda_getCurrentRawStream(device.index)  # the handle alone, without a Stream object
    return None


@contextlib.contextmanager
def _on(device, stream):
    """Makes `device` and the call's stream (by default the device's current one) the
    current ones, so that what a call allocates belongs to its stream."""
    if stream is None:
        with torch.cuda.device(device):
            yield
    else:
        if stream.device != device:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to {device}")
        with torch.cuda.stream(stream):
            yield


class _Plan:
    """A checked configuration and the workspace bytes of each call."""

    def __init__(self, cfg: CacheConfig):
        _ca._check(lib().capattn_cache_validate_config(ctypes.byref(cfg)), "KVCache")
        self.cfg = cfg
        self.ref = ctypes.byref(cfg)
        self.bytes = [cache_workspace_bytes(cfg, c) for c in range(4)]
        self.lse_like = None  # a tensor of lse's shape, which new ones are made like
        self.paged = None      # workspace bytes of the calls in paged.py


class KVCache:
    """A paged cache and what its calls share.

    k, v [num_pages, Hkv, page_size, D] (bf16 or fp32); table [B, max_pages]
    int32; lens [B] int32 (tokens held, at most max_len = max_pages *
    page_size); optional weights [B, Hkv, max_len] fp32 (attention weight
    received so far), pos [B, Hkv, max_len] int32 with qpos [B] int32
    (positions of the cached tokens and of each sequence's newest one).  All of
    them are the caller's; the cache adds one workspace, which grows to what its
    calls need.  Calls that may overlap on the GPU (two streams, two captured
    graphs) need a KVCache each (the tensors may be the same); keep a KVCache until
    the work that it enqueued on other streams has finished, and as long as a graph
    that captured its calls is replayed.  The calls are for serving: they record no
    gradients."""

    def __init__(self, k, v, table, lens, weights=None, pos=None, qpos=None):
        if k.dim() != 4 or table.dim() != 2:
            raise ValueError("k is [num_pages, Hkv, page_size, D] and table [B, max_pages]")
        if k.dtype not in DTYPES:
            raise ValueError(f"unsupported dtype {k.dtype}")
        if k.device.type != "cuda":
            raise ValueError(f"the cache has to be on a GPU, got {k.device}")
        self.num_pages, self.Hkv, self.page_size, self.D = k.shape
        self.B, self.max_pages = table.shape
        self.max_len = self.max_pages * self.page_size
        self.device, self.dtype = k.device, k.dtype
        slots = (self.B, self.Hkv, self.max_len)
        self._k_shape = k.shape
        _want(k, "k", k.shape, k.dtype, k.device)
        _want(v, "v", k.shape, k.dtype, k.device)
        _want(table, "table", table.shape, torch.int32, k.device)
        _want(lens, "lens", (self.B,), torch.int32, k.device)
        _want(weights, "weights", slots, torch.float32, k.device)
        _want(pos, "pos", slots, torch.int32, k.device)
        _want(qpos, "qpos", (self.B,), torch.int32, k.device)
        if pos is not None and qpos is None:
            raise ValueError("pos needs qpos, the position of each sequence's newest token")
        self.k, self.v, self.table, self.lens = k, v, table, lens
        self.weights, self.pos, self.qpos = weights, pos, qpos
        self._slots = torch.Size(slots)
        self._seen = (k, v, table, lens)  # checked above
        self._plans = {}       # by Hq and the parameters that count
        self._workspace_at = self._workspace_bytes = 0
        self._workspaces = []  # the last one is used; earlier ones may live in captured graphs

    def plan(self, Hq: int, ap: AttnParams | None = None) -> _Plan:
        key = (Hq,) if ap is None else (Hq, ap.sm_scale, ap.cap_method, ap.cap, ap.alpha, ap.beta, ap.window_len)
        got = self._plans.get(key)
        if got is None:
            cfg = make_cache_config(ap or AttnParams(sm_scale=1.0), self.B, Hq, self.Hkv, self.D, self.dtype,
                                    self.num_pages, self.page_size, self.max_pages)
            got = self._plans[key] = _Plan(cfg)
        return got

    def workspace(self, plan: _Plan, call: int) -> tuple[int, int]:
        """The cache's workspace (its address and bytes), at least as large as `call` needs.  A larger call's
        first use adds a larger one (so make that call once before a graph is
        captured); the earlier ones stay, since captured graphs may hold them."""
        return self._room(plan.bytes[call])

    def _room(self, n: int) -> tuple[int, int]:
        if self._workspace_bytes < n:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the cache's workspace would grow during a graph capture: "
                                   "make the call once before capturing it")
            new = torch.empty(n, dtype=torch.uint8, device=self.device)
            new[:HEADER_BYTES].zero_()  # the status word and the counters
            self._workspaces.append(new)
            self._workspace_at, self._workspace_bytes = new.data_ptr(), n
        return self._workspace_at, self._workspace_bytes

    def _tensors(self):
        """Addresses of the cache's own tensors.  They are the caller's to replace: a
        new one is checked as the first was."""
        k, v, table, lens = now = (self.k, self.v, self.table, self.lens)
        seen = self._seen
        if k is not seen[0] or v is not seen[1] or table is not seen[2] or lens is not seen[3]:
            B, dev = self.B, self.device
            if not (_fits(k, self._k_shape, self.dtype, dev) and _fits(v, self._k_shape, self.dtype, dev)):
                raise ValueError(f"the cache's k and v have to stay {tuple(self._k_shape)} {self.dtype} on {dev}")
            _want(table, "table", (B, self.max_pages), torch.int32, dev)
            _want(lens, "lens", (B,), torch.int32, dev)
            self._seen = now
        return k.data_ptr(), v.data_ptr(), table.data_ptr(), lens.data_ptr()

    def _positions(self):
        if self.pos is None:
            return None, None
        if self.qpos is None:
            raise ValueError("pos needs qpos, the position of each sequence's newest token")
        return (_want(self.pos, "pos", self._slots, torch.int32, self.device),
                _want(self.qpos, "qpos", (self.B,), torch.int32, self.device))

    def status(self, stream=None) -> tuple[int, int]:
        """Synchronises `stream` (the current one); returns (status, raw bits) of the calls so
        far, on other streams of those that have finished, and clears them."""
        status, raw = 0, 0
        with _on(self.device, stream):
            for w in self._workspaces:
                bits = ctypes.c_uint32(0)
                st = lib().capattn_device_status(w.data_ptr(), torch.cuda.current_stream().cuda_stream, ctypes.byref(bits))
                status, raw = status or int(st), raw | int(bits.value)
        return status, raw


def cache_append(cache: KVCache, k_new, v_new, cu_new=None, stream=None) -> None:
    """Writes new tokens into the cache.  k_new, v_new [N, Hkv, D] (rows may be
    strided, as slices of a fused projection are); the rows of sequence b are
    cu_new[b] .. cu_new[b + 1] - 1 (cu_new [B + 1] int32; None: one row a
    sequence).  cache.lens (and qpos) already count the new tokens: the n rows of
    sequence b go to slots lens[b] - n .. lens[b] - 1.  Their weights start at 0."""
    s = _raw_stream(cache.device, stream)
    if s is None:
        with _on(cache.device, stream):
            return cache_append(cache, k_new, v_new, cu_new)
    N = k_new.shape[0]
    shape = (N, cache.Hkv, cache.D)
    ks = _rows(k_new, "k_new", shape, cache.dtype, cache.device)
    vs = _rows(v_new, "v_new", shape, cache.dtype, cache.device)
    if cu_new is None and N != cache.B:
        raise ValueError(f"without cu_new there is one new row a sequence: got {N} rows, {cache.B} sequences")
    cu = _want(cu_new, "cu_new", (cache.B + 1,), torch.int32, cache.device)
    weights = _want(cache.weights, "weights", cache._slots, torch.float32, cache.device)
    k, v, table, lens = cache._tensors()
    pos, qpos = cache._positions()
    plan = cache.plan(cache.Hkv)
    ws, ws_bytes = cache.workspace(plan, CALL_APPEND)
    st = _lib_handle.capattn_cache_append(plan.ref, k_new.data_ptr(), v_new.data_ptr(), ks, vs, N, cu, k, v, table,
                                          lens, weights, pos, qpos, ws, ws_bytes, s)
    _ca._check(st, "capattn_cache_append")


def cache_decode(q, cache: KVCache, ap: AttnParams, temp=None, accumulate=False, out=None, stream=None):
    """Attention of one new token per sequence over its cached tokens.  q [B, Hq, D]
    (rows may be strided); temp [B] fp32 optional.  Returns (o [B, Hq, D],
    lse [B, Hq]); a sequence without live tokens gives o = 0, lse = -inf.  With
    accumulate, every cached token's share of the group's attention is added to
    cache.weights.  out: preallocated (o, lse).  ap's z_loss_weight plays no
    part, and causal none either: the query stands behind every cached token."""
    s = _raw_stream(cache.device, stream)
    if s is None:
        with _on(cache.device, stream):
            return cache_decode(q, cache, ap, temp, accumulate, out)
    if q.dim() != 3:
        raise ValueError("q is [B, Hq, D]")
    Hq, dev = q.shape[1], cache.device
    shape = (cache.B, Hq, cache.D)
    flat = q.is_contiguous()
    if flat and q.shape == shape and q.dtype is cache.dtype and q.device == dev:
        qs = Hq * cache.D
    else:
        qs = _rows(q, "q", shape, cache.dtype, dev)
    tp = None if temp is None else _want(temp, "temp", (cache.B,), torch.float32, dev)
    weights = pos = qpos = None
    if accumulate:
        if cache.weights is None:
            raise ValueError("accumulate needs a cache with weights")
        weights = _want(cache.weights, "weights", cache._slots, torch.float32, dev)
    k, v, table, lens = cache._tensors()
    if cache.pos is not None:
        pos, qpos = cache._positions()
    plan = cache.plan(Hq, ap)
    if out is None:
        o = torch.empty_like(q) if flat else torch.empty(shape, dtype=q.dtype, device=dev)
        if plan.lse_like is None:
            plan.lse_like = torch.empty((cache.B, Hq), dtype=torch.float32, device=dev)
        lse = torch.empty_like(plan.lse_like)  # (half the time of naming shape, type and device)
    else:
        o, lse = out
        _want(o, "o", shape, cache.dtype, dev)
        _want(lse, "lse", (cache.B, Hq), torch.float32, dev)
    ws, ws_bytes = cache.workspace(plan, CALL_DECODE_WEIGHTS if accumulate else CALL_DECODE)
    st = _lib_handle.capattn_cache_decode(plan.ref, q.data_ptr(), qs, k, v, table, lens, tp, pos, qpos, o.data_ptr(),
                                          lse.data_ptr(), weights, ws, ws_bytes, s)
    if st:
        _ca._check(st, "capattn_cache_decode")
    return o, lse


def cache_evict(cache: KVCache, budget: int, keep_first: int = 0, keep_last: int = 0, out=None, want_src=True,
                stream=None):
    """Keeps at most `budget` tokens of every (sequence, KV head): the first
    keep_first and last keep_last positions, then the heaviest (ties: the lower
    slot).  Kept tokens behind the budget move into the freed slots; lens,
    weights and pos follow, in place, or into out = (lens, weights, pos) (pos None
    without positions).  Returns src [B, Hkv, budget] int32, the slot each kept
    token came from (-1: none), or None without want_src.  Without pos a moved
    token loses its place in the text: windows and later keep_last then go by
    slots."""
    s = _raw_stream(cache.device, stream)
    if s is None:
        with _on(cache.device, stream):
            return cache_evict(cache, budget, keep_first, keep_last, out, want_src)
    if cache.weights is None:
        raise ValueError("eviction needs a cache with weights")
    if budget < 1 or budget > cache.max_len or keep_first < 0 or keep_last < 0 or keep_first + keep_last > budget:
        raise ValueError(f"want 1 <= budget <= {cache.max_len} and keep_first + keep_last <= budget, got "
                         f"{budget}, {keep_first}, {keep_last}")
    dev = cache.device
    weights = _want(cache.weights, "weights", cache._slots, torch.float32, dev)
    k, v, table, lens = cache._tensors()
    pos, qpos = cache._positions()
    if out is None:
        lens_out, weights_out, pos_out = lens, weights, pos
    else:
        if (out[2] is None) != (cache.pos is None):
            raise ValueError("pos_out goes with the cache's pos")
        lens_out = _want(out[0], "lens_out", (cache.B,), torch.int32, dev)
        weights_out = _want(out[1], "weights_out", cache._slots, torch.float32, dev)
        pos_out = _want(out[2], "pos_out", cache._slots, torch.int32, dev)
    plan = cache.plan(cache.Hkv)
    src = torch.empty((cache.B, cache.Hkv, budget), dtype=torch.int32, device=dev) if want_src else None
    ws, ws_bytes = cache.workspace(plan, CALL_EVICT)
    st = _lib_handle.capattn_cache_evict(plan.ref, budget, keep_first, keep_last, k, v, table, lens, weights, pos, qpos,
                                         lens_out, weights_out, pos_out, None if src is None else src.data_ptr(),
                                         ws, ws_bytes, s)
    _ca._check(st, "capattn_cache_evict")
    return src


@functools.lru_cache(maxsize=64)
def _prompt_plan(ap: AttnParams, B: int, L: int, Hq: int, Hkv: int, D: int, dtype: torch.dtype, Lk: int):
    """A checked configuration of key_weights, its reference and workspace bytes."""
    cfg = _ca.make_config(ap, B, L, Hq, Hkv, D, dtype, Lk=Lk)
    n = int(lib().capattn_key_weights_workspace_bytes(ctypes.byref(cfg)))
    if n == 0:
        _ca._check(lib().capattn_validate_config(ctypes.byref(cfg)), "capattn_key_weights_workspace_bytes")
    return cfg, ctypes.byref(cfg), n


def new_key_weights_workspace(q, k, ap: AttnParams) -> torch.Tensor:
    """Workspace of key_weights for q [B, L, Hq, D] and k [B, Lk, Hkv, D]."""
    B, L, Hq, D = q.shape
    n = _prompt_plan(ap, B, L, Hq, k.shape[2], D, q.dtype, k.shape[1])[2]
    ws = torch.empty(n, dtype=torch.uint8, device=q.device)
    ws[:256].zero_()  # the status word
    return ws


def key_weights(q, k, lse, ap: AttnParams, temp=None, seg=None, bounds=None, rows=None, out=None, workspace=None,
                stream=None):
    """The attention weight that each key received: w[b, g, j] = sum over the query
    heads of group g and the counted rows i of exp(t_ij - lse_i), with the masks
    and the lse of capattn_fwd for the same inputs.  rows [B, 2] int32: the
    counted query rows lo <= i < hi (None: all).  Returns w [B, Hkv, W] fp32, W =
    Lk, or `out` with W >= Lk (a cache's weights, for instance), of which the
    entries j < Lk are overwritten."""
    dev = q.device
    if dev.type != "cuda":
        raise ValueError(f"q has to be on a GPU, got {dev}")
    s = _raw_stream(dev, stream)
    if s is None:
        with _on(dev, stream):
            return key_weights(q, k, lse, ap, temp, seg, bounds, rows, out, workspace)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q is [B, L, Hq, D] and k [B, Lk, Hkv, D]")
    B, L, Hq, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    qp = _want(q, "q", q.shape, q.dtype, dev)
    kp = _want(k, "k", (B, Lk, Hkv, D), q.dtype, dev)
    lp = _want(lse, "lse", (B, Hq, L), torch.float32, dev)
    tp = _want(temp, "temp", (B, L), torch.float32, dev)
    sp = _want(seg, "seg", (B, L), torch.int32, dev)
    bp = _want(bounds, "bounds", (B, 4), torch.int32, dev)
    rp = _want(rows, "rows", (B, 2), torch.int32, dev)
    cfg, ref, _ = _prompt_plan(ap, B, L, Hq, Hkv, D, q.dtype, Lk)
    if out is None:
        out = torch.empty((B, Hkv, Lk), dtype=torch.float32, device=dev)
    elif out.dim() != 3 or out.shape[2] < Lk:
        raise ValueError(f"out is [B, Hkv, W] with W >= {Lk}, got {tuple(out.shape)}")
    W = out.shape[2]
    op = _want(out, "out", (B, Hkv, W), torch.float32, dev)
    if workspace is None:
        workspace = new_key_weights_workspace(q, k, ap)
    _want(workspace, "workspace", workspace.shape, torch.uint8, dev)
    st = lib().capattn_key_weights(ref, qp, kp, lp, tp, sp, bp, rp, op, W, workspace.data_ptr(), workspace.numel(), s)
    _ca._check(st, "capattn_key_weights")
    return out
