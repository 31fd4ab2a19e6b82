"""Python binding of the steps with many new tokens per sequence over the paged cache
(argument checks and marshalling only).

The calls mirror include/capattn_paged.h and share a ``kv_cache.KVCache``:
``cache_plan`` makes a step's lengths, tables and slot maps from request lengths,
``cache_attend`` is attention of whole prompts, chunks of prompts or trees of drafted
tokens over what the cache holds, ``cache_verify`` accepts the drafted tokens that the
model agrees with and ``cache_accept`` a path that the caller chose.  A step::

    cu, slots, positions = cache_plan(cache, pool, n_new, rows)
    cache_append(cache, k, v, cu_new=cu)
    o, lse = cache_attend(q, cache, ap, cu, parents=parents)     # parents=None: a prompt
    path, count, token = cache_verify(cache, cu, tokens, predicted, parents, width)

Everything that depends on lengths stays on the device, so a step whose buffers have a
fixed size can be captured into a CUDA graph.  There is no fallback: if the shared
library is missing, every call raises.
"""

from __future__ import annotations

import ctypes

import torch

from . import capattn as _ca
from .capattn import AttnParams
from .kv_cache import KVCache, _on, _raw_stream, _rows, _want
from .kv_cache import lib as _cache_lib
from .kv_cache import CacheConfig

EXPORTED_SYMBOLS = ("capattn_paged_workspace_bytes", "capattn_paged_attend", "capattn_paged_plan",
                    "capattn_paged_accept")
CALL_ATTEND, CALL_PLAN, CALL_ACCEPT = 0, 1, 2

_lib_handle = None


def lib() -> ctypes.CDLL:
    """The loaded library with these calls' signatures; raises if it has not been built."""
    global _lib_handle
    if _lib_handle is None:
        h = _cache_lib()
        vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        cfgp = ctypes.POINTER(CacheConfig)
        h.capattn_paged_workspace_bytes.restype = sz
        h.capattn_paged_workspace_bytes.argtypes = [cfgp, ctypes.c_int]
        h.capattn_paged_attend.restype = ctypes.c_int
        h.capattn_paged_attend.argtypes = [cfgp, vp, i64, i32] + [vp] * 12 + [sz, vp]
        h.capattn_paged_plan.restype = ctypes.c_int
        h.capattn_paged_plan.argtypes = [cfgp] + [vp] * 11 + [i32] + [vp] * 4 + [sz, vp]
        h.capattn_paged_accept.restype = ctypes.c_int
        h.capattn_paged_accept.argtypes = [cfgp, vp, i32, vp, vp, vp, i32] + [vp] * 13 + [sz, vp]
        _lib_handle = h
    return _lib_handle


def _workspace(cache: KVCache, plan, call: int):
    if plan.paged is None:
        plan.paged = [int(lib().capattn_paged_workspace_bytes(plan.ref, c)) for c in range(3)]
    return cache._room(plan.paged[call])


class PagePool:
    """The pages of a cache that no sequence owns, and how many each sequence does.

    free [num_pages] int32, n_free [1] int32: a stack, free[:n_free]; held [B] int32: the
    pages of sequence b, table[b, :held[b]], at least those of its lens[b] tokens.  All of
    them are the caller's.  Sequences that share pages (a common prefix) cannot be planned:
    each page belongs to one sequence or to the stack."""

    def __init__(self, free, n_free, held):
        self.free, self.n_free, self.held = free, n_free, held

    @classmethod
    def full(cls, cache: KVCache) -> "PagePool":
        """A pool of all of the cache's pages; no sequence holds one."""
        i32 = dict(dtype=torch.int32, device=cache.device)
        return cls(torch.arange(cache.num_pages - 1, -1, -1, **i32), torch.full((1,), cache.num_pages, **i32),
                   torch.zeros(cache.B, **i32))


def cache_plan(cache: KVCache, pool: PagePool, n_new, rows: int, out=None, want_slots=True, stream=None):
    """The lengths, tables and slot maps of a step.  n_new [B] int32: tokens that each
    sequence is about to get, negative: it ends.  cache.lens (and, with positions,
    cache.qpos), pool.held and pool.n_free move on in place, or into out = (lens, qpos,
    held, n_free) (qpos None without positions); the table and the stack are written in
    place.  Returns cu_new [B + 1] int32, slots [rows] int64 (page * page_size + offset of
    each new token, -1 behind the last) and positions [rows] int32, the latter two None
    without want_slots.  A step that does not fit (pages, rows, max_len) changes nothing and
    sets a status bit; its cu_new is 0, so that the calls that follow do nothing."""
    s = _raw_stream(cache.device, stream)
    if s is None:
        with _on(cache.device, stream):
            return cache_plan(cache, pool, n_new, rows, out, want_slots)
    B, dev, i32 = cache.B, cache.device, torch.int32
    if rows < 0:
        raise ValueError(f"rows cannot be negative, got {rows}")
    nn = _want(n_new, "n_new", (B,), i32, dev)
    free = _want(pool.free, "pool.free", (cache.num_pages,), i32, dev)
    n_free = _want(pool.n_free, "pool.n_free", (1,), i32, dev)
    held = _want(pool.held, "pool.held", (B,), i32, dev)
    _, _, table, lens = cache._tensors()
    qpos = None if cache.pos is None else cache._positions()[1]
    if out is None:
        lens_out, qpos_out, held_out, n_free_out = lens, qpos, held, n_free
    else:
        if (out[1] is None) != (qpos is None):
            raise ValueError("qpos_out goes with the cache's positions")
        lens_out = _want(out[0], "lens_out", (B,), i32, dev)
        qpos_out = _want(out[1], "qpos_out", (B,), i32, dev)
        held_out = _want(out[2], "held_out", (B,), i32, dev)
        n_free_out = _want(out[3], "n_free_out", (1,), i32, dev)
    plan = cache.plan(cache.Hkv)
    ws, ws_bytes = _workspace(cache, plan, CALL_PLAN)
    cu = torch.empty(B + 1, dtype=i32, device=dev)
    slots = positions = None
    if want_slots:
        slots, positions = torch.empty(rows, dtype=torch.int64, device=dev), torch.empty(rows, dtype=i32, device=dev)
    st = _lib_handle.capattn_paged_plan(plan.ref, nn, table, lens, qpos, held, free, n_free, lens_out, qpos_out, held_out,
                                        n_free_out, rows, cu.data_ptr(), slots.data_ptr() if want_slots else None,
                                        positions.data_ptr() if want_slots else None, ws, ws_bytes, s)
    if st:
        _ca._check(st, "capattn_paged_plan")
    return cu, slots, positions


def cache_attend(q, cache: KVCache, ap: AttnParams, cu_new, parents=None, temp=None, out=None, stream=None):
    """Attention of new tokens over their sequence's cached tokens, their own among them
    (append them first).  q [N, Hq, D] (rows may be strided); the rows of sequence b are
    cu_new[b] .. cu_new[b + 1] - 1 (cu_new [B + 1] int32), its last tokens in the cache.
    Row i sees the slots up to its own, or with parents [N] int32 (a row's index within the
    sequence that it continues, less than its own; -1: none) the slots before the new
    tokens, itself and its ancestors; ap's window goes by positions, a drafted token's by
    its depth.  A tree has at most 8192 tokens.  temp [N] fp32 optional.  Returns (o [N, Hq, D], lse [N, Hq]); out:
    preallocated (o, lse; o apart from q), of which rows that belong to no sequence are left as they are.
    ap's causal and z_loss_weight play no part."""
    s = _raw_stream(cache.device, stream)
    if s is None:
        with _on(cache.device, stream):
            return cache_attend(q, cache, ap, cu_new, parents, temp, out)
    if q.dim() != 3:
        raise ValueError("q is [N, Hq, D]")
    N, Hq, dev = q.shape[0], q.shape[1], cache.device
    shape = (N, Hq, cache.D)
    qs = _rows(q, "q", shape, cache.dtype, dev)
    cu = _want(cu_new, "cu_new", (cache.B + 1,), torch.int32, dev)
    up = None if parents is None else _want(parents, "parents", (N,), torch.int32, dev)
    tp = None if temp is None else _want(temp, "temp", (N,), torch.float32, dev)
    k, v, table, lens = cache._tensors()
    pos = qpos = None
    if cache.pos is not None:
        pos, qpos = cache._positions()
    plan = cache.plan(Hq, ap)
    if out is None:
        o = torch.empty_like(q) if qs == Hq * cache.D and q.is_contiguous() else torch.empty(shape, dtype=q.dtype, device=dev)
        lse = torch.empty((N, Hq), dtype=torch.float32, device=dev)
    else:
        o, lse = out
        _want(o, "o", shape, cache.dtype, dev)
        _want(lse, "lse", shape[:2], torch.float32, dev)
    ws, ws_bytes = _workspace(cache, plan, CALL_ATTEND)
    st = _lib_handle.capattn_paged_attend(plan.ref, q.data_ptr(), qs, N, cu, up, k, v, table, lens, tp, pos, qpos,
                                          o.data_ptr(), lse.data_ptr(), ws, ws_bytes, s)
    if st:
        _ca._check(st, "capattn_paged_attend")
    return o, lse


def _accept(cache, cu_new, N, tokens, predicted, parents, path, width, count, nxt, out, s):
    """The call itself, on addresses; raises what it returns."""
    B, dev, i32 = cache.B, cache.device, torch.int32
    cu = _want(cu_new, "cu_new", (B + 1,), i32, dev)
    weights = None if cache.weights is None else _want(cache.weights, "weights", cache._slots, torch.float32, dev)
    k, v, table, lens = cache._tensors()
    pos = qpos = None
    if cache.pos is not None:
        pos, qpos = cache._positions()
    if out is None:
        lens_out, qpos_out = lens, qpos
    else:
        if (out[1] is None) != (qpos is None):
            raise ValueError("qpos_out goes with the cache's positions")
        lens_out = _want(out[0], "lens_out", (B,), i32, dev)
        qpos_out = _want(out[1], "qpos_out", (B,), i32, dev)
    plan = cache.plan(cache.Hkv)
    ws, ws_bytes = _workspace(cache, plan, CALL_ACCEPT)
    st = _lib_handle.capattn_paged_accept(plan.ref, cu, N, tokens, predicted, parents, width, path, count, nxt, k, v, table,
                                          lens, weights, pos, qpos, lens_out, qpos_out, ws, ws_bytes, s)
    if st:
        _ca._check(st, "capattn_paged_accept")


def cache_verify(cache: KVCache, cu_new, tokens, predicted, parents, width: int, out=None, stream=None):
    """Accepts the drafted tokens that the model agrees with.  tokens, predicted, parents [N]
    int32: the new tokens, the token that the model predicts behind each, and the row of its
    sequence that each continues.  A sequence's row 0 (the last sure token) is accepted, and
    from an accepted row the walk goes on to its first child whose token is what the model
    predicted there, up to `width` tokens.  Accepted tokens move to the front of the new
    slots, the others leave the cache: cache.lens (and qpos) follow, in place, or into out =
    (lens, qpos) (qpos None without positions).  Returns path [B, width] int32 (-1 behind
    its end), count [B] int32 and the next token [B] int32, predicted behind the last
    accepted one (-1 for a sequence without new tokens)."""
    dev, i32 = cache.device, torch.int32
    s = _raw_stream(dev, stream)
    if s is None:
        with _on(dev, stream):
            return cache_verify(cache, cu_new, tokens, predicted, parents, width, out)
    if width < 1:
        raise ValueError(f"width has to be at least 1, got {width}")
    B, rows = cache.B, tuple(tokens.shape)
    if len(rows) != 1:
        raise ValueError(f"tokens is [N], got {rows}")
    t = _want(tokens, "tokens", rows, i32, dev)
    m = _want(predicted, "predicted", rows, i32, dev)
    u = _want(parents, "parents", rows, i32, dev)
    path = torch.empty((B, width), dtype=i32, device=dev)
    count, nxt = torch.empty(B, dtype=i32, device=dev), torch.empty(B, dtype=i32, device=dev)
    if rows[0] == 0:  # nothing is drafted (an empty tensor has no address that says so)
        path.fill_(-1)
        count.zero_()
        nxt.fill_(-1)
        _accept(cache, cu_new, 0, None, None, None, path.data_ptr(), width, count.data_ptr(), None, out, s)
    else:
        _accept(cache, cu_new, rows[0], t, m, u, path.data_ptr(), width, count.data_ptr(), nxt.data_ptr(), out, s)
    return path, count, nxt


def cache_accept(cache: KVCache, cu_new, path, count, out=None, stream=None):
    """Accepts a path that the caller chose (by sampling, for instance): path [B, width]
    int32, strictly increasing rows of the sequence's new tokens, of which the first count[b]
    (count [B] int32) stay; the rest as in cache_verify."""
    dev, i32 = cache.device, torch.int32
    s = _raw_stream(dev, stream)
    if s is None:
        with _on(dev, stream):
            return cache_accept(cache, cu_new, path, count, out)
    if path.dim() != 2 or path.shape[1] < 1:
        raise ValueError("path is [B, width]")
    width = path.shape[1]
    at = _want(path, "path", (cache.B, width), i32, dev)
    _accept(cache, cu_new, 2 ** 31 - 1, None, None, None, at, width, _want(count, "count", (cache.B,), i32, dev), None, out, s)
