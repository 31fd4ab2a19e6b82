"""Plain forms of the steps with many new tokens, in 64 bits, and the error bounds that
their tests use."""

import math

import torch

from kv_cache_utils import EPS32, cap64


def chain(n):
    return list(range(-1, n - 1))


def ancestors(up):
    """For each row, itself and its ancestors; its depth is one less than their number."""
    kin = []
    for i, u in enumerate(up):
        kin.append((kin[u] if u >= 0 else []) + [i])
    return kin


def live_of(n, L, window, up=None, pos=None, newest=None):
    """[heads or 1, n, L] bool: the live slots of n new tokens behind L - n cached ones.  pos
    [heads, L] and newest: positions of the slots and of the last new token."""
    base = L - n
    j = torch.arange(L)
    live = torch.zeros(n, L, dtype=torch.bool)
    kin = ancestors(up) if up is not None else None
    depth = [len(k) - 1 for k in kin] if kin else list(range(n))
    for i in range(n):
        if kin:
            live[i, :base] = True
            live[i, [base + x for x in kin[i]]] = True
        else:
            live[i, :base + i + 1] = True
    if window <= 0:
        return live[None]
    first = base if newest is None else newest - n + 1  # position of the first new token
    at = j[None].clone() if pos is None else pos[:, :L].long().clone()
    if kin:
        at[:, base:] = first + torch.tensor(depth)
    place = first + torch.tensor(depth)
    return live[None] & (at[:, None, :] > place[None, :, None] - window)


class Attend:
    """o, lse of packed rows; per (row, head) the sum of P |v| that o's roundings are relative
    to, and per row the error of t and the largest |t|."""

    def __init__(self, q, k, v, table, lens, cu, ap, parents=None, temp=None, pos=None, qpos=None):
        N, Hq, D = q.shape
        Hkv, page = k.shape[1], k.shape[2]
        G, f8 = Hq // Hkv, dict(dtype=torch.float64)
        self.o, self.size = torch.zeros(N, Hq, D, **f8), torch.zeros(N, Hq, D, **f8)
        self.lse = torch.full((N, Hq), -math.inf, **f8)
        self.et, self.top, self.keys = torch.zeros(N, **f8), torch.zeros(N, **f8), torch.zeros(N, **f8)
        self.rows = torch.zeros(N, dtype=torch.bool)
        for b, L in enumerate(lens):
            n = cu[b + 1] - cu[b]
            if n == 0:
                continue
            r = slice(cu[b], cu[b + 1])
            self.rows[r] = True
            pages = table[b, :-(-L // page)].long()
            kb, vb = (x[pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].double() for x in (k, v))
            up = None if parents is None else parents[r].tolist()
            live = live_of(n, L, ap.window_len, up, None if pos is None else pos[b], None if pos is None else int(qpos[b]))
            for h in range(Hq):
                g = h // G
                on = live[g if live.shape[0] > 1 else 0]
                s = q[r, h].double() @ torch.nan_to_num(kb[g]).T * ap.sm_scale
                s = torch.where(on, s, 0.0)
                tb = torch.ones(n, 1, **f8) if temp is None else temp[r, None].double()
                t = cap64(s, ap.cap_method, ap.cap, ap.alpha, ap.beta) * tb
                dots = torch.where(on, q[r, h].double().abs() @ torch.nan_to_num(kb[g]).abs().T, 0.0)
                et = tb[:, 0].abs() * EPS32 * 1.5 * ((D + 8) * abs(ap.sm_scale) * dots.amax(1) + 16 * s.abs().amax(1))
                self.et[r] = torch.maximum(self.et[r], et)
                self.top[r] = torch.maximum(self.top[r], t.abs().amax(1))
                self.keys[r] = on.sum(1).double()
                t = t.masked_fill(~on, -math.inf)
                norm = torch.logsumexp(t, -1)
                p = torch.where(on, torch.exp(t - torch.where(torch.isinf(norm), 0.0, norm)[:, None]), 0.0)
                self.o[r, h] = p @ torch.nan_to_num(vb[g])
                self.size[r, h] = p @ torch.nan_to_num(vb[g]).abs()
                self.lse[r, h] = norm


def check(got, want, dtype):
    """t is off by at most et, so each P by 2 et relative (its own t and the sum's); an
    exponential adds 1.5 half steps of its argument, which is at most twice the largest |t|
    and 8 (its own and a rescaling's), and 8 steps of its own; sums of n terms in any order
    round by n half steps.  bf16: P enters the tensor cores rounded, by at most half a step
    of its type."""
    o, lse = got[0].double().cpu()[want.rows], got[1].double().cpu()[want.rows]
    o64, lse64, size = want.o[want.rows], want.lse[want.rows], want.size[want.rows]
    et, top, n = (x[want.rows] for x in (want.et, want.top, want.keys))
    half = torch.finfo(dtype).eps / 2
    exps = (2 * 1.5 * (2 * top + 8) + 8) * EPS32
    p_err = 2 * et + 2 * exps + (2 * n + 64) * EPS32 + (half if dtype == torch.bfloat16 else 0)
    assert torch.isfinite(o).all()
    off, bound = (o - o64).abs(), 1.0001 * half * o64.abs() + size * p_err[:, None, None]
    assert (off <= bound).all(), float((off / bound.clamp(min=1e-300)).max())
    empty = torch.isneginf(lse64)
    assert torch.equal(torch.isneginf(lse), empty)
    lse_err = (et + exps + (n + 64) * EPS32)[:, None] + 4 * EPS32 * torch.where(empty, 0.0, lse64).abs()
    off = (lse - torch.where(empty, 0.0, lse64)).abs()
    assert (off <= lse_err)[~empty].all(), float((off / lse_err)[~empty].max())


def plan(table, lens, held, free, n_free, n_new, page, rows, qpos=None):
    """The step done a sequence at a time, with lists; None where it does not fit."""
    table, free, top = [list(t) for t in table], list(free), n_free
    after = [0 if n < 0 else x + n for x, n in zip(lens, n_new)]
    need = [-(-x // page) for x in after]
    if any(n > len(t) for n, t in zip(need, table)) or sum(max(n, 0) for n in n_new) > rows:
        return None
    for b, n in enumerate(need):
        for x in range(n, held[b]):
            free[top:top + 1] = [table[b][x]]
            top += 1
    for b, n in enumerate(need):
        for x in range(held[b], n):
            top -= 1
            if top < 0:
                return None
            table[b][x] = free[top]
    cu, slots, positions = [0], [], []
    for b, n in enumerate(n_new):
        for i in range(max(n, 0)):
            s = lens[b] + i
            slots.append(table[b][s // page] * page + s % page)
            positions.append(s if qpos is None else qpos[b] + 1 + i)
        cu.append(len(slots))
    pad = [-1] * (rows - len(slots))
    q = None if qpos is None else [-1 if n < 0 else x + n for x, n in zip(qpos, n_new)]
    return dict(table=table, free=free, n_free=top, lens=after, held=need, cu=cu, slots=slots + pad,
                positions=positions + pad, qpos=q)


def walk(parents, tokens, says, width):
    """Path and next token of one sequence's rows."""
    if not parents:
        return [], -1
    path = [0]
    while len(path) < width:
        at = path[-1]
        hits = [c for c in range(at + 1, len(parents)) if parents[c] == at and tokens[c] == says[at]]
        if not hits:
            break
        path.append(hits[0])
    return path, says[path[-1]]
