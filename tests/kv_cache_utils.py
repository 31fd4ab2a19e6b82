"""Plain forms of the paged cache's calls in 64 bits, on the CPU, and the error
bounds that their tests use."""

import math

import torch

EPS32 = 2.0 ** -24          # half a step of fp32, relative
# tight caps bend most scores (the kernels' one-by-one forms), wide ones few (their
# polynomials), the one between takes both and tanh's longer polynomial
CAPS = {"none": (0.0, 0.0, 0.0), "tanh": (5.0, 0.0, 0.0), "soft_sign": (3.0, 0.0, 0.0), "alsc": (4.0, 2.0, 0.5),
        "tanh15": (15.0, 0.0, 0.0), "tanh50": (50.0, 0.0, 0.0), "alsc30": (30.0, 2.0, 0.5), "alsc90": (90.0, 2.0, 0.5)}


def method_of(cap):
    return cap.rstrip("0123456789")


def cap64(x, method, cap, alpha, beta):
    if method == "none" or cap <= 0:
        return x
    if method == "tanh":
        return cap * torch.tanh(x / cap)
    if method == "soft_sign":
        return x / (1 + x.abs() / cap)
    sb = 1 / (1 + math.exp(-alpha * beta))
    return cap * (torch.sigmoid(alpha * (x / cap + beta)) - sb) / (sb * (1 - sb) + 1e-12)


def rows64(pool, table_row, n):
    """[Hkv, n, D] of a pool [pages, Hkv, page, D]."""
    page = pool.shape[2]
    pages = table_row[:-(-n // page)].long()
    x = pool[pages].transpose(0, 1)
    return x.reshape(x.shape[0], -1, x.shape[-1])[:, :n].double()


def decode64(q, k, v, table, lens, ap, temp=None, pos=None, qpos=None):
    """o [B, Hq, D], lse [B, Hq], the weights' additions [B, Hkv, n_max] and the
    bound on an error of t, per sequence."""
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    n_max = max(1, max(lens))
    o, lse = torch.zeros(B, Hq, D, dtype=torch.float64), torch.full((B, Hq), -math.inf, dtype=torch.float64)
    add, et = torch.zeros(B, Hkv, n_max, dtype=torch.float64), torch.zeros(B, dtype=torch.float64)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        kb, vb = rows64(k, table[b], n), rows64(v, table[b], n)
        qb = q[b].double().reshape(Hkv, G, D)
        at = pos[b, :, :n].double() if pos is not None else torch.arange(n).double().expand(Hkv, n)
        newest = float(qpos[b]) if pos is not None else n - 1
        live = torch.ones(Hkv, n, dtype=torch.bool)
        if ap.window_len > 0:
            live = at > newest - ap.window_len
        s = torch.einsum("hgd,hnd->hgn", qb, torch.where(live[..., None], kb, 0.0)) * ap.sm_scale
        t = cap64(s, ap.cap_method, ap.cap, ap.alpha, ap.beta)
        tb = 1.0 if temp is None else float(temp[b])
        t = (t * tb).masked_fill(~live[:, None], -math.inf)
        some = live.any(-1)
        norm = torch.logsumexp(t, -1)
        p = torch.where(some[:, None, None], torch.exp(t - torch.where(torch.isinf(norm), 0.0, norm)[..., None]), 0.0)
        o[b] = torch.einsum("hgn,hnd->hgd", p, torch.where(live[..., None], vb, 0.0)).reshape(Hq, D)
        lse[b] = norm.reshape(-1)
        add[b, :, :n] = p.sum(1)
        # t: a dot product of D terms in fp32 (any order), the scale, the cap (a few
        # roundings of its value, or of its argument, whose slope is at most 1, alsc's
        # at most 1 / (4 sb (1 - sb))) and the temperature
        dots = (qb.abs()[:, :, None] * torch.where(live[..., None], kb, 0.0).abs()[:, None]).sum(-1).max()
        et[b] = abs(tb) * EPS32 * 1.5 * ((D + 8) * abs(ap.sm_scale) * dots + 16 * s.abs().max())
    return o, lse, add, et


def key_weights64(q, k, lse, ap, live, temp=None, rows=None):
    """w [B, Hkv, Lk] and the bound on an error of t; live [B, L, Lk] bool."""
    B, L, Hq, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    qd, kd = q.double().permute(0, 2, 1, 3).reshape(B, Hkv, G, L, D), k.double().permute(0, 2, 1, 3)
    s = torch.einsum("bhgid,bhjd->bhgij", qd, kd) * ap.sm_scale
    t = cap64(s, ap.cap_method, ap.cap, ap.alpha, ap.beta)
    if temp is not None:
        t = t * temp.double()[:, None, None, :, None]
    use = live.clone()
    if rows is not None:
        i = torch.arange(L)
        use &= ((i >= rows[:, :1]) & (i < rows[:, 1:]))[:, :, None]
    use = use[:, None, None].expand_as(t)
    n = lse.double().reshape(B, Hkv, G, L, 1)
    p = torch.where(use, torch.exp(torch.where(use, t - n, 0.0)), 0.0)
    dots = torch.einsum("bhgid,bhjd->bhgij", qd.abs(), kd.abs()).max()
    top = 1.0 if temp is None else float(temp.abs().max())
    return p.sum((2, 3)), top * EPS32 * 1.5 * ((D + 8) * abs(ap.sm_scale) * dots + 16 * s.abs().max())


def evict_row(w, pos, newest, n, budget, first, last):
    """The slots that one (sequence, head) keeps, by the rule itself: returns src,
    a list of the old slot of every new one."""
    if n <= budget:
        return list(range(n))
    def rank(j):
        at = pos[j] if pos is not None else j
        if at < first or at > newest - last:
            return (-2, 0.0, j)
        x = float(w[j])
        return (1, 0.0, j) if math.isnan(x) else (0, -x, j)
    kept = set(sorted(range(n), key=rank)[:budget])
    src = list(range(budget))
    freed = [j for j in range(budget) if j not in kept]
    for hole, mover in zip(freed, sorted(j for j in kept if j >= budget)):
        src[hole] = mover
    return src


def live_mask(B, L, Lk, causal, window, seg=None, bounds=None):
    i, j = torch.arange(L)[:, None], torch.arange(Lk)[None, :]
    live = torch.ones(B, L, Lk, dtype=torch.bool)
    if causal:
        live &= i >= j
    if window:
        live &= j > i - window
    if seg is not None:
        live &= seg[:, :, None] == seg[:, None, :]
    if bounds is not None:
        for b in range(B):
            hl, hu, cl, cu = (int(x) for x in bounds[b])
            in_h = lambda x: (x >= hl) & (x < hu)  # noqa: E731
            in_c = lambda x: (x >= cl) & (x < cu)  # noqa: E731
            live[b] &= (in_h(j) & (in_h(i) | in_c(i))) | (in_c(i) & (i == j))
    return live


class Pool:
    """A cache on the CPU: shuffled pages, NaN wherever no token is, -1 in unused table entries."""

    def __init__(self, lens, Hkv, D, page, dtype, seed, max_len=None, spare=2):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.lens, self.page = list(lens), page
        self.max_pages = max(1, -(-max(max(lens), max_len or 0) // page))
        used = [-(-n // page) for n in lens]
        order = torch.randperm(sum(used) + spare, generator=g).to(torch.int32)
        self.table = torch.full((B, self.max_pages), -1, dtype=torch.int32)
        shape = (sum(used) + spare, Hkv, page, D)
        self.k, self.v = torch.full(shape, math.nan, dtype=dtype), torch.full(shape, math.nan, dtype=dtype)
        at = 0
        for b, n in enumerate(lens):
            pages = order[at:at + used[b]]
            self.table[b, :used[b]] = pages
            at += used[b]
            for x in (self.k, self.v):
                rows = torch.full((used[b] * page, Hkv, D), math.nan)
                rows[:n] = torch.randn(n, Hkv, D, generator=g)
                x[pages.long()] = rows.reshape(used[b], page, Hkv, D).transpose(1, 2).to(dtype)
        self.gen = g

    def cuda(self, **kw):
        from soft_capped_attention_gb300 import kv_cache as kv
        d = lambda x: None if x is None else x.cuda()  # noqa: E731
        return kv.KVCache(self.k.cuda(), self.v.cuda(), self.table.cuda(),
                          torch.tensor(self.lens, dtype=torch.int32).cuda(), **{n: d(x) for n, x in kw.items()})
