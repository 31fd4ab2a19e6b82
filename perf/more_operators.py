"""Cases of the serving operators for many new tokens per sequence over the paged
cache: attention of packed prompts or chunks of prompts, attention of trees of
drafted tokens, the tables and slot maps of a step built from request lengths, and
the acceptance of a drafted path.

Names of a case: B sequences, Hq query and Hkv key heads, D head dim, page the tokens
of a page, lo..hi the sequences' lengths with their new tokens (spread evenly over
that range), new_lo..new_hi their new or drafted tokens.  ``run`` computes an
operator's plain form, or with ``own`` makes the framework's calls; ``exact`` is the
definition in 64 bits.
"""

import math

import torch

own = False

_CAPS = {"none": (0.0, 0.0, 0.0), "tanh": (50.0, 0.0, 0.0), "soft_sign": (20.0, 0.0, 0.0), "alsc": (30.0, 2.0, 0.5)}
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_LARGEST_CACHE = 540_000_000         # bytes of keys and values of the largest listed cache
_LARGEST_SCORES = 32 * 4096 * 16384  # (query head, new token, key) triples of the largest listed prompt, padded
_LARGEST_FP32 = 1 << 27              # the same in full precision


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # a chat's next turn behind what its cache holds: latency counts
        {"name": "prompt_turn", "op": "prompt", "B": 1, "Hq": 16, "Hkv": 16, "D": 128, "dtype": "bf16", "page": 16, "lo": 1114, "hi": 1114, "new_lo": 93, "new_hi": 93, "cap": "tanh", "window": 0, "temp": False},
        # prompts of unequal lengths, packed, entering an empty cache
        {"name": "prompt_packed", "op": "prompt", "B": 9, "Hq": 16, "Hkv": 16, "D": 128, "dtype": "bf16", "page": 64, "lo": 128, "hi": 3969, "new_lo": 128, "new_hi": 3969, "cap": "soft_sign", "window": 0, "temp": False},
        # a sliding-window layer of four long prompts, grouped heads, a temperature a token
        {"name": "prompt_window", "op": "prompt", "B": 4, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 32, "lo": 4096, "hi": 4096, "new_lo": 4096, "new_hi": 4096, "cap": "alsc", "window": 1024, "temp": True},
        # the last chunk of a long document that is read in pieces
        {"name": "prompt_chunk", "op": "prompt", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "lo": 16384, "hi": 16384, "new_lo": 4096, "new_hi": 4096, "cap": "tanh", "window": 0, "temp": False},
        # a small model in full precision
        {"name": "prompt_fp32", "op": "prompt", "B": 4, "Hq": 4, "Hkv": 2, "D": 64, "dtype": "fp32", "page": 16, "lo": 333, "hi": 1021, "new_lo": 61, "new_hi": 333, "cap": "none", "window": 0, "temp": False},
        # one user's tree of drafted tokens: latency counts
        {"name": "tree_one", "op": "tree", "B": 1, "Hq": 16, "Hkv": 16, "D": 128, "dtype": "bf16", "page": 16, "lo": 1045, "hi": 1045, "new_lo": 24, "new_hi": 24, "cap": "tanh", "window": 0, "temp": False},
        # a served batch, a small tree a sequence
        {"name": "tree_batch", "op": "tree", "B": 32, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "lo": 916, "hi": 4016, "new_lo": 16, "new_hi": 16, "cap": "alsc", "window": 0, "temp": False},
        # one long document: the cache's length has to be split
        {"name": "tree_long", "op": "tree", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "lo": 131009, "hi": 131009, "new_lo": 32, "new_hi": 32, "cap": "tanh", "window": 0, "temp": False},
        # a decoding step of a served batch, one token a sequence
        {"name": "plan_step", "op": "plan", "B": 64, "page": 16, "lo": 900, "hi": 4000, "new_lo": 1, "new_hi": 1, "ends": 0},
        # a step that mixes prompts, running sequences and ended ones
        {"name": "plan_mixed", "op": "plan", "B": 512, "page": 64, "lo": 0, "hi": 4096, "new_lo": 1, "new_hi": 257, "ends": 40},
        # one user: three drafted continuations, one of them right for some tokens
        {"name": "accept_one", "op": "accept", "B": 1, "Hkv": 16, "D": 128, "dtype": "bf16", "page": 16, "lo": 1046, "hi": 1046, "chains": 3, "chain": 8},
        # a served batch, four continuations a sequence
        {"name": "accept_batch", "op": "accept", "B": 128, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "lo": 933, "hi": 4033, "chains": 4, "chain": 8},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt"] * 4 + ["tree"] * 4 + ["plan"] * 2 + ["accept"] * 2)
    D, dtype, page = rng.choice([64, 128, 128]), rng.choice(["bf16"] * 4 + ["fp32"]), rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 512)
        hi = _log(rng, 1, 4096)
        new_hi = rng.choice([1, _log(rng, 1, 257)])
        return {"op": op, "B": B, "page": page, "lo": rng.randint(0, hi), "hi": hi, "new_lo": rng.randint(0, 1), "new_hi": new_hi, "ends": rng.randint(0, B // 3)}
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "accept":
        chains, chain = rng.randint(1, 5), rng.randint(1, 9)
        n = chains * chain + 1
        B = _log(rng, 1, 128)
        most = _LARGEST_CACHE // (B * Hkv * D * 2 * (4 if dtype == "fp32" else 2))
        hi = _log(rng, n, max(n, min(4096, most)))
        return {"op": op, "B": B, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page, "lo": rng.randint(n, hi), "hi": hi, "chains": chains, "chain": chain}
    G, cap, temp = rng.choice([1, 1, 2, 3, 4, 4, 5, 8, 16]), rng.choice(sorted(_CAPS)), rng.random() < 0.3
    B = _log(rng, 1, 48)
    scores = (_LARGEST_FP32 if dtype == "fp32" else _LARGEST_SCORES) // (B * Hkv * G)
    held = _LARGEST_CACHE // (B * Hkv * D * 2 * (4 if dtype == "fp32" else 2))
    if op == "tree":
        new_hi = _log(rng, 1, 64)
        hi = _log(rng, new_hi, max(new_hi, min(131072, held, scores // new_hi)))
        new_lo = new_hi if rng.random() < 0.5 else rng.randint(0, new_hi)
    else:
        hi = _log(rng, 2, min(16384, held, int(math.sqrt(scores)) * 2))
        new_hi = min(hi, max(1, scores // hi), _log(rng, 1, hi))
        new_lo = new_hi if rng.random() < 0.4 else rng.randint(0, new_hi)
    lo = hi if rng.random() < 0.4 else rng.randint(new_lo, hi)
    return {"op": op, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi,
            "cap": cap, "window": _log(rng, 5, 4096) if rng.random() < 0.3 else 0, "temp": temp}


def _spread(lo, hi, B, turn=0):
    """B numbers from hi down to lo, in an order that `turn` rotates."""
    x = [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]
    return [x[(b * 7 + turn) % B] if math.gcd(7, B) == 1 else x[(b + turn) % B] for b in range(B)]


def _lengths(case, turn=0):
    """Lengths with the new tokens, and the new tokens."""
    lens = _spread(case["lo"], case["hi"], case["B"], turn)
    if case["op"] == "accept":
        return lens, [case["chains"] * case["chain"] + 1] * case["B"]
    return lens, [min(n, x) for n, x in zip(lens, _spread(case["new_lo"], case["new_hi"], case["B"], turn))]


# ---------------------------------------------------------------- inputs
def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _sums(new):
    return _ints([0] + torch.tensor(new).cumsum(0).tolist())


def _tables(used, max_pages, spare, gen):
    """A table of shuffled pages, `used` of each sequence, and the pages that are left."""
    order = torch.randperm(sum(used) + spare, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(used), max_pages), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(max_pages, device="cuda") < _ints(used)[:, None]
    table[held] = order[:sum(used)]
    return table, order[sum(used):]


def _prepare_plan(case, seed, gen):
    """Sequences of `lens` tokens with the pages that hold them (some one more than they need, as after an
    eviction) and a stack of free pages; the step adds n_new tokens, -1 ends a sequence."""
    B, page = case["B"], case["page"]
    lens, _ = _lengths(case, seed)
    new = _spread(case["new_lo"], case["new_hi"], B, seed + 3)
    new = [-1 if (b * 5 + seed) % B < case["ends"] and math.gcd(5, B) == 1 else n for b, n in enumerate(new)]
    used = [-(-n // page) + (1 if (b + seed) % 7 == 0 else 0) for b, n in enumerate(lens)]
    most = _spread(case["new_lo"], case["new_hi"], B)
    max_pages = max(1, -(-(max(lens) + max(most)) // page) + 1)
    # room for every sequence's tokens, whichever end; a step's buffers have a fixed size
    num_pages = sum(-(-n // page) + 1 for n in lens) + sum(-(-n // page) + 1 for n in most) + 5
    rows = -(-max(1, sum(most)) // 64) * 64
    table, left = _tables(used, max_pages, num_pages - sum(used), gen)
    free = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    free[:left.numel()] = left
    return {"table": table, "lens": _ints(lens), "n_new": _ints(new), "held": _ints(used), "free": free, "n_free": _ints([left.numel()]),
            "rows": rows, "lens_out": _ints([0] * B), "held_out": _ints([0] * B), "n_free_out": _ints([0]),
            "k": torch.zeros(num_pages, 1, page, 64, dtype=torch.bfloat16, device="cuda"), "case": case, "ws": None}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "plan":
        return _prepare_plan(case, seed, gen)
    dtype = _TYPES[case["dtype"]]
    B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
    lens, new = _lengths(case, seed)
    max_pages = max(1, -(-max(lens) // page))
    table, _ = _tables([-(-n // page) for n in lens], max_pages, 3, gen)
    shape = (sum(-(-n // page) for n in lens) + 3, Hkv, page, D)
    k, v = (_normal(shape, dtype, gen) for _ in range(2))
    s = {"k": k, "v": v, "table": table, "lens": _ints(lens), "cu_new": _sums(new), "most": max(1, max(new)), "case": case, "ws": None}
    N = sum(new)
    if case["op"] == "accept":
        # continuations of `chain` tokens behind the last sure token (row 0); what the model says agrees with
        # one of them for a while
        chains, chain, n = case["chains"], case["chain"], new[0]
        i = torch.arange(n, device="cuda")
        parents = torch.where((i - 1) % chain == 0, 0, i - 1).to(torch.int32)
        parents[0] = -1
        tokens = torch.randint(0, 32000, (B, n), generator=gen, device="cuda", dtype=torch.int32)
        says = torch.randint(32000, 64000, (B, n), generator=gen, device="cuda", dtype=torch.int32)
        right = torch.randint(0, chains, (B, 1), generator=gen, device="cuda")
        good = torch.randint(0, chain + 1, (B, 1), generator=gen, device="cuda")
        step = torch.arange(chain, device="cuda")
        at, to = torch.where(step == 0, 0, right * chain + step), right * chain + 1 + step
        says.scatter_(1, at, torch.where(step < good, tokens.gather(1, to), says.gather(1, at)))
        return dict(s, parents=parents.repeat(B), tokens=tokens.reshape(-1), says=says.reshape(-1), lens_out=torch.zeros_like(s["lens"]))
    s["q"] = _normal((N, case["Hq"], D), dtype, gen)
    s["temp"] = 0.5 + torch.rand(N, generator=gen, device="cuda") if case["temp"] else None
    s["parents"] = None
    if case["op"] == "tree":  # each drafted token continues an earlier one, the first of a sequence what the cache holds
        i = torch.arange(N, device="cuda") - s["cu_new"][:-1].long().repeat_interleave(torch.tensor(new, device="cuda"))
        u = torch.rand(N, generator=gen, device="cuda")
        s["parents"] = torch.where(i > 0, torch.minimum((u * i).floor().long(), i - 1), -1).to(torch.int32)
    return s


# ---------------------------------------------------------------- plain forms
def _cap(s, method):
    cap, alpha, beta = _CAPS[method]
    if method == "tanh":
        return cap * torch.tanh(s / cap)
    if method == "soft_sign":
        return s / (1.0 + s.abs() / cap)
    if method == "alsc":  # a difference of two sigmoids that are close together: in 64 bits
        base = 1.0 / (1.0 + math.exp(-alpha * beta))
        x = torch.sigmoid(alpha * (s.double() / cap + beta)) - base
        return (cap * x / (base * (1.0 - base) + 1e-12)).to(s.dtype)
    return s


def _gathered(pool, table):
    """[B, Hkv, max_len, D] in fp32 of a pool [pages, Hkv, page, D]."""
    x = pool[table.clamp(min=0).long()]
    B, n, Hkv, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * page, D).float()


def _padded(x, s, fill):
    """[B, most, ...] of packed rows."""
    i = torch.arange(s["most"], device="cuda")
    at = s["cu_new"][:-1, None].long() + i
    inside = at < s["cu_new"][1:, None]
    y = x[torch.where(inside, at, 0)]
    return torch.where(inside.reshape(inside.shape + (1,) * (y.dim() - 2)), y, torch.full_like(y, fill)), inside, at


def _ancestors(s):
    """[B, most, most]: whether column j is row i or one of its ancestors; and the depth of each."""
    up, inside, _ = _padded(s["parents"], s, -1)
    i = torch.arange(s["most"], device="cuda")
    seen = (i[:, None] == i).expand(up.shape[0], -1, -1)
    link = (up[..., None] == i).float()
    for _ in range(max(1, (s["most"] - 1).bit_length())):  # reached in 1, 2, 4, ... steps
        seen = seen | (torch.matmul(link, seen.float()) > 0)
        link = torch.matmul(link, link)
    return seen, seen.sum(-1) - 1


def _attended(s):
    case = s["case"]
    B, Hq, Hkv, D, n = case["B"], case["Hq"], case["Hkv"], case["D"], s["most"]
    q, inside, at = _padded(s["q"], s, 0.0)
    k, v = _gathered(s["k"], s["table"]), _gathered(s["v"], s["table"])
    L, G = k.shape[2], Hq // Hkv
    i, j = torch.arange(n, device="cuda"), torch.arange(L, device="cuda")
    base = (s["lens"] - (s["cu_new"][1:] - s["cu_new"][:-1])).long()[:, None]
    if s["parents"] is None:
        place = base + i
        live = j <= place[..., None]
    else:
        kin, depth = _ancestors(s)
        place = base + depth
        own_column = (j - base).clamp(0, n - 1)
        live = torch.where((j < base)[:, None], True, (j < base + n)[:, None] & kin.gather(2, own_column[:, None].expand(-1, n, -1)))
        held = torch.where(j < base, j, base + depth.gather(1, own_column))
    if case["window"]:
        live = live & ((j if s["parents"] is None else held[:, None]) > place[..., None] - case["window"])
    q = q.float().reshape(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    t = _cap(torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D)), case["cap"]).reshape(B, Hkv, G, n, L)
    if s["temp"] is not None:
        t = t * _padded(s["temp"], s, 1.0)[0][:, None, None, :, None]
    t = t.masked_fill_(~live[:, None, None], float("-inf"))
    m = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, G * n, L), v).reshape(B, Hkv, G, n, D) / l
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[inside].to(s["q"].dtype)
    lse = (m + torch.log(l)).permute(0, 3, 1, 2, 4).reshape(B, n, Hq)[inside]
    return [o, lse]


def _planned(s):
    page, table = s["case"]["page"], s["table"]
    add = s["n_new"].clamp(min=0)
    lens = torch.where(s["n_new"] < 0, 0, s["lens"] + add)
    need, held, p = ((lens + page - 1) // page)[:, None], s["held"][:, None], torch.arange(table.shape[1], device="cuda")
    back, fresh = (p >= need) & (p < held), (p >= held) & (p < need)
    order = lambda x: x.reshape(-1).long().cumsum(0).reshape(x.shape) - 1  # noqa: E731
    top = s["n_free"] + back.sum()
    room = s["free"].numel()
    free = torch.cat([s["free"], s["free"][:1]])
    free.scatter_(0, torch.where(back, s["n_free"] + order(back), room).reshape(-1), table.reshape(-1))
    s["free"].copy_(free[:room])
    table.copy_(torch.where(fresh, s["free"][(top - 1 - order(fresh)).clamp(0, room - 1)], table))
    s["lens_out"].copy_(lens)
    s["held_out"].copy_(need[:, 0])
    s["n_free_out"].copy_(top - fresh.sum())
    cu = torch.cat([torch.zeros_like(add[:1]), add.cumsum(0).to(torch.int32)])
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(cu[1:].long(), r, right=True)
    some = b < add.numel()
    b = b.clamp(max=add.numel() - 1)
    slot = torch.where(some, lens[b] - (cu[b + 1] - r), 0)
    place = table[b, slot // page].long() * page + slot % page
    slots, positions = torch.where(some, place, -1), torch.where(some, slot, -1).to(torch.int32)
    return [cu, slots, positions, s["lens_out"], s["held_out"], s["n_free_out"], table, s["free"]]


def _accepted(s):
    case, page, width = s["case"], s["case"]["page"], s["case"]["chain"] + 1
    (up, _, _), (tokens, _, _), (says, _, _) = (_padded(s[x], s, -2) for x in ("parents", "tokens", "says"))
    B = up.shape[0]
    node = torch.zeros(B, 1, dtype=torch.long, device="cuda")
    alive = torch.ones(B, 1, dtype=torch.bool, device="cuda")
    path = [node]
    last = node
    for _ in range(width - 1):  # the first continuation that holds what the model says
        hit = (up == last) & (tokens == says.gather(1, last))
        alive = alive & hit.any(1, keepdim=True)
        last = torch.where(alive, hit.int().argmax(1, keepdim=True), last)
        path.append(torch.where(alive, last, -1))
    path = torch.cat(path, 1)
    count = (path >= 0).sum(1)
    b = torch.arange(B, device="cuda")[:, None]
    base = (s["lens"] - (s["cu_new"][1:] - s["cu_new"][:-1])).long()[:, None]
    to = base + torch.arange(width, device="cuda")
    fro = torch.where(path >= 0, base + path, to)
    pt, pf = s["table"][b, to // page].long(), s["table"][b, fro // page].long()
    s["k"][pt, :, to % page] = s["k"][pf, :, fro % page]
    s["v"][pt, :, to % page] = s["v"][pf, :, fro % page]
    s["lens_out"].copy_(base[:, 0] + count)
    return [s["k"], s["v"], path.to(torch.int32), count.to(torch.int32), says.gather(1, last)[:, 0], s["lens_out"]]


def run(state):
    if own:
        return _own(state)
    return {"prompt": _attended, "tree": _attended, "plan": _planned, "accept": _accepted}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from soft_capped_attention_gb300 import capattn as ca
    from soft_capped_attention_gb300 import kv_cache as kv
    from soft_capped_attention_gb300 import paged

    case = s["case"]
    if s["ws"] is None:  # kept for the state's later passes, as a program keeps it
        cache = kv.KVCache(s["k"], s.get("v", s["k"]), s["table"], s["lens"])
        s["ws"] = (cache, paged.PagePool(s["free"], s["n_free"], s["held"])) if case["op"] == "plan" else (cache,)
    cache = s["ws"][0]
    if case["op"] == "plan":
        cu, slots, positions = paged.cache_plan(cache, s["ws"][1], s["n_new"], s["rows"], out=(s["lens_out"], None, s["held_out"], s["n_free_out"]))
        return [cu, slots, positions, s["lens_out"], s["held_out"], s["n_free_out"], s["table"], s["free"]]
    if case["op"] == "accept":
        path, count, says = paged.cache_verify(cache, s["cu_new"], s["tokens"], s["says"], s["parents"], case["chain"] + 1, out=(s["lens_out"], None))
        return [s["k"], s["v"], path, count, says, s["lens_out"]]
    cap, alpha, beta = _CAPS[case["cap"]]
    ap = ca.AttnParams(sm_scale=1.0 / math.sqrt(case["D"]), cap_method=case["cap"], cap=cap, alpha=alpha, beta=beta, causal=True, window_len=case["window"])
    return list(paged.cache_attend(s["q"], cache, ap, s["cu_new"], parents=s["parents"], temp=s["temp"]))


# ---------------------------------------------------------------- cost
def work(case):
    lens, new = _lengths(case)
    B = case["B"]
    if case["op"] == "plan":
        page = case["page"]
        rows = sum(_spread(case["new_lo"], case["new_hi"], B))
        return {"bytes": 32 * B + 12 * rows + 8 * (rows // page + 1), "flops": 0}
    e = 4 if case["dtype"] == "fp32" else 2
    Hkv, D = case["Hkv"], case["D"]
    N = sum(new)
    if case["op"] == "accept":  # half of the paths lie elsewhere than they go, half of each is right
        moved = B * (1 - 1 / case["chains"]) * case["chain"] / 2
        return {"bytes": max(1.0, 12 * N + moved * Hkv * 4 * D * e), "flops": 0}
    W, Hq = case["window"] or 1 << 30, case["Hq"]
    below = lambda x, n: n * x + n * (n + 1) // 2  # noqa: E731  pairs of n tokens behind x cached ones
    if case["op"] == "prompt":
        pairs = sum(below(L - n, n) - (below(L - n - W, n) if L - n >= W else max(0, L - W) * (max(0, L - W) + 1) // 2) for L, n in zip(lens, new))
    else:
        pairs = sum(n * (min(L - n, W - 1) + 1) for L, n in zip(lens, new))
    keys = sum(min(L, n + W - 1) for L, n in zip(lens, new) if n)
    return {"bytes": max(1, Hkv * keys * 2 * D * e + N * Hq * (2 * D * e + 4)), "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- the definition in 64 bits
def _capped(x, method):
    c, a, b = _CAPS[method]
    if method == "none":
        return x
    if method == "tanh":
        e = torch.exp(-2.0 * x.abs() / c)
        return torch.sign(x) * c * (1.0 - e) / (1.0 + e)
    if method == "soft_sign":
        return c * x / (c + x.abs())
    s0 = 1.0 / (1.0 + math.exp(-a * b))
    return c / (s0 * (1.0 - s0) + 1e-12) * (1.0 / (1.0 + torch.exp(-(a * x / c + a * b))) - s0)


def _exact_plan(s):
    """The step done a sequence at a time, with lists."""
    page = s["case"]["page"]
    table, lens, held, free = s["table"].tolist(), s["lens"].tolist(), s["held"].tolist(), s["free"].tolist()
    top, cu, slots, positions = int(s["n_free"]), [0], [], []
    after = [0 if n < 0 else x + n for x, n in zip(lens, s["n_new"].tolist())]
    need = [-(-x // page) for x in after]
    for b, n in enumerate(need):
        for x in range(n, held[b]):
            free[top], top = table[b][x], top + 1
    for b, n in enumerate(need):
        for x in range(held[b], n):
            top -= 1
            table[b][x] = free[top]
    for b, n in enumerate(s["n_new"].tolist()):
        for slot in range(after[b] - max(n, 0), after[b]):
            slots.append(table[b][slot // page] * page + slot % page)
            positions.append(slot)
        cu.append(len(slots))
    pad = [-1] * (s["rows"] - len(slots))
    return [_ints(cu), torch.tensor(slots + pad, device="cuda"), _ints(positions + pad), _ints(after), _ints(need), _ints([top]), _ints(table), _ints(free)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    Hkv, D, page, f8 = case["Hkv"], case["D"], case["page"], torch.float64
    lens, cu = s["lens"].tolist(), s["cu_new"].tolist()
    if case["op"] == "accept":
        k, v = s["k"].to(f8), s["v"].to(f8)
        up, tokens, says = (s[x].tolist() for x in ("parents", "tokens", "says"))
        for b, n in enumerate(lens):
            first, count = cu[b], cu[b + 1] - cu[b]
            at, path = 0, [0]
            while len(path) <= case["chain"]:
                nxt = [c for c in range(at + 1, count) if up[first + c] == at and tokens[first + c] == says[first + at]]
                if not nxt:
                    break
                at = nxt[0]
                path.append(at)
            for to, fro in enumerate(path):
                to, fro = n - count + to, n - count + fro
                pt, pf = int(s["table"][b, to // page]), int(s["table"][b, fro // page])
                for x, y in ((k, s["k"]), (v, s["v"])):
                    x[pt, :, to % page] = y[pf, :, fro % page].to(f8)
        return [k, v, None, None, None, None]
    N, Hq, G, W = s["q"].shape[0], case["Hq"], case["Hq"] // Hkv, case["window"] or 1 << 30
    o, lse = torch.zeros(N, Hq, D, dtype=f8, device="cuda"), torch.zeros(N, Hq, dtype=f8, device="cuda")
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        rows, base = slice(cu[b], cu[b + 1]), L - n
        key = torch.arange(L, device="cuda")
        live = key[None, :] <= base + torch.arange(n, device="cuda")[:, None]
        place, at = key[base:], key
        if s["parents"] is not None:
            up = s["parents"][rows].tolist()
            kin, depth = [], []
            for i in range(n):
                kin.append((kin[up[i]] if up[i] >= 0 else []) + [i])
                depth.append(len(kin[i]) - 1)
            live = (key < base).expand(n, L).clone()
            for i in range(n):
                live[i, [base + x for x in kin[i]]] = True
            place = base + torch.tensor(depth, device="cuda")
            at = torch.cat([key[:base], place])
        live = live & (at[None, :] > place[:, None] - W)
        pages = s["table"][b, :-(-L // page)].long()
        keys, values = (x[pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].to(f8) for x in (s["k"], s["v"]))
        for h in range(Hq):
            x = _capped(s["q"][rows, h].to(f8) @ keys[h // G].T / math.sqrt(D), case["cap"])
            if s["temp"] is not None:
                x = x * s["temp"][rows, None].to(f8)
            x = x.masked_fill(~live, -math.inf)
            lse[rows, h] = torch.logsumexp(x, -1)
            o[rows, h] = torch.exp(x - lse[rows, h, None]) @ values[h // G]
    return [o, lse]
