"""Cases of the serving operators: a paged key-value cache, attention of one
new token over it with the soft caps, the attention weight each key of a prompt
received, and eviction by accumulated weight.

Names of a case: B sequences, Hq query and Hkv key heads, D head dim, page the
tokens of a page, lo..hi the sequences' lengths (spread evenly over that
range), L a prompt's length.  ``run`` computes an operator's plain form, or
with ``own`` makes the framework's calls; ``exact`` is the definition in 64 bits.
"""

import math

import numpy as np
import torch

own = False

_CAPS = {"none": (0.0, 0.0, 0.0), "tanh": (50.0, 0.0, 0.0), "soft_sign": (20.0, 0.0, 0.0), "alsc": (30.0, 2.0, 0.5)}
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
_LARGEST_CACHE = 540_000_000   # bytes of keys and values of the largest listed cache
_LARGEST_PAIRS = 1 << 29       # (query head, query, key) triples of the largest listed prompt


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decoding step's new keys and values of a served batch, one token a sequence
        {"name": "append_step", "op": "append", "B": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 16, "lo": 900, "hi": 4000, "new_lo": 1, "new_hi": 1},
        # packed prompts of unequal lengths entering an empty cache
        {"name": "append_prompts", "op": "append", "B": 9, "Hkv": 16, "D": 128, "dtype": "bf16", "page": 64, "lo": 128, "hi": 3969, "new_lo": 128, "new_hi": 3969},
        # a single user's chat turn: latency counts
        {"name": "decode_one", "op": "decode", "B": 1, "Hq": 16, "Hkv": 16, "D": 128, "dtype": "bf16", "page": 16, "lo": 1021, "hi": 1021, "cap": "tanh", "window": 0, "temp": False, "acc": False},
        # ranker serving: a batch of users with histories of 1024 to 3968 items
        {"name": "decode_ranker", "op": "decode", "B": 32, "Hq": 8, "Hkv": 2, "D": 128, "dtype": "bf16", "page": 64, "lo": 1024, "hi": 3968, "cap": "alsc", "window": 0, "temp": False, "acc": False},
        # a sliding-window layer of a served batch: only the window's keys count
        {"name": "decode_window", "op": "decode", "B": 64, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 32, "lo": 90, "hi": 4099, "cap": "alsc", "window": 1024, "temp": True, "acc": False},
        # one long document: the cache's length has to be split
        {"name": "decode_long", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "lo": 130977, "hi": 130977, "cap": "tanh", "window": 0, "temp": False, "acc": False},
        # a batch whose cache is pruned by weight: the step's weights are added up too
        {"name": "decode_weights", "op": "decode", "B": 16, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "lo": 2050, "hi": 8192, "cap": "soft_sign", "window": 0, "temp": False, "acc": True},
        # a small model in full precision
        {"name": "decode_fp32", "op": "decode", "B": 4, "Hq": 4, "Hkv": 2, "D": 64, "dtype": "fp32", "page": 16, "lo": 333, "hi": 2048, "cap": "none", "window": 0, "temp": False, "acc": False},
        # the weights that start a pruned cache: a batch of two prompts, one of them padded
        {"name": "weights_prompts", "op": "weights", "B": 2, "L": 2048, "Hq": 16, "Hkv": 16, "D": 128, "dtype": "bf16", "cap": "tanh", "window": 0, "temp": False, "rows_lo": 1531},
        # the same for one long prompt of a windowed grouped-query layer
        {"name": "weights_window", "op": "weights", "B": 1, "L": 4096, "Hq": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "cap": "alsc", "window": 1024, "temp": True, "rows_lo": 4096},
        # a served batch cut back to 2048 tokens a sequence
        {"name": "evict_batch", "op": "evict", "B": 16, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "lo": 2049, "hi": 4096, "budget": 2048, "first": 4, "last": 128},
        # one long document cut to an eighth
        {"name": "evict_long", "op": "evict", "B": 1, "Hkv": 8, "D": 128, "dtype": "bf16", "page": 64, "lo": 130977, "hi": 130977, "budget": 16384, "first": 4, "last": 1024},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode"] * 5 + ["evict"] * 2 + ["weights"] * 2 + ["append"] * 2)
    D, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16"] * 4 + ["fp32"])
    cap, temp = rng.choice(sorted(_CAPS)), rng.random() < 0.3
    if op == "weights":
        G, Hkv, B = rng.choice([1, 1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 8]), _log(rng, 1, 6)
        most = int(math.sqrt(_LARGEST_PAIRS / (B * Hkv * G))) // (2 if dtype == "fp32" else 1)
        L = _log(rng, 17, min(4096, most))
        return {"op": op, "B": B, "L": L, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "dtype": dtype, "cap": cap,
                "window": _log(rng, 5, L) if rng.random() < 0.3 else 0, "temp": temp, "rows_lo": rng.randint(1, L)}
    G, Hkv, page = rng.choice([1, 1, 2, 3, 4, 4, 8, 16]), rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([16, 32, 64, 128])
    B = _log(rng, 1, 96)
    most = _LARGEST_CACHE // (B * Hkv * D * 2 * (4 if dtype == "fp32" else 2))
    hi = _log(rng, 1 if op != "evict" else 64, min(131072, most))
    lo = hi if rng.random() < 0.4 else rng.randint(0, hi)
    case = {"op": op, "B": B, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page, "lo": lo, "hi": hi}
    if op == "append":
        n = rng.randint(0, lo)
        return dict(case, new_lo=min(1, lo), new_hi=min(1, lo)) if rng.random() < 0.5 else dict(case, new_lo=n, new_hi=rng.randint(n, lo))
    if op == "decode":
        return dict(case, Hq=Hkv * G, cap=cap, window=_log(rng, 5, 4096) if rng.random() < 0.3 else 0, temp=temp, acc=rng.random() < 0.3)
    budget = rng.randint(33, hi)
    return dict(case, budget=budget, first=rng.randint(0, 8), last=rng.randint(0, budget // 4))


def _spread(lo, hi, B, turn=0):
    """B lengths from hi down to lo, in an order that `turn` rotates."""
    x = [hi - (hi - lo) * i // max(1, B - 1) for i in range(B)]
    return [x[(b * 7 + turn) % B] if math.gcd(7, B) == 1 else x[(b + turn) % B] for b in range(B)]


# ---------------------------------------------------------------- inputs
def _pool(case, lens, gen):
    """A cache's pages, shuffled, and its table: every page in use belongs to one sequence."""
    page, B = case["page"], case["B"]
    max_pages = max(1, -(-max(lens) // page))
    used = [-(-n // page) for n in lens]
    order = torch.randperm(sum(used) + 3, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (sum(used) + 3, case["Hkv"], page, case["D"])
    k, v = (_normal(shape, _TYPES[case["dtype"]], gen) for _ in range(2))
    return {"k": k, "v": v, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "max_len": max_pages * page}


def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _weights(shape, gen):
    """Accumulated attention weights: heavy-tailed, and some that underflowed to zero."""
    z = torch.randn(shape, generator=gen, device="cuda")
    return torch.where(z > -1.0, torch.exp(2.0 * z), torch.zeros_like(z))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _TYPES[case["dtype"]]
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    if case["op"] == "weights":
        L, Hq = case["L"], case["Hq"]
        s = {"q": _normal((B, L, Hq, D), dtype, gen), "k": _normal((B, L, Hkv, D), dtype, gen)}
        s["temp"] = 0.5 + torch.rand(B, L, generator=gen, device="cuda") if case["temp"] else None
        s["rows"] = torch.tensor([[0, n] for n in _spread(case["rows_lo"], L, B, seed)], dtype=torch.int32, device="cuda")
        s["out"] = torch.zeros(B, Hkv, L, device="cuda")
        t = _prompt_scores(case, s).double()
        s["lse"] = torch.logsumexp(t, -1).float().reshape(B, Hq, L)
        return dict(s, case=case, ws=None)
    lens = _spread(case["lo"], case["hi"], B, seed)
    s = _pool(case, lens, gen)
    if case["op"] == "decode":
        s["q"] = _normal((B, case["Hq"], D), dtype, gen)
        s["temp"] = 0.5 + torch.rand(B, generator=gen, device="cuda") if case["temp"] else None
        s["weights"] = _weights((B, Hkv, s["max_len"]), gen) if case["acc"] else None
    elif case["op"] == "append":
        new = [min(n, m) for n, m in zip(lens, _spread(case["new_lo"], case["new_hi"], B, seed))]
        s["k_new"], s["v_new"] = (_normal((sum(new), Hkv, D), dtype, gen) for _ in range(2))
        s["cu_new"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        s["weights"] = _weights((B, Hkv, s["max_len"]), gen)
    else:
        s["weights"] = _weights((B, Hkv, s["max_len"]), gen)
        # positions of what the cache holds after earlier evictions: the newest token is at qpos
        s["pos"] = torch.arange(s["max_len"], dtype=torch.int32, device="cuda").expand(B, Hkv, -1).contiguous()
        s["qpos"] = s["lens"] - 1
        s["weights_out"], s["pos_out"] = torch.zeros_like(s["weights"]), torch.zeros_like(s["pos"])
        s["lens_out"] = torch.zeros_like(s["lens"])
    return dict(s, case=case, ws=None)


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


def _prompt_scores(case, s):
    """Masked tempered scores [B, Hkv, G, L, L] of a causal prompt."""
    B, L, Hq, Hkv, D = case["B"], case["L"], case["Hq"], case["Hkv"], case["D"]
    q = s["q"].float().reshape(B, L, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    k = s["k"].float().permute(0, 2, 3, 1).unsqueeze(2)
    t = _cap(torch.matmul(q, k) * (1.0 / math.sqrt(D)), case["cap"])
    if s["temp"] is not None:
        t = t * s["temp"][:, None, None, :, None]
    i = torch.arange(L, device="cuda")
    live = i[:, None] >= i[None, :]
    if case["window"]:
        live = live & (i[None, :] > i[:, None] - case["window"])
    return t.masked_fill(~live, float("-inf"))


def _prompt_weights(s):
    case = s["case"]
    i = torch.arange(case["L"], device="cuda")
    counted = (i[None, :] >= s["rows"][:, :1]) & (i[None, :] < s["rows"][:, 1:])
    p = torch.exp(_prompt_scores(case, s) - s["lse"].reshape(case["B"], case["Hkv"], -1, case["L"], 1))
    p = torch.where(counted[:, None, None, :, None], p, torch.zeros_like(p))
    s["out"].copy_(p.sum(dim=(2, 3)))
    return s["out"]


def _gathered(pool, table):
    """[B, Hkv, max_len, D] in fp32 of a pool [pages, Hkv, page, D]."""
    x = pool[table.clamp(min=0).long()]
    B, n, Hkv, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * page, D).float()


def _decoded(s):
    case = s["case"]
    B, Hq, Hkv, D, n = case["B"], case["Hq"], case["Hkv"], case["D"], s["max_len"]
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, D)
    t = _cap(torch.matmul(q, _gathered(s["k"], s["table"]).transpose(-1, -2)) * (1.0 / math.sqrt(D)), case["cap"])
    if s["temp"] is not None:
        t = t * s["temp"][:, None, None, None]
    j, lens = torch.arange(n, device="cuda"), s["lens"][:, None]
    live = j[None, :] < lens
    if case["window"]:
        live = live & (j[None, :] >= lens - case["window"])
    t = t.masked_fill(~live[:, None, None, :], float("-inf"))
    m = t.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(t - m)
    l = p.sum(-1, keepdim=True)
    lse = (m + torch.log(l)).reshape(B, Hq)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    o = torch.matmul(p, _gathered(s["v"], s["table"])).to(s["q"].dtype).reshape(B, Hq, D)
    if s["weights"] is None:
        return [o, lse]
    s["weights"] += p.sum(2)
    return [o, lse, s["weights"]]


def _appended(s):
    case, page = s["case"], s["case"]["page"]
    r = torch.arange(s["k_new"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu_new"][1:].long(), r, right=True)
    slot = s["lens"][b].long() - (s["cu_new"][b + 1].long() - r)
    at = s["table"][b, slot // page].long()
    s["k"][at, :, slot % page] = s["k_new"]
    s["v"][at, :, slot % page] = s["v_new"]
    s["weights"][b, :, slot] = 0.0
    return [s["k"], s["v"], s["weights"]]


def _evicted(s):
    """Keeps the `budget` heaviest tokens of each head, the first and last ones among them: a kept token
    behind the budget moves, in order, to the place of one that goes."""
    case, n, page, budget = s["case"], s["max_len"], s["case"]["page"], s["case"]["budget"]
    B, Hkv = case["B"], case["Hkv"]
    j = torch.arange(n, device="cuda")
    lens, held = s["lens"].long()[:, None, None], s["pos"]
    inside = j < lens
    safe = (held < case["first"]) | (held > s["qpos"][:, None, None] - case["last"])
    rank = torch.where(safe, torch.full_like(s["weights"], float("inf")), s["weights"])
    rank = torch.where(inside, rank, torch.full_like(rank, float("-inf")))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    keep = torch.zeros(B, Hkv, n, dtype=torch.bool, device="cuda")
    keep.scatter_(2, order[..., :min(budget, n)], True)
    keep &= inside
    hole, mover = ~keep & inside & (j < budget), keep & (j >= budget)
    src = torch.where(keep & (j < budget), j, torch.full_like(j, -1)).to(torch.int32)
    src[hole] = j.expand(B, Hkv, n)[mover].to(torch.int32)
    src = src[..., :min(budget, n)].contiguous()
    bb, hh, dst = hole.nonzero(as_tuple=True)
    old = mover.nonzero(as_tuple=True)[2]
    to, fro = s["table"][bb, dst // page].long(), s["table"][bb, old // page].long()
    s["k"][to, hh, dst % page] = s["k"][fro, hh, old % page]
    s["v"][to, hh, dst % page] = s["v"][fro, hh, old % page]
    bb, hh, dst = (src >= 0).nonzero(as_tuple=True)
    old = src[bb, hh, dst].long()
    s["weights_out"][bb, hh, dst] = s["weights"][bb, hh, old]
    s["pos_out"][bb, hh, dst] = s["pos"][bb, hh, old]
    s["lens_out"].copy_(s["lens"].clamp(max=budget))
    full = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device="cuda")
    full[..., :src.shape[-1]] = src
    return [s["k"], s["v"], s["weights_out"], s["pos_out"], s["lens_out"], full]


def run(state):
    if own:
        return _own(state)
    return {"append": _appended, "decode": _decoded, "weights": _prompt_weights, "evict": _evicted}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    from soft_capped_attention_gb300 import capattn as ca
    from soft_capped_attention_gb300 import kv_cache as kv

    case = s["case"]
    if case["op"] in ("decode", "weights"):
        cap, alpha, beta = _CAPS[case["cap"]]
        ap = ca.AttnParams(sm_scale=1.0 / math.sqrt(case["D"]), cap_method=case["cap"], cap=cap, alpha=alpha, beta=beta,
                           causal=True, window_len=case["window"])
    if case["op"] == "weights":
        if s["ws"] is None:  # kept for the state's later passes, as a program keeps it
            s["ws"] = kv.new_key_weights_workspace(s["q"], s["k"], ap)
        return kv.key_weights(s["q"], s["k"], s["lse"], ap, temp=s["temp"], rows=s["rows"], out=s["out"], workspace=s["ws"])
    if s["ws"] is None:
        s["ws"] = kv.KVCache(s["k"], s["v"], s["table"], s["lens"], weights=s.get("weights"), pos=s.get("pos"), qpos=s.get("qpos"))
    cache = s["ws"]
    if case["op"] == "append":
        one = s["k_new"].shape[0] == case["B"] and case["new_hi"] == 1
        kv.cache_append(cache, s["k_new"], s["v_new"], cu_new=None if one else s["cu_new"])
        return [s["k"], s["v"], s["weights"]]
    if case["op"] == "decode":
        o, lse = kv.cache_decode(s["q"], cache, ap, temp=s["temp"], accumulate=case["acc"])
        return [o, lse, s["weights"]] if case["acc"] else [o, lse]
    src = kv.cache_evict(cache, case["budget"], keep_first=case["first"], keep_last=case["last"], out=(s["lens_out"], s["weights_out"], s["pos_out"]))
    return [s["k"], s["v"], s["weights_out"], s["pos_out"], s["lens_out"], src]


# ---------------------------------------------------------------- cost
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    if case["op"] == "weights":
        L, Hq, W = case["L"], case["Hq"], case["window"] or case["L"]
        live = lambda n: sum(min(i + 1, W) for i in range(n))  # noqa: E731
        rows = _spread(case["rows_lo"], L, B)
        read = sum(n * Hq * (D * e + 4) + min(n, L) * Hkv * D * e for n in rows)
        return {"bytes": read + B * Hkv * L * 4, "flops": 2 * D * Hq * sum(live(n) for n in rows)}
    lens = _spread(case["lo"], case["hi"], B)
    if case["op"] == "append":
        n = sum(min(a, b) for a, b in zip(lens, _spread(case["new_lo"], case["new_hi"], B)))
        return {"bytes": max(1, n) * Hkv * (4 * D * e + 4), "flops": 0}
    if case["op"] == "decode":
        n = sum(min(x, case["window"] or x) for x in lens)
        return {"bytes": Hkv * n * (2 * D * e + (8 if case["acc"] else 0)) + 2 * B * case["Hq"] * D * e + B * case["Hq"] * 4,
                "flops": 4 * n * case["Hq"] * D}
    # eviction: every weight and position once, and the rows that move
    total = 0.0
    for n in lens:
        m = min(n, case["budget"])
        total += 8 * n + 12 * m
        if n > case["budget"]:
            behind, last = n - case["budget"], case["last"]
            kept = min(last, behind) + max(0, behind - last) * (case["budget"] - last) / max(1, n - last)
            total += kept * 4 * D * e
    return {"bytes": max(1.0, Hkv * total), "flops": 0}


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


def exact(case, seed):
    s = prepare(case, seed)
    B, Hkv, D, f8 = case["B"], case["Hkv"], case["D"], torch.float64
    if case["op"] == "weights":
        L, G, out = case["L"], case["Hq"] // case["Hkv"], torch.zeros(B, Hkv, case["L"], dtype=f8, device="cuda")
        i = torch.arange(L, device="cuda")
        for b in range(B):
            first, last = (int(x) for x in s["rows"][b])
            for h in range(case["Hq"]):
                x = _capped(s["q"][b, first:last, h].to(f8) @ s["k"][b, :, h // G].to(f8).T / math.sqrt(D), case["cap"])
                if s["temp"] is not None:
                    x = x * s["temp"][b, first:last, None].to(f8)
                gap = i[first:last, None] - i[None, :]
                dead = (gap < 0) | (gap >= (case["window"] or L + 1))
                out[b, h // G] += (torch.exp(x - s["lse"][b, h, first:last, None].to(f8)) * ~dead).sum(0)
        return out
    lens = s["lens"].tolist()
    rows = lambda pool, b, n: pool[s["table"][b, :-(-n // case["page"])].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :n]  # noqa: E731
    if case["op"] == "decode":
        G = case["Hq"] // Hkv
        o, lse = torch.zeros(B, case["Hq"], D, dtype=f8, device="cuda"), torch.full((B, case["Hq"]), -math.inf, dtype=f8, device="cuda")
        w = s["weights"].to(f8) if case["acc"] else None
        for b, n in enumerate(lens):
            at = max(0, n - case["window"]) if case["window"] else 0
            if n == 0:
                continue
            k, v = rows(s["k"], b, n)[:, at:].to(f8), rows(s["v"], b, n)[:, at:].to(f8)
            x = _capped(torch.einsum("hgd,hnd->hgn", s["q"][b].to(f8).reshape(Hkv, G, D), k) / math.sqrt(D), case["cap"])
            x = x * float(s["temp"][b]) if s["temp"] is not None else x
            norm = torch.logsumexp(x, -1)
            p = torch.exp(x - norm[..., None])
            o[b], lse[b] = torch.einsum("hgn,hnd->hgd", p, v).reshape(-1, D), norm.reshape(-1)
            if w is not None:
                w[b, :, at:n] += p.sum(1)
        return [o, lse, w] if case["acc"] else [o, lse]
    page, table = case["page"], s["table"].cpu().numpy()
    k, v, w = s["k"].to(f8), s["v"].to(f8), s["weights"].to(f8)
    if case["op"] == "append":
        cu = s["cu_new"].tolist()
        for b, n in enumerate(lens):
            new = cu[b + 1] - cu[b]
            slot = np.arange(n - new, n)
            at, off = torch.from_numpy(table[b, slot // page].astype(np.int64)).cuda(), torch.from_numpy(slot % page).cuda()
            k[at, :, off], v[at, :, off] = s["k_new"][cu[b]:cu[b + 1]].to(f8), s["v_new"][cu[b]:cu[b + 1]].to(f8)
            w[b, :, n - new:n] = 0.0
        return [k, v, w]
    heavy, kept_w = s["weights"].cpu().numpy().astype(np.float64), torch.zeros_like(w)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            if n == 0:
                continue
            a = heavy[b, h, :n].copy()
            if n > case["budget"]:
                a[:case["first"]] = np.inf
                a[n - case["last"]:] = np.inf
                chosen = np.sort(np.lexsort((np.arange(n), -a))[:case["budget"]])
                gone = np.setdiff1d(np.arange(case["budget"]), chosen)
                came = chosen[chosen >= case["budget"]]
                held = np.arange(case["budget"])
                held[gone] = came
                to, fro = table[b, gone // page].astype(np.int64), table[b, came // page].astype(np.int64)
                k[to, h, gone % page], v[to, h, gone % page] = k[fro, h, came % page], v[fro, h, came % page]
            else:
                held = np.arange(n)
            kept_w[b, h, :len(held)] = w[b, h][torch.from_numpy(held).cuda()]
    return [k, v, kept_w, None, None, None]
