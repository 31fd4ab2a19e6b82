"""The split of a decode over its CTAs (csrc/cache_sched.cuh), restated on the CPU: which
pieces each CTA has for given lengths."""

GROUP_COST, WHOLE_TILES, SMS = 1, 4, 152


def decode_ctas(lens, Hq, Hkv, D, dtype_bytes, max_len):
    """(keys of a tile, CTAs launched) of the fp32 kernel (4 bytes) or the bf16 one (2)."""
    G = Hq // Hkv
    VH = Hkv * -(-G // 16)
    tk = 32 if dtype_bytes == 4 else 8192 // D
    per_sm = 2
    if dtype_bytes == 4:
        heads = 1 if G <= 1 else 4 if G <= 4 else 16
        smem = 4 * (4 * 32 * (D + 4) + heads * (D + 32 + 3) + (heads if D == 64 else 1) * 64 + 33)
        per_sm = min(3, 227 * 1024 // (-(-smem // 16) * 16 + 1024))
    return tk, min(len(lens) * VH * -(-max_len // tk), SMS * per_sm)


def pieces(lens, Hq, Hkv, D, dtype_bytes, max_len, window=0):
    """(CTA, sequence, group, first tile, tiles, whole) of every piece, a CTA's in order."""
    tk, grid = decode_ctas(lens, Hq, Hkv, D, dtype_bytes, max_len)
    VH = Hkv * -(-(Hq // Hkv) // 16)
    first = [max(0, n - window) // tk if window else 0 for n in lens]
    tiles = [-(-n // tk) - f for n, f in zip(lens, first)]
    groups = max(tiles) <= (2 if 2 * len(lens) * VH >= grid else 1) * WHOLE_TILES
    unit = [1 if groups else t + GROUP_COST for t in tiles]
    units = sum(unit) * VH
    ctas = min(grid, max(1, units // (1 if groups else 2)))
    q, more = divmod(units, ctas)
    begin = [q * c + min(c, more) for c in range(ctas)] + [units]
    out, u, c = [], 0, 0
    for b in range(len(lens)):
        for vh in range(VH):
            t0 = 0
            while t0 < unit[b]:
                while u >= begin[c + 1]:
                    c += 1
                take = min(unit[b] - t0, begin[c + 1] - u)
                if groups:
                    out.append((c, b, vh, first[b], tiles[b], True))
                else:
                    at = max(0, t0 - GROUP_COST)
                    out.append((c, b, vh, first[b] + at, max(0, t0 + take - GROUP_COST) - at, take == unit[b]))
                t0 += take
                u += take
    return out


def split_without_tiles(ps):
    """Pieces of split groups that have no tile of their own."""
    return [p for p in ps if p[4] == 0 and not p[5]]


def empty_before_others(ps):
    """Whole pieces without tiles (empty sequences) that are not their CTA's last."""
    return [x for x, y in zip(ps, ps[1:]) if x[4] == 0 and x[5] and x[0] == y[0] and y[4] > 0]
