"""The split of attention over many new tokens, as csrc/paged_sched.cuh computes it."""

TILE_COST, WHOLE_STEPS = 2, 2


def floor_sum(n, m, a, b):
    total = 0
    while True:
        if a >= m:
            total += n * (n - 1) // 2 * (a // m)
            a %= m
        if b >= m:
            total += n * (b // m)
            b %= m
        y = a * n + b
        if y < m:
            return total
        n, b = divmod(y, m)
        m, a = a, m


class Split:
    """seqs: (new tokens, length) of each sequence."""

    def __init__(self, seqs, parts, tokens, TK, grid, min_units, window=0, tree=False):
        self.seqs, self.parts, self.tokens, self.TK, self.window, self.tree = seqs, parts, tokens, TK, window, tree
        self.count = [-(-n // tokens) for n, _ in seqs]
        ends = [self.steps(s, t) for s, c in enumerate(self.count) for t in (c - 1, c - 2) if t >= 0]
        self.whole = max(ends, default=0) <= WHOLE_STEPS
        self.units = parts * sum(self.of(s) for s in range(len(seqs)))
        want = self.units // (1 if self.whole else min_units)
        self.ctas = max(1, min(grid, want))
        self.q, self.more = divmod(self.units, self.ctas)

    def first_slot(self, s, t):
        n, length = self.seqs[s]
        if self.window <= 0:
            return 0
        return max(0, length - n + (0 if self.tree else t * self.tokens) - self.window + 1)

    def steps(self, s, t):
        n, length = self.seqs[s]
        last = length - n + min(n, (t + 1) * self.tokens)
        return -(-last // self.TK) - self.first_slot(s, t) // self.TK

    def before(self, s, t):
        n, length = self.seqs[s]
        if self.whole or t == 0:
            return t
        base = length - n
        total = floor_sum(t, self.TK, self.tokens, base + self.tokens + self.TK - 1) + t * TILE_COST
        if self.window > 0:
            x0 = base - self.window + 1
            if self.tree:
                total -= t * (max(0, x0) // self.TK)
            else:
                skip = -(x0 // self.tokens) if x0 < 0 else 0
                if t > skip:
                    total -= floor_sum(t - skip, self.TK, self.tokens, x0 + skip * self.tokens)
        return total

    def of(self, s):
        c = self.count[s]
        if c == 0 or self.whole:
            return c
        return self.before(s, c - 1) + self.steps(s, c - 1) + TILE_COST

    def begin_of(self, c):
        return self.units if c >= self.ctas else self.q * c + min(c, self.more)

    def cta_of(self, x):
        cut = (self.q + 1) * self.more
        return x // (self.q + 1) if x < cut else self.more + (x - cut) // self.q

    def pieces(self, cta):
        """(sequence, part, tile, first step, steps, whole, slot, c0, c1) of one CTA."""
        u, end = self.begin_of(cta), self.begin_of(cta + 1)
        if u >= end:
            return
        begin, at = u, 0
        for s in range(len(self.seqs)):
            if u < at + self.parts * self.of(s):
                break
            at += self.parts * self.of(s)
        part, rest = divmod(u - at, self.of(s))
        t = max(t for t in range(self.count[s]) if self.before(s, t) <= rest)
        at = rest - self.before(s, t)
        while u < end:
            steps, cost = self.steps(s, t), 0 if self.whole else TILE_COST
            units = 1 if self.whole else steps + cost
            take = min(units - at, end - u)
            lo, hi = (0, steps) if self.whole else (max(0, at - cost), max(0, at + take - cost))
            if hi > lo:
                s0 = u - at + cost
                whole = hi - lo == steps
                slot = c0 = c1 = 0
                if not whole:
                    c0, c1 = self.cta_of(s0), self.cta_of(s0 + steps - 1)
                    slot = 2 * cta + (1 if cta == c0 and s0 > self.begin_of(c0) else 0)
                yield s, part, t, lo, hi - lo, whole, slot, c0, c1
            u += take
            at = 0
            if u < end:
                t += 1
                if t == self.count[s]:
                    t, part = 0, part + 1
                    if part == self.parts:
                        part, s = 0, s + 1
                        while self.count[s] == 0:
                            s += 1
