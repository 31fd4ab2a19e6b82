"""The split of attention over many new tokens: every step of every query tile belongs to
one piece, the pieces of a shared tile know one another, and no two of them share a slot."""

import random

import pytest

from paged_model import TILE_COST, Split, floor_sum


def test_floor_sum():
    rng = random.Random(1)
    for _ in range(2000):
        n, m, a, b = rng.randint(0, 50), rng.randint(1, 140), rng.randint(0, 300), rng.randint(0, 10 ** 6)
        assert floor_sum(n, m, a, b) == sum((a * i + b) // m for i in range(n))


def cases():
    rng = random.Random(2)
    yield [(1, 1)], 1, 64, 64, 304, 4, 0, False
    yield [(32, 131009)], 8, 32, 128, 152, 4, 0, True
    yield [(0, 5), (0, 0)], 2, 16, 64, 304, 4, 0, False
    for _ in range(100):
        seqs = []
        for _ in range(rng.choice([1, 1, 2, 5, 40])):
            n = rng.choice([0, 1, rng.randint(1, 40), rng.randint(1, 3000)])
            seqs.append((n, n + rng.choice([0, rng.randint(0, 300), rng.randint(0, 20000)])))
        yield (seqs, rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 12, 16, 21, 25, 32, 64, 128]), rng.choice([64, 128]),
               rng.choice([152, 304]), rng.choice([1, 2, 4, 8]), rng.choice([0, 0, 1, 7, 100, 1024, 30000]), rng.random() < 0.4)


@pytest.mark.parametrize("case", list(cases()), ids=lambda c: f"{len(c[0])}x{c[1]}")
def test_pieces(case):
    sp = Split(*case)
    for s, c in enumerate(sp.count):
        if not sp.whole:
            assert all(sp.before(s, t + 1) - sp.before(s, t) == sp.steps(s, t) + TILE_COST for t in range(c - 1))
        assert all(sp.steps(s, t) >= 1 for t in range(c))
    seen, slots, parts = {}, set(), {}
    for cta in range(min(case[4], sp.ctas + 1)):
        for s, part, t, lo, n, whole, slot, c0, c1 in sp.pieces(cta):
            assert n > 0 and c0 <= (cta if not whole else c0)
            seen.setdefault((s, part, t), []).append((lo, lo + n))
            if not whole:
                assert slot not in slots
                slots.add(slot)
                parts.setdefault((s, part, t), []).append((cta, c0, c1))
    want = {(s, part, t) for s, c in enumerate(sp.count) for part in range(case[1]) for t in range(c)}
    assert set(seen) == want
    for (s, part, t), spans in seen.items():
        at = 0
        for lo, hi in spans:
            assert lo == at
            at = hi
        assert at == sp.steps(s, t)
    starts = set()
    for tile, got in parts.items():
        c0, c1 = got[0][1:]
        assert [g[0] for g in got] == list(range(c0, c1 + 1)) and all(g[1:] == (c0, c1) for g in got)
        assert c0 not in starts  # the counter of a CTA serves one tile
        starts.add(c0)
