"""bf16 attention over the paged cache: no order of its warps, copies and products stops it, loses
a result or reads a buffer that is not what it takes it for."""

import random

import pytest

from paged_cases import MANY_PIECES, split_of
from paged_roles import QUADS, Cta, Stuck, random_pieces

LENGTHS = [[1], [2], [3], [4], [5], [1, 2], [2, 3], [1, 2, 3, 4, 5]]


def ids(x):
    return "-".join(map(str, x)) if isinstance(x, list) else str(x)


@pytest.mark.parametrize("HD", [64, 128])
@pytest.mark.parametrize("exchanged", ["none", "all"])
@pytest.mark.parametrize("lengths", LENGTHS, ids=ids)
def test_every_order_ends(lengths, exchanged, HD):
    """With a cap no quad exchanges its first scores, without one all do."""
    rng = random.Random(len(lengths) + 10 * HD)
    for _ in range(6):
        cta = Cta(random_pieces(rng, lengths, exchanged), HD, rng)
        cta.run()
        assert all(n == 1 for row in cta.results for n in row) and len(cta.results[0]) == QUADS


def test_one_barrier_for_every_exchange_is_too_few():
    """The model sees it: the group that begins two pieces in turn may arrive for both before the
    other group has looked at the first."""
    rng = random.Random(5)
    stuck = 0
    for _ in range(10):
        try:
            Cta(random_pieces(rng, [2], "all"), 128, rng, tops_by="one").run()
        except Stuck:
            stuck += 1
    assert stuck


@pytest.mark.parametrize("drains", ["issued", "always"])
def test_a_wait_that_gives_up_ends_every_role(drains):
    """And at once: none waits on its way out for a copy that nobody issued (which takes as long as
    the wait that gave up)."""
    rng = random.Random(9)
    stuck = 0
    for _ in range(60):
        cta = Cta(random_pieces(rng, [1, 2, 3], rng.choice(["all", "none"])), rng.choice([64, 128]), rng, drains=drains,
                  gives_up=rng.randint(1, 900))
        try:
            cta.run()
            assert cta.abort
        except Stuck:
            stuck += 1
    assert (stuck > 0) == (drains == "always")


@pytest.mark.parametrize("name", MANY_PIECES)
def test_the_batches_give_every_cta_many_pieces(name):
    """Of the lengths that they are there for, one after another in the same CTA."""
    lens, new, Hq, Hkv, _, window, tree, want = MANY_PIECES[name]
    sp = split_of(lens, new, Hq, Hkv, window, tree)
    ctas = [[n for _, _, _, _, n, *_ in sp.pieces(c)] for c in range(sp.ctas)]
    assert sp.ctas == 152 and sum(len(c) >= 3 for c in ctas) > 100
    assert want <= {n for c in ctas for n in c}
    followed = {n for c in ctas for n in c[:-1]}  # a piece of that length, then another one
    assert want <= followed


def test_the_batches_split_end_in_every_order():
    """The pieces of some CTAs of each batch, through the roles."""
    rng = random.Random(3)
    for name, (lens, new, Hq, Hkv, _, window, tree, _) in MANY_PIECES.items():
        sp = split_of(lens, new, Hq, Hkv, window, tree)
        for c in (0, 75, 151):
            pieces = [(n, {n - 1}, tuple(range(QUADS))) for _, _, _, _, n, *_ in sp.pieces(c)]
            Cta(pieces, rng.choice([64, 128]), rng).run()
