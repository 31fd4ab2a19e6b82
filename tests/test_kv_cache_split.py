"""CPU checks of the decode's split: the model gives every tile to one piece, and the GPU
tests' lengths have the pieces that they are chosen for."""

import pytest

from split_cases import FP32_CASES
from split_model import decode_ctas, empty_before_others, pieces, split_without_tiles


def max_len_of(lens, page):
    return max(1, -(-max(lens) // page)) * page


@pytest.mark.parametrize("lens, window", [([2048, 1476, 905, 333], 0), ([5, 0, 100_000], 0), ([4099, 90, 1000] * 30, 1024),
                                          ([40] * 70, 0), ([0], 0), ([0, 0, 900] * 200, 0)], ids=["four", "long", "window",
                                                                                                 "whole", "none", "many"])
@pytest.mark.parametrize("e", [2, 4])
def test_every_tile_belongs_to_one_piece(lens, window, e):
    n = max_len_of(lens, 16)
    tk, grid = decode_ctas(lens, 4, 2, 64, e, n)
    seen = {}
    last = (-1, 0)
    for c, b, vh, tile, tiles, whole in pieces(lens, 4, 2, 64, e, n, window):
        assert 0 <= c < grid and c >= last[0]
        last = (c, b)
        seen.setdefault((b, vh), []).extend(range(tile, tile + tiles))
    for b, x in enumerate(lens):
        first = max(0, x - window) // tk if window else 0
        for vh in range(2):
            assert seen[b, vh] == list(range(first, -(-x // tk)))


@pytest.mark.parametrize("case", FP32_CASES, ids=lambda c: str(c)[:40])
def test_the_cases_have_pieces_without_tiles(case):
    lens, Hq, Hkv, D, page = case
    ps = pieces(lens, Hq, Hkv, D, 4, max_len_of(lens, page))
    assert split_without_tiles(ps) or empty_before_others(ps)


def test_both_kinds_are_among_the_cases():
    every = [pieces(lens, Hq, Hkv, D, 4, max_len_of(lens, page)) for lens, Hq, Hkv, D, page in FP32_CASES]
    assert sum(bool(split_without_tiles(p)) for p in every) >= 2 and any(empty_before_others(p) for p in every)
