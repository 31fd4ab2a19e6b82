"""fp32 decodes some of whose pieces have no tile: a CTA's range that ends right behind a
group's first unit, and empty sequences in front of others.  lens, Hq, Hkv, D, page."""

FP32_CASES = [
    ([2048, 1476, 905, 333], 4, 2, 64, 16),
    ([700, 300], 16, 2, 128, 64),
    ([0, 500] * 20, 2, 2, 64, 16),
    ([0, 700] * 100, 2, 2, 64, 16),
    ([0, 0, 3000, 0, 1300, 0], 8, 2, 128, 16),
    ([1000 + 37 * i for i in range(12)], 5, 1, 128, 32),
]
