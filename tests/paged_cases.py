"""Batches whose attention gives every CTA many pieces of query tiles, and how they are split."""

from paged_model import Split

# name: lens, new, Hq, Hkv, page, window, tree, the whole pieces' steps that it is there for
MANY_PIECES = {
    "one_step": ([90 + b % 38 for b in range(300)], [1 + b % 5 for b in range(300)], 4, 4, 16, 0, False, {1}),
    "two_steps": ([129 + (37 * b) % 128 for b in range(300)], [1 + b % 5 for b in range(300)], 4, 4, 32, 0, False, {2}),
    "two_steps_full": ([256] * 60, [128] * 60, 8, 8, 64, 0, False, {2}),
    "three_steps": ([257 + (37 * b) % 128 for b in range(250)], [1 + b % 9 for b in range(250)], 4, 4, 16, 0, False, {3}),
    "mixed": ([1 + (131 * b) % 640 for b in range(250)], [min(1 + (131 * b) % 640, b % 9) for b in range(250)], 4, 4, 16, 0, False, {1, 2, 3, 4, 5}),
    "prompts_of_256": ([256] * 48, [256] * 48, 8, 8, 16, 0, False, {1, 2}),
    "prompts": ([64 * x + 5 for x in range(1, 13)], [64 * x + 5 for x in range(1, 13)], 16, 16, 32, 0, False, {1, 2, 3, 4}),
    "window": ([2048], [2048], 32, 8, 64, 100, False, {1, 2}),
    "trees": ([216] * 64, [16] * 64, 32, 8, 16, 0, True, {2}),
    "mixed_trees": ([1 + (131 * b) % 600 for b in range(120)], [min(1 + (131 * b) % 600, 1 + b % 31) for b in range(120)], 16, 8, 32, 0, True, {1, 2, 3, 4, 5}),
    "windowed_trees": ([1 + (131 * b) % 600 for b in range(120)], [min(1 + (131 * b) % 600, 1 + b % 31) for b in range(120)], 16, 8, 16, 90, True, {1, 2}),
}


def split_of(lens, new, Hq, Hkv, window, tree, fp32=False, D=128):
    rows = 64 if fp32 else 128
    G = Hq // Hkv
    parts = -(-G // rows)
    heads = -(-G // parts)
    return Split(list(zip(new, lens)), Hkv * parts, rows // heads, 64 if fp32 else 128, 304 if fp32 and D == 64 else 152, 2,
                 window, tree)
