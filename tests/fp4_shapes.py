"""Sizes of 4-bit products that reach every tile kernel: the plan each is to have
(the tile's columns, w the larger operand, pairs that share a tile's K, the least
number of tiles of the busiest of 76 pairs)."""

# (M, N, K): (columns, swapped, splits, tiles)
PLANS = {
    (8200, 2050, 800): (256, False, 1, 3), (8200, 2056, 800): (256, False, 1, 3), (2050, 8200, 800): (256, True, 1, 3),
    (9000, 1700, 320): (128, False, 1, 3), (9000, 1704, 320): (128, False, 1, 3), (1700, 9000, 320): (128, True, 1, 3),
    (70000, 61, 320): (64, False, 1, 3), (70000, 64, 320): (64, False, 1, 3), (61, 70000, 320): (64, True, 1, 3),
    (30000, 130, 64): (64, False, 1, 3),
    (64, 200, 4096): (64, True, 4, 1), (200, 63, 4096): (64, False, 4, 1), (40, 4096, 2048): (64, True, 2, 1), (4100, 40, 2080): (64, False, 2, 1),
}
