"""Sizes of the experts' products whose sums are dealt out over the GPU by steps and joined, beside
ones that are done in whole tiles.  tests/test_step_abi.py holds the rule to these lists on the CPU,
tests/test_gpu_grouped.py runs them."""

# (tokens of each expert, out_features, in_features): several experts, some without a token (a tile
# that counts a step and has none), with few and with many, whose tiles begin and end inside a part
GRADS_IN_PARTS = [
    ((7000, 3), 200, 500), ((9000, 0, 900), 184, 412), ((0, 12000, 1, 7999, 0), 300, 300),
    ((20000, 1, 0, 63, 64, 65, 129, 9000, 0, 5000, 4000, 1700), 100, 104),
]
# features along the sum first: o of the input gradient, i of the product
PRODUCTS_IN_PARTS = [((300, 0, 200), 6000, 512), ((1, 0, 700, 0, 90), 5000, 264), ((20, 3, 0, 9), 4160, 300)]
# the same with weights whose rows start anywhere
ODD_PRODUCTS_IN_PARTS = [((300, 0, 200), 6101, 513), ((1, 0, 700, 0, 90), 5001, 265), ((20, 3, 0, 9), 4161, 301)]

# whole tiles: too short sums, or enough tiles
GRADS_WHOLE = [((0, 1500, 0, 7, 2600, 0), 200, 104), ((2, 3000), 72, 64), ((513, 100), 96, 1032),
               ((2048,) * 8, 4096, 4096)]
PRODUCTS_WHOLE = [((5, 0, 20), 2003, 3001), ((1000, 24), 256, 2056), ((256, 256), 512, 256),
                  ((2048,) * 8, 4096, 11008)]
