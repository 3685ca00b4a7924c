"""Sizes that reach each kernel of the grouped and dense bf16 products: the tile that a
workgroup computes there, and whether sums are taken in parts.  ``test_train_tiles.py`` holds them
to the rule that chooses (without a GPU), ``test_gpu_train_tiles.py`` runs them.

More than 128 columns in 128 rows are a run of tiles.
"""

# (T, k, E, N, K, B, tile, parts), either way round (K and N multiples of 8)
ROWS = [
    (300, 2, 4, 264, 200, 64, (64, 64), False),
    (5, 2, 4, 136, 4104, 64, (64, 64), True),
    (1000, 4, 8, 2056, 264, 256, (64, 128), False),
    (5, 2, 4, 1040, 4104, 64, (64, 128), True),
    (2000, 2, 4, 4096, 520, 128, (128, 128), False),
    (1500, 4, 8, 2056, 520, 256, (256, 256), False),
    (1500, 4, 8, 4104, 1032, 256, (256, 256), False),
]

# (T, k, E, N, K, tile, parts): weight gradients of several experts (K a multiple of 16)
SUMS = [
    (70, 2, 4, 264, 272, (64, 64), False),
    (4000, 1, 3, 72, 80, (64, 64), True),
    (100, 2, 32, 264, 208, (64, 128), False),
    (3000, 2, 8, 72, 2064, (128, 128), False),
    (1500, 4, 8, 520, 1040, (128, 128), False),
    (4000, 1, 3, 4104, 1040, (256, 256), False),
    (100, 2, 32, 520, 208, (128, 256), False),
    (100, 2, 32, 520, 1040, (128, 512), False),
    # blocks past 64 x 64, whose search takes another way
    (300000, 1, 5, 72, 80, (128, 128), True),
]

# (M, N, K, tile, parts): sums over all rows
DENSE = [
    (300, 264, 272, (64, 64), False),
    (20000, 72, 80, (64, 64), True),
    (300, 1040, 1040, (64, 128), False),
    (8200, 520, 528, (64, 128), True),
    (2050, 1040, 4112, (128, 128), False),
    (8200, 2056, 208, (128, 128), True),
    (8200, 4104, 2064, (256, 256), False),
    (64, 4104, 4112, (128, 256), False),
]

# operands of 2 GiB and more.  (T, N, K, B, tile): rows of X, either way round
WIDE = (1 << 17) + 40                                 # rows of 8208 columns: 2^31 bytes and more
WIDE_ROWS = [
    (WIDE, 136, 8208, 64, (64, 64)),
    (WIDE, 264, 8208, 128, (128, 128)),
    (WIDE, 520, 8208, 256, (256, 256)),
]
# (T, N, K, transposed, tile): one expert's weights, in parts
WIDE_WEIGHTS = [
    (40, 8208, 131080, True, (64, 128)),
    (4, 264, 1 << 22, False, (64, 64)),
]
# (rows, E, N, K, codes, tile): sums; of one expert, the dense ones too.  A has N columns, B K
WIDE_SUMS = [
    (WIDE, 1, 64, 8208, False, (64, 128)),            # taken as 64 x 64
    (WIDE, 1, 200, 8208, False, (128, 128)),
    (WIDE, 1, 1280, 8208, False, (256, 256)),
    (WIDE, 1, 8208, 16, False, (64, 64)),
    (WIDE, 1, 8208, 208, True, (128, 128)),
    (WIDE, 1, 8208, 1264, False, (256, 256)),
    (WIDE, 2, 200, 8208, False, (128, 128)),
    (WIDE, 2, 520, 8208, False, (256, 256)),
    (WIDE, 2, 8208, 16, True, (64, 64)),
    (2 * WIDE, 1, 8, 8208, True, (64, 128)),          # 2^31 codes and more
    (2 * WIDE, 1, 200, 8208, True, (128, 128)),
    (2 * WIDE, 2, 200, 8208, True, (128, 128)),
    (2 * WIDE, 2, 1296, 8208, True, (256, 256)),
]
