"""Sizes of the INT8 product that reach each of its kernels (which ones, test_matmul_plan.py checks without a GPU).

A pair's 256-column tile leaves through two 128-column halves, each in two pieces of 64: `r` columns past a whole tile
end in the first or second piece of either half, one column of a piece included.
"""
PAIR_T, PAIR_N = 3001, 4096
UNALIGNED = [1, 2, 3, 4, 5, 6, 7, 63, 65, 66, 127, 129, 190, 255]      # r; rows of every alignment
ALIGNED = [0, 8, 40, 136, 248]
PAIRS = [(PAIR_T, 272 if r % 2 else 1040, PAIR_N + r) for r in UNALIGNED + ALIGNED] + \
    [(4001, 16, 9001), (4001, 128, 9000), (65, 8192, 30000), (200, 1040, 40003), (257, 2048, 9001)]
# clusters: (tile's tokens, split): a size of each
FEW = {(16, 1): (1, 2560, 10576), (16, 2): (9, 6016, 8901), (16, 4): (8, 5120, 2560), (16, 8): (5, 8192, 512),
       (32, 1): (17, 640, 10001), (32, 2): (19, 5680, 7275), (32, 4): (31, 4096, 4096), (32, 8): (32, 4096, 300),
       (64, 1): (64, 2560, 10576), (64, 2): (50, 4096, 7000), (64, 4): (64, 4096, 2048), (64, 8): (33, 4096, 777),
       (128, 1): (512, 8192, 4096), (128, 2): (200, 8192, 3000), (128, 4): (128, 5120, 2560), (128, 8): (129, 8192, 700)}
LONGEST_K = 131056
EXTREME = [(3, 160, 0), (200, 160, 0), (1000, 2048, 1), (1000, 2050, 1)]      # tokens, channels, on pairs
