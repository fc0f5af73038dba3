"""Sizes at which the linear layer's product with adapters is cut in every way that
there is, for test_adapters_cuts.py (which says that they are) and
test_gpu_adapters_cuts.py (which runs them)."""

# (M, N, K): {tile edge (0: row by row), slices of a sum: none, all tiles' or some tiles', operands: as they are by
# 64×64 tiles (loose), copied first or direct}
TILES = {
    (66, 100, 24): (64, "none", "direct"), (68, 80, 2056): (64, "all", "direct"), (1177, 1701, 4056): (64, "some", "direct"),
    (65, 130, 57): (64, "none", "loose"), (79, 70, 2010): (64, "all", "loose"), (5465, 359, 4661): (64, "some", "loose"),
    (197, 8483, 24): (128, "none", "direct"), (4106, 71, 5056): (128, "all", "direct"), (595, 6682, 768): (128, "some", "direct"),
    (8238, 193, 34): (128, "none", "copied"), (1515, 67, 16001): (128, "all", "copied"), (6624, 588, 737): (128, "some", "copied"),
    (8294, 457, 16): (256, "none", "direct"), (129, 5535, 14248): (256, "all", "direct"), (3432, 4747, 672): (256, "some", "direct"),
    (8380, 457, 17): (256, "none", "copied"), (5515, 129, 13277): (256, "all", "copied"), (2247, 7216, 492): (256, "some", "copied"),
}
# at most 64 rows, which tiles take: T is written for them by the kernel for few rows
FEW_IN_TILES = {
    (40, 90, 6840): (64, "all", "direct"), (17, 8401, 1104): (64, "none", "direct"), (33, 90, 9157): (64, "all", "loose"),
    (34, 4182, 1463): (64, "none", "loose"), (32, 7412, 11584): (64, "all", "direct"), (55, 1024, 6463): (64, "all", "loose"),
}
# row by row, blocks of 32 rows of W; blocks of 16 rows of X
ROW_BY_ROW = {(1, 8291, 16): 1, (17, 8481, 16): 2, (33, 8197, 33): 3, (64, 8200, 64): 4}
