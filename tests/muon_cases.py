"""The lists of matrices that tests/test_gpu_muon_tiles.py runs, here so that a
test without a GPU can look at which kernels they reach."""

# products of 64, 128 and 256 a side, whole and ragged, wide and tall
LARGE = [[(1000, 1000)] * 4, [(2048, 2048)] * 4, [(2047, 2049), (2049, 2047)] * 2, [(2500, 2500)] * 3,
         [(1500, 4000), (4000, 1500)], [(1700, 3401)] * 3, [(4001, 9003)], [(9003, 4001)]]
# of no one's multiples, and past what one workgroup takes; the last two split
# the depth of X X^T
TILED = [[(257, 259)], [(259, 257)], [(300, 1030)], [(1030, 300)], [(257, 259), (1030, 300), (300, 1030), (259, 257)],
         [(170, 4100)], [(1601, 150)]]
SMALL = [[(70, 90)], [(90, 70)], [(64, 96)], [(1, 300)]]
