"""Shapes that take each way of cutting the products behind la_linear_* (csrc/linear_cut.hpp), with several steps of
128 bytes and ragged edges.  test_proj_tiles.py pins which way that is, test_gpu_proj_more.py runs them.
"""
FEW, T256, T128, T64, DEEP = -1, 0, 1, 2, 3  # the few tokens' kernel; tiles of 256, 128, 64, and 64 with four steps in LDS
SLOTS = {T256: 256, T128: 512, T64: 768, DEEP: 512}  # workgroups that the chip holds

# M, N, K, tiles, more than one round of them
FORWARD = [
    (64, 35, 144, FEW, False),
    (33, 4090, 4112, DEEP, False),
    (67, 17, 272, DEEP, False),
    (862, 3477, 400, DEEP, True),
    (24856, 73, 16, DEEP, True),
    (25615, 65, 144, DEEP, True),
    (527, 3898, 272, T64, False),
    (1112, 3789, 144, T64, True),
    (1291, 3141, 288, T64, True),
    (862, 3527, 1648, T128, False),
    (33060, 66, 1040, T128, False),
    (2433, 3849, 464, T128, True),
    (3589, 3437, 176, T128, True),
    (29181, 705, 144, T128, True),
    (34805, 584, 32, T128, True),
    (2192, 3810, 1536, T256, False),
    (7946, 3484, 160, T256, True),
    (7557, 3210, 336, T256, True),
    (38479, 651, 272, T256, True),
]

# M, N, K, (tiles, parts of the sum, more than one round) of dx and of dweight, one launch of both
GRADIENTS = [
    (2000, 1552, 512, (DEEP, 1, False), (DEEP, 1, False), True),
    (309, 795, 1872, (T64, 1, False), (T64, 1, False), True),
    (650, 965, 1920, (T128, 1, False), (T128, 1, False), True),
    (65, 2700, 1120, (DEEP, 8, False), (DEEP, 1, True), False),
    (25485, 17, 80, (DEEP, 1, True), (DEEP, 16, False), False),
    (71, 3450, 1168, (T64, 16, False), (T64, 1, True), False),
    (73, 1118, 1824, (DEEP, 4, False), (T64, 1, False), False),
    (467, 1531, 1136, (T64, 4, False), (DEEP, 1, False), False),
    (22451, 17, 144, (T64, 1, True), (DEEP, 16, False), False),
    (2436, 321, 656, (DEEP, 1, False), (T64, 8, False), False),
    (17684, 3541, 16, (T64, 8, True), (DEEP, 8, False), False),
    (414, 2049, 1648, (DEEP, 2, False), (T128, 1, False), False),
    (971, 3677, 1072, (T128, 4, False), (T128, 1, False), False),
    (4469, 203, 1888, (T128, 1, True), (DEEP, 4, False), False),
    (3215, 627, 1632, (T128, 1, False), (T128, 4, False), False),
    (40000, 1571, 560, (T256, 1, True), (T128, 16, True), False),
    (8460, 274, 928, (T256, 1, False), (T64, 8, False), False),
    (33058, 69, 672, (T256, 1, True), (DEEP, 16, False), False),
    (2503, 3684, 1440, (T256, 4, False), (T128, 1, False), False),
    (4578, 1449, 1696, (T128, 1, False), (T256, 4, False), False),
    (9000, 2100, 1040, (T256, 1, False), (T256, 4, False), False),
    (12974, 2448, 1664, (T256, 1, True), (T256, 8, True), False),
]
