"""Sizes of the grouped products' tests: rows of each expert, rows behind the last
expert's, K, O."""

# no rows, one row, one expert with everything, empty experts at both ends, groups
# around every tile edge, reductions that end inside a slice, more columns than a
# tile; from 64 experts on the streaming weight gradient: reductions of one to many
# slices in a row, several tiles to a workgroup, experts without rows, widths that
# end inside a tile
GROUPS = [
    ([0, 0, 0], 5, 64, 32), ([1], 0, 8, 8), ([0, 1, 0], 3, 72, 24), ([1, 1, 1, 1, 1, 1, 1, 1], 0, 2048, 768),
    ([3, 0, 7, 1], 2, 136, 264), ([15, 16, 17], 1, 520, 40), ([0, 0, 64, 0], 0, 64, 128), ([63, 65], 9, 200, 136),
    ([127, 0, 129, 1], 4, 264, 72), ([300], 20, 328, 520), ([255, 257], 0, 72, 264), ([2] * 70, 3, 128, 64),
    ([513, 3], 5, 136, 776), ([40, 0, 500, 260, 31], 100, 1032, 200), ([33] * 5 + [0] * 130 + [50], 7, 40, 72),
    ([700, 20], 0, 64, 1544), ([900], 1, 264, 264),
    ([1] * 64, 0, 136, 136), ([0] * 63 + [5], 2, 264, 136), ([0, 1, 64, 65, 129, 3, 200, 7] * 10, 11, 264, 136),
    ([70, 2, 0, 128, 1, 63, 0, 300] * 9, 0, 520, 520), ([1300] + [1, 0] * 40, 5, 264, 264),
    ([20] * 40, 0, 520, 1032),
    # few experts with many rows: the weight gradient's reduction in parts, some of them empty
    ([1600, 0, 3, 1900], 9, 264, 392), ([2500, 70], 5, 136, 264), ([4000], 30, 72, 128),
]

# many full tiles, compared in some rows: experts below and above the tiles' heights
LARGE = [
    ([400 + 37 * i % 220 for i in range(33)], 50, 2056, 4104),
    ([60 + 5 * i % 40 for i in range(64)], 0, 1032, 2056),
    ([3500, 0, 1] + [30 + 97 * i % 350 for i in range(61)], 7, 1544, 1032),
    ([260 + 3 * i % 50 for i in range(16)], 9, 712, 1032),
]

# Every form of the kernels: each size with silu and swiglu, gathered and not.  A few
# rows to an expert (the panels of 16 weight rows): one to three row tiles of 16, an
# expert without rows, reductions that 64 does not divide, columns that end inside a
# panel; experts of one to four units of 64 rows to a tile and of several tiles, also
# where the streaming kernels hold many experts; one expert of 64 or 128 with
# rows, and four.
FORMS = [
    ([1, 0, 5, 17, 3], 2, 1096, 72), ([2, 0, 17], 3, 1032, 264), ([40, 0, 1], 4, 1160, 40), ([1], 0, 1024, 8),
    ([8] * 64, 0, 1032, 72), ([0, 1, 64, 65, 9, 3, 127, 130] * 7 + [513, 260, 0, 1, 5, 20, 40, 33], 7, 520, 264),
    ([0, 1, 64, 65, 9, 3, 127, 130] * 7 + [513, 260, 0, 1, 5, 20, 40, 33], 7, 520, 520),
    ([0, 1, 64, 65, 129, 3, 200, 257] * 9, 11, 72, 776), ([0] * 70 + [1500] + [0] * 57, 9, 520, 264), ([0] * 20 + [3300] + [0] * 43, 7, 520, 520),
    ([0] * 30 + [300, 1, 0, 129, 600] + [0] * 93, 0, 264, 520), ([0, 1, 64, 65, 129, 200, 257, 300], 5, 520, 1032),
    ([200, 0, 300, 257, 129, 333, 191, 190], 4, 1544, 200), ([90, 0, 31], 4, 72, 4112), ([2500, 0, 70], 3, 136, 264),
]
FORM_ACTS = ("silu", "swiglu")
