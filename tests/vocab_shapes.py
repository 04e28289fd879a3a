"""Shapes (tokens, rows, columns, dx's type, dw's, added) that reach every form of the
vocabulary loss's tiles, most at 16 stages and more, ragged in every direction."""

B, F = "bfloat16", "float32"
SHAPES = [
    (167, 201, 216, B, F, False), (2087, 217, 200, B, F, True), (189, 67, 1032, B, B, True),
    (1785, 593, 1032, F, F, True), (2251, 1051, 1064, F, F, True), (151, 69, 48, F, B, False),
    (3575, 1167, 1712, B, F, False), (511, 1025, 1120, B, F, False), (2219, 3721, 1032, F, B, True),
    (29, 1097, 32, F, F, True), (195, 11829, 112, B, B, True), (167, 10561, 32, B, F, False),
    (1237, 1167, 6600, B, F, True), (1365, 1421, 504, B, B, True), (399, 10047, 136, B, B, False),
    (2991, 2487, 1432, B, B, False), (153, 695, 1688, F, B, False), (195, 1615, 1248, F, F, True),
    (199, 885, 2344, F, B, True), (183, 10907, 280, F, B, False), (199, 6623, 520, F, F, False),
    (151, 3269, 1208, B, F, True), (179, 69, 36304, F, B, False), (209, 301, 17096, B, F, False),
    (157, 1847, 4104, F, B, True),
    # the forms of a large head: 65 stages
    (97, 20011, 4104, B, B, False), (201, 20011, 4104, B, F, True), (501, 14001, 4104, F, B, False),
    (63, 60013, 2056, B, B, False),
    # dw stored past the caches
    (49, 5965, 5664, B, F, False), (47, 18193, 1864, B, F, True), (127, 105567, 368, F, F, True),
    (53, 344677, 120, B, F, False), (41, 10389, 6536, F, B, False), (51, 720087, 96, B, B, False),
]
# the same in small tiles: few rows of many columns, or the other way round
PAST = [(3, 49, 701560, B, F, False), (169, 127, 267624, B, F, True), (579, 546983, 64, B, F, False),
        (405, 123, 618640, B, B, False)]
