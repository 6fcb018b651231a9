"""Sizes of the 8-bit float products beside those of f8_forms.py, in the same order: kind, rows, N, K,
experts, bits of the result, tile rows and columns, splits.

DEEP: tiles whose contraction is not split, over 9 to 14 blocks of 128 with one to three behind the last
whole four, so that the four-stage loop comes round and every way out of it is taken.  One layer's last
row tile is at most half full.
SPLIT: split forms of 256-row tiles, and of the gated block for every curve of the join."""
DEEP = [
    ("fwd", 8399, 812, 1089, 1, 16, 224, 256, 1), ("fwd", 926, 8358, 1281, 1, 16, 224, 256, 1),
    ("fwd", 6592, 1063, 1153, 3, 16, 224, 256, 1), ("fwd", 7519, 1793, 1032, 1, 16, 256, 256, 1),
    ("fwd", 1586, 8372, 1288, 1, 16, 256, 256, 1), ("fwd", 1060, 8399, 1153, 3, 16, 256, 256, 1),
    ("fwd", 8510, 262, 1345, 1, 16, 128, 256, 1), ("fwd", 7444, 260, 1089, 4, 16, 128, 256, 1),
    ("fwd", 500, 82, 1153, 3, 16, 64, 256, 1), ("fwd", 8894, 266, 1281, 1, 32, 128, 256, 1),
    ("fwd", 8278, 319, 1151, 4, 32, 128, 256, 1), ("fwd", 4818, 40, 1153, 3, 32, 64, 256, 1),
    ("gated_fwd", 8377, 414, 1089, 1, 16, 224, 128, 1), ("gated_fwd", 8592, 389, 1288, 1, 16, 224, 128, 1),
    ("gated_fwd", 464, 6283, 1153, 3, 16, 224, 128, 1), ("gated_fwd", 2052, 3282, 1025, 1, 16, 256, 128, 1),
    ("gated_fwd", 4415, 1615, 1288, 1, 16, 256, 128, 1), ("gated_fwd", 1107, 4082, 1160, 3, 16, 256, 128, 1),
    ("gated_fwd", 8890, 138, 1288, 1, 16, 128, 128, 1), ("gated_fwd", 7533, 130, 1025, 4, 16, 128, 128, 1),
    ("gated_fwd", 360, 57, 1153, 3, 16, 64, 128, 1), ("gated_fwd", 8197, 131, 1371, 1, 32, 128, 128, 1),
    ("gated_fwd", 8638, 132, 1151, 4, 32, 128, 128, 1), ("gated_fwd", 546, 250, 1153, 3, 32, 64, 128, 1),
    ("dgrad", 4757, 1032, 1612, 1, 16, 224, 256, 1), ("dgrad", 8370, 1371, 788, 1, 16, 224, 256, 1),
    ("dgrad", 822, 1153, 8000, 3, 16, 224, 256, 1), ("dgrad", 8736, 1032, 1578, 1, 16, 256, 256, 1),
    ("dgrad", 5951, 1288, 2333, 1, 16, 256, 256, 1), ("dgrad", 1277, 1160, 7345, 3, 16, 256, 256, 1),
    ("dgrad", 8586, 1407, 282, 1, 16, 128, 256, 1), ("dgrad", 8060, 1032, 263, 4, 16, 128, 256, 1),
    ("dgrad", 654, 1153, 63, 3, 16, 64, 256, 1), ("dgrad", 8455, 1345, 282, 1, 32, 128, 256, 1),
    ("dgrad", 8396, 1025, 287, 4, 32, 128, 256, 1), ("dgrad", 4610, 1160, 40, 3, 32, 64, 256, 1),
    ("gated_bwd", 1654, 520, 4873, 1, 16, 224, 256, 1), ("gated_bwd", 8610, 833, 771, 1, 16, 224, 256, 1),
    ("gated_bwd", 6377, 513, 1086, 3, 16, 224, 256, 1), ("gated_bwd", 1809, 520, 7814, 1, 16, 256, 256, 1),
    ("gated_bwd", 1831, 769, 7281, 1, 16, 256, 256, 1), ("gated_bwd", 1364, 513, 6960, 3, 16, 256, 256, 1),
    ("gated_bwd", 8202, 577, 274, 1, 16, 128, 256, 1), ("gated_bwd", 7538, 513, 268, 4, 16, 128, 256, 1),
    ("gated_bwd", 314, 513, 131, 3, 16, 64, 256, 1), ("gated_bwd", 8505, 513, 288, 1, 32, 128, 256, 1),
    ("gated_bwd", 8530, 513, 259, 4, 32, 128, 256, 1), ("gated_bwd", 4940, 513, 40, 3, 32, 64, 256, 1),
]
SPLIT = [
    ("fwd", 9132, 4, 3435, 3, 16, 256, 256, 5), ("dgrad", 9860, 5519, 22, 1, 16, 256, 256, 6),
    ("gated_fwd", 9707, 11, 15765, 2, 16, 256, 128, 5), ("gated_fwd", 25, 39, 1280, 1, 32, 64, 128, 3),
    ("gated_fwd", 27, 32, 1168, 1, 16, 64, 128, 3),
]
CURVES = ("silu", "gelu", "gelu_tanh")


def with_curves(forms):
    """Each form with each curve that it is compiled for or told (the gated forward), or with one."""
    return [(*f, act) for f in forms for act in (CURVES if f[0] == "gated_fwd" else CURVES[:1])]


def stages(kind, n, k):
    """Blocks of 128 along the contraction."""
    blocks = -(-(n if kind in ("dgrad", "gated_bwd") else k) // 128)
    return 2 * blocks if kind == "gated_bwd" else blocks
