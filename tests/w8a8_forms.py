"""Shapes that reach each form of the 8-bit products' kernels.  The planners choose a form by modelled
time, so a change of the model can move a shape to another one: `form` asks the library, and the CPU
tests hold every entry of these tables to it."""
from w4_gemm_amd._lib import i8_form

# (tile rows, tile columns, K split): (m, n, k) of one layer
FWD = {
    (16, 16, False): (40, 70, 512),
    (16, 32, False): (1, 10947, 1792),
    (32, 64, False): (21, 4507, 2048),
    (64, 64, False): (34, 10247, 1536),
    (64, 256, False): (65, 10276, 256),
    (64, 256, True): (622, 83, 15616),
    (128, 256, False): (4584, 781, 256),
    (128, 256, True): (705, 258, 9472),
    (224, 256, False): (1029, 7545, 256),
    (256, 256, False): (3000, 4701, 256),
}
# (tile rows, tail in parts): (m, n, k) of one layer
GRAD = {
    (64, False): (65, 67, 256),
    (64, True): (303, 1538, 256),
    (128, False): (328, 64, 11008),
    (128, True): (2510, 2931, 3328),
}
# plans that split, with several experts: (m, n, k, groups)
FWD_SPLIT = {64: (698, 98, 11264, 3), 128: (463, 136, 12800, 19)}
GRAD_SPLIT = {64: (317, 1801, 256, 3), 128: (3725, 3947, 2304, 3)}
# few rows of many experts, the gradient's tail in parts
GRAD_SPLIT_MANY = [(12, 1294, 256, 19), (12, 1284, 256, 79)]


def form(m, n, k, groups=1, rank=16, dgrad=False):
    """Key of the tables above, for the plan of this call."""
    rows, cols, splits, _, _ = i8_form(m, n, k, groups, rank, dgrad)
    return (rows, splits > 1) if dgrad else (rows, cols, splits > 1)
