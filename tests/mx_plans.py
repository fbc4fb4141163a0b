"""Products for every kernel that gemm_mx chooses between, as a device of 256 compute
units gets them: (M, N, K, (tile_m, tile_n, stages), K split). Shapes come out of a search
over random sizes for the plans; each kernel has an even and an odd number of 128-value
stretches (a stage is two of them) and M and N that end inside a tile."""

PLANS = [
    # few rows of A: partial last steps (the 8 waves take 4 stretches at a time), one and two rounds
    (1, 587, 4096, (16, 16, 0), False),
    (7, 1030, 5000, (16, 16, 0), False),
    (16, 17, 1063, (16, 16, 0), False),
    (2, 2100, 8000, (16, 16, 0), False),
    (13, 3143, 6880, (16, 16, 0), False),
    (17, 33, 3390, (32, 16, 0), False),
    (20, 1030, 4096, (32, 16, 0), False),
    (31, 700, 4000, (32, 16, 0), False),
    (250, 4300, 9000, (64, 64, 4), False),
    (1250, 1111, 2049, (64, 64, 4), False),
    (100, 70, 33000, (64, 64, 4), True),
    (31, 1025, 4097, (64, 64, 4), True),
    (413, 2330, 101, (128, 128, 4), False),
    (2300, 1745, 1500, (128, 128, 4), False),
    (2301, 1745, 1150, (128, 128, 4), False),
    (580, 1, 25684, (128, 128, 4), True),
    (515, 513, 20001, (128, 128, 4), True),
    (4099, 914, 106, (128, 128, 2), False),
    (3700, 3784, 1500, (128, 128, 2), False),
    (1038, 3670, 545, (128, 128, 2), False),
    (70, 4369, 24881, (128, 128, 2), True),
    (679, 3241, 39905, (128, 128, 2), True),
    (3140, 1286, 5175, (256, 128, 2), False),
    (2801, 1503, 5350, (256, 128, 2), False),
    (424, 2387, 34463, (256, 128, 2), True),
    (3386, 3782, 1561, (256, 256, 2), False),
    (3659, 3472, 1717, (256, 256, 2), False),
    (2048, 2048, 66001, (256, 256, 2), True),
    (1793, 2000, 80000, (256, 256, 2), True),
]
IDS = [f"{m}x{n}x{k}" for m, n, k, _, _ in PLANS]


def is_plan(p, tile, split):
    return (p.tile_m, p.tile_n, p.stages) == tile and (p.split_k > 1) == split
