"""Sizes of the experts' operators by the form that their rules choose for them on a GB300 (152 SMs, which
hold 76 clusters of 2 CTAs at once, 36 of 4 and 15 of 8): so that a rule that changes does not leave a
form without a test."""
import torch


def spread(rows: int, groups: int, seed: int = 0) -> list[int]:
    """Uneven sizes of `groups` groups, one of three or more empty, that add up to `rows`."""
    g = torch.Generator().manual_seed(seed + rows)
    p = torch.exp(0.7 * torch.randn(groups, generator=g))
    if groups > 2:
        p[groups // 2] = 0
    return torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=groups).tolist()


# (rows of a tile, units that share its K, sizes of the groups, N, K)
PRODUCTS = [
    (32, 1, spread(44, 40), 136, 2160), (32, 1, spread(34, 24), 1408, 2888), (32, 1, [12], 10000, 2064),
    (32, 2, [10, 0, 1], 2880, 264), (32, 2, spread(28, 8), 976, 2152),
    (32, 4, [1], 3448, 1448), (32, 4, spread(9, 16), 136, 1992), (32, 4, spread(20, 40), 72, 2280),
    (32, 8, [2, 1], 136, 3080), (32, 8, [1], 1760, 2288),
    (64, 1, [400, 58], 1064, 576), (64, 1, spread(326, 40), 264, 2864),
    (64, 1, spread(413, 40), 848, 1944), (64, 1, spread(206, 24), 776, 2064),  # several tiles to a pair; planned
    (128, 1, [300, 0, 172], 3184, 240), (128, 1, spread(1181, 1), 1304, 2304),
    (128, 1, spread(392, 16), 3200, 1000), (128, 1, spread(332, 40), 1328, 2216),
    (128, 2, [128], 2048, 2048), (128, 2, [256], 2048, 2048), (128, 2, [1000], 512, 2048), (128, 2, [129, 36], 2472, 1464),
    (128, 2, spread(49, 5), 1560, 2096), (128, 2, spread(131, 16), 448, 2360),
    (128, 4, [300], 1024, 2048), (128, 4, [417, 41], 536, 1496), (128, 4, [1433], 200, 2888), (128, 4, spread(992, 8), 168, 3064),
    (256, 1, [45], 80, 32), (256, 1, spread(199, 24), 288, 2088),
    (256, 1, spread(1836, 24), 2752, 240), (256, 1, spread(346, 40), 3408, 2200),
    (512, 1, [2300, 198, 0], 2744, 200), (512, 1, spread(3643, 24), 552, 2304),
    (512, 1, [7000, 741], 3976, 104), (512, 1, [2000, 700, 513, 0, 255, 1, 1500, 448], 3568, 1992),
]

# Groups of whole stages, with remainders, of one row and none, 40 of them: under 384 rows on average, and more.
SHORT = [128, 0, 100, 64, 1, 192, 17, 256, 33, 90] * 4
LONG = [512, 384, 0, 640, 401, 768, 1, 1024, 130, 600] * 4

# (operands' and result's type, added, rows of a stage, stored by TMA, sizes, N, K): 5 or 4 rounds of tiles
GRADIENTS_16 = [
    ("bf16", "bf16", True, 64, True, SHORT, 512, 1032), ("fp16", "fp16", True, 64, True, SHORT, 520, 776),
    ("bf16", "bf16", False, 64, True, SHORT[:36], 264, 776), ("bf16", "fp32", False, 64, True, SHORT[:36], 264, 776),
    ("bf16", "bf16", False, 64, False, SHORT, 512, 1032), ("fp16", "fp16", False, 64, False, SHORT, 520, 776),
    ("fp16", "fp32", False, 64, False, SHORT, 512, 1032), ("bf16", "fp32", True, 64, False, SHORT, 264, 1032),
    ("bf16", "bf16", True, 128, True, LONG, 512, 1032), ("fp16", "fp16", True, 128, True, LONG, 520, 776),
    ("bf16", "fp32", False, 128, True, LONG, 512, 1032), ("fp16", "fp16", False, 128, True, LONG[:36], 264, 776),
    ("bf16", "bf16", False, 128, False, LONG, 512, 1032), ("fp16", "fp16", False, 128, False, LONG, 520, 776),
    ("bf16", "fp32", True, 128, False, LONG, 512, 1032), ("fp16", "fp32", True, 128, False, LONG, 264, 776),
]
# (result's type, added, stored by TMA, sizes, N, K)
GRADIENTS_8 = [
    ("bf16", False, True, SHORT, 512, 1024), ("fp16", True, True, SHORT, 384, 1024), ("bf16", True, True, LONG, 512, 1024),
    ("fp32", False, True, LONG, 512, 1024), ("fp32", False, True, SHORT[:36], 384, 896),
    ("fp32", False, False, SHORT, 512, 1024), ("fp32", True, False, SHORT, 384, 1024), ("fp32", True, False, LONG, 512, 1024),
]
