"""Sizes that send the 8-bit product and each product grouped by expert through every
tile shape of its rule for longer than the shape's LDS ring, with ragged rows,
columns and k.  The host test holds the rules to that, so that new costs cannot take a
shape out of the tests unnoticed."""
import torch

# M, N, K, each with bf16 and fp32 outputs
INT8 = [(1, 16, 2592), (1, 4656, 1312), (17, 4368, 1376), (34, 4768, 1312), (73, 5424, 672), (74, 5904, 736), (195, 4688, 608),
        (269, 4240, 544), (386, 4640, 672), (1335, 3248, 416), (1953, 6000, 1312), (1800, 7200, 480)]
# T, E, N, K, each with bf16 and fp32 outputs
GROUPED = [(1, 1, 16, 672), (1, 1, 16, 1632), (2, 1, 16, 1376), (1, 1, 16, 3296), (15, 12, 1776, 352), (8668, 21, 16, 288),
           (44, 12, 896, 544), (8408, 23, 16, 544), (50, 18, 1808, 352), (59, 34, 624, 672), (93, 40, 560, 1376),
           (131, 39, 512, 1696), (762, 15, 1840, 224), (8637, 1, 176, 224), (371, 16, 1904, 544), (2852, 37, 1088, 416),
           (3439, 40, 1440, 288), (7410, 6, 1424, 224), (7141, 34, 1040, 416), (5717, 2, 2480, 416)]
# T, E, N, K, each with bf16 and fp32 dw, both gradients and either alone
GROUPED_BWD = [(1, 1, 656, 32), (650, 1, 16, 32), (469, 34, 16, 992), (428, 28, 16, 1504), (12, 5, 352, 2016), (36, 11, 320, 1504),
               (15, 25, 224, 2400), (11, 6, 1248, 3104), (570, 36, 1696, 160), (267, 19, 208, 3360), (538, 28, 448, 928),
               (4162, 30, 224, 1824), (3941, 25, 2448, 224)]


def counts(T, E):
    """One expert takes half of the rows, the others what is left, some of them none."""
    if E == 1:
        return [T]
    big = T - T // 2
    g = torch.Generator().manual_seed(T + E)
    want = torch.rand(E, generator=g) * (torch.rand(E, generator=g) < 0.7)
    want[E // 3] = 0.0
    rest = torch.floor(want / want.sum().clamp(min=1e-6) * (T - big)).long()
    rest[E // 3] = T - int(rest.sum())
    return rest.tolist()
