"""Sizes that send the 8-bit product and each product grouped by expert through every
tile shape of its rule for longer than the shape's LDS ring, with ragged rows,
columns and k.  The host test holds the rules to that, so that new costs cannot take a
shape out of the tests unnoticed."""
import torch

# M, N, K, each with bf16 and fp32 outputs
INT8 = [(1, 16, 2592), (1, 4656, 1312), (17, 4368, 1376), (34, 4768, 1312), (73, 5424, 672), (74, 5904, 736), (195, 4688, 608),
        (269, 4240, 544), (386, 4640, 672), (1335, 3248, 416), (1953, 6000, 1312), (1800, 7200, 480)]
# T, E, N, K, each with bf16 and fp32 outputs
GROUPED = [(1, 1, 16, 672), (1, 1, 16, 1632), (1, 1, 16, 3296), (114, 40, 80, 672), (3, 2, 2064, 1376), (30, 15, 1120, 352),
           (15, 12, 1776, 352), (8668, 21, 16, 288), (8408, 23, 16, 544), (50, 35, 592, 672), (3162, 29, 48, 544),
           (26, 18, 1072, 1056), (31, 18, 1600, 800), (4695, 5, 160, 352), (4406, 27, 144, 672), (4394, 10, 448, 224),
           (2018, 33, 928, 224), (2852, 37, 1088, 416), (3439, 40, 1440, 288), (7410, 6, 1424, 224),
           (5717, 2, 2480, 416)]
# T, E, N, K, each with bf16 and fp32 dw, both gradients and either alone
GROUPED_BWD = [(1, 1, 656, 32), (650, 1, 16, 32), (469, 34, 16, 992), (422, 25, 16, 1440), (11, 3, 336, 2848), (36, 11, 320, 1504),
               (22, 18, 688, 736), (245, 32, 432, 928), (1944, 32, 144, 1952), (8602, 3, 208, 416),
               (4162, 30, 224, 1824), (7432, 21, 960, 736)]


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
