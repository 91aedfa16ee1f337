"""Sizes that send each feed-forward product through every tile shape of its rule
for longer than the shape's LDS ring (4-bit: than its ring of scales too), with
ragged rows, columns and k.  The host test holds the rule to that, so that new
costs cannot take a shape out of the tests unnoticed."""

# M, I, H
GATED = [(7, 48, 1312), (13, 2352, 672), (50, 1328, 736), (103, 1216, 672), (160, 1648, 352), (137, 4128, 352), (902, 4128, 224)]
# M, N, K, each with bf16 and fp32 outputs
MXFP4 = [(13, 48, 5216), (9, 4752, 2752), (67, 2384, 3392), (77, 4848, 2784), (65, 5520, 2720), (245, 10144, 2144), (1668, 5872, 2080),
         (1049, 7984, 2144)]
# M, N, K, each with bf16 and fp32 dw
LINEAR_BWD = [(84, 1440, 672), (442, 544, 480), (105, 1648, 1120), (1, 400, 2848), (1, 736, 4064), (40, 816, 4000), (148, 400, 4128),
              (275, 656, 7520), (1304, 1552, 3360), (5, 8208, 32), (35, 416, 1568), (342, 80, 96), (389, 2576, 160), (408, 1968, 160),
              (353, 3872, 224), (344, 1424, 480), (227, 1040, 3904)]
