"""The gated linear layer, the backward passes and MXFP4 on the GPU: against
64-bit references with derived bounds, bit for bit where the inputs make every
step exact, row by row across batch sizes, with strides, poisoned padding,
captured graphs and other streams, and as one feed-forward layer."""
import pytest

torch = pytest.importorskip("torch")

from tests import ffn_ref as ref
from tests.gpu_util import banner

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("deterministic_persistent_gemm_amd")
BF = torch.bfloat16
GATES = [0, 1]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, shape, std=1.0, dtype=BF):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def ints(g, shape, lo, hi, dtype=BF):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(dtype)


def padded(t, extra=8, fill=float("nan"), rows=3):
    """The same matrix as a view of a wider, longer buffer filled with `fill`."""
    buf = torch.full((t.shape[0] + rows, t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    v = buf[:t.shape[0], :t.shape[1]]
    v.copy_(t)
    return v, buf


def within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), float(err[bad][0]), float(bound[bad][0]))


def same(a, b, what=""):
    assert a.dtype == b.dtype and a.shape == b.shape, what
    bits = {2: torch.int16, 4: torch.int32, 1: torch.uint8}[a.element_size()]
    d = a.contiguous().view(bits) != b.contiguous().view(bits)
    assert not d.any(), (what, int(d.sum()), d.nonzero()[:4].tolist())


# Ms that reach every tile shape and its edges; layers with odd numbers of
# 16-wide and 32-wide steps
MS = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 129, 200, 255, 257, 511, 640]
LAYERS = [(32, 16), (96, 48), (256, 128), (544, 208), (2048, 768)]      # (H, I)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("H,I", LAYERS)
@pytest.mark.parametrize("M", [1, 5, 16, 33, 64, 130, 300, 513])
def test_gated_against_64_bits(M, H, I, gate):
    banner(f"gated M={M} H={H} I={I} gate={gate}")
    g = gen(M * 7 + H + I)
    x, w = randn(g, (M, H)), randn(g, (2 * I, H), 2.0 / H ** 0.5)
    y, h = bi.bi_gated_linear_bf16(x, w.t(), gate, save_h=True)
    wy, wh, by, bh = ref.gated(x, w, gate)
    within(h, wh, bh, "h")
    within(y, wy, by, "y")
    same(bi.bi_gated_linear_bf16(x, w.t(), gate), y, "y does not depend on h")


@pytest.mark.parametrize("H,I", LAYERS)
def test_gated_rows_do_not_depend_on_the_batch(H, I):
    g = gen(H + I)
    x, w = randn(g, (640, H)), randn(g, (2 * I, H), 2.0 / H ** 0.5)
    full, hfull = bi.bi_gated_linear_bf16(x, w.t(), save_h=True)
    for M in MS:
        banner(f"gated invariance M={M} H={H} I={I}")
        for at in {0, (640 - M) // 2, 640 - M}:
            y, h = bi.bi_gated_linear_bf16(x[at:at + M], w.t(), save_h=True)
            same(y, full[at:at + M], f"y M={M} at {at}")
            same(h, hfull[at:at + M], f"h M={M} at {at}")


@pytest.mark.parametrize("M,H,I", [(1, 4096, 4096), (8, 4096, 1536), (700, 4096, 2048), (1100, 1024, 4112), (2049, 512, 1040)])
def test_gated_large(M, H, I):
    banner(f"gated large M={M} H={H} I={I}")
    g = gen(M + H)
    x, w = randn(g, (M, H)), randn(g, (2 * I, H), 1.0 / H ** 0.5)
    y, h = bi.bi_gated_linear_bf16(x, w.t(), 1, save_h=True)
    wy, wh, by, bh = ref.gated(x, w, 1)
    within(h, wh, bh, "h")
    within(y, wy, by, "y")
    y1 = bi.bi_gated_linear_bf16(x[M - 1:], w.t(), 1)
    same(y1, y[M - 1:], "the last row alone")


# sizes that reach each tile shape of the gated layer with ragged rows, columns
# and k (one slice, an odd number of slices, more slices than a ring holds)
GATED_SHAPES = [(1, 480, 16), (1, 32, 16), (20, 96, 3536), (34, 96, 3024), (17, 32, 4560), (129, 544, 4560), (17, 32, 8496),
                (300, 352, 8496), (387, 32, 8752), (387, 96, 8752), (515, 672, 8752), (1030, 2080, 2064)]


@pytest.mark.parametrize("M,H,I", GATED_SHAPES)
def test_gated_every_tile_shape(M, H, I):
    """Integer operands: h is exact before its rounding, in every tile shape."""
    banner(f"gated shapes M={M} H={H} I={I}")
    g = gen(M + H + I)
    x, w = ints(g, (M, H), -3, 3), ints(g, (2 * I, H), -2, 2)
    xp, _ = padded(x)
    wp, _ = padded(w)
    y, h = bi.bi_gated_linear_bf16(xp, wp.t(), 1, save_h=True)
    wh = ref.mm(x, w.t().contiguous())
    same(h + 0.0, wh.to(BF) + 0.0, "h")
    wy = ref.act(wh[:, :I], 1)[0] * wh[:, I:]
    within(y, wy, (ref.HALF_BF16 + ref.ACT_REL) * (1 + ref.HALF_BF16) * wy.abs() + ref.TINY, "y")


@pytest.mark.parametrize("N,K", [(4096, 1024), (1536, 768), (8192, 352)])
def test_projections_equal_the_linear_layer(N, K):
    """h is what bi_linear_bf16 computes, bit for bit, where that key's recipe is
    fully chained: both thread one accumulator through k in the same order."""
    assert bi.bi_describe_recipe(bi.BI_BF16, N, K).block_k == K
    g = gen(N + K)
    x, w = randn(g, (600, K)), randn(g, (N, K), 0.05)
    for M in (1, 40, 600):
        banner(f"h against bi_linear_bf16 M={M} N={N} K={K}")
        same(bi.bi_gated_linear_bf16(x[:M], w.t(), save_h=True)[1], bi.bi_linear_bf16(x[:M], w.t()), f"M={M}")


def test_gated_extreme_projections():
    """act over the whole range: projections of the diagonal layer are the inputs."""
    H = I = 64
    w = torch.zeros((2 * I, H), dtype=BF, device="cuda")
    w[:I, :32] = torch.eye(32, dtype=BF, device="cuda").repeat(2, 1)[:I]
    w[I:, 32:] = torch.eye(32, dtype=BF, device="cuda").repeat(2, 1)[:I]
    x = torch.zeros((8, H), dtype=BF, device="cuda")
    vals = [0.0, -0.0, 1e-20, -1e-20, 5.0, -5.0, 40.0, -40.0, 100.0, -100.0, 3e4, -3e4, 1e30, -1e30, float("inf"), 88.7]
    x[:, :16] = torch.tensor(vals, dtype=BF)
    x[:, 32:] = 1.0
    x[:, :32] = torch.where(torch.isinf(x[:, :32]), torch.zeros_like(x[:, :32]), x[:, :32])
    for gate in GATES:
        y = bi.bi_gated_linear_bf16(x, w.t(), gate)
        want, _ = ref.act(x[:, :32].double(), gate)
        assert torch.isfinite(y).all()
        within(y[:, :32], want, ref.HALF_BF16 * want.abs() + ref.ACT_REL * want.abs() + 1e-30, f"gate {gate}")


@pytest.mark.parametrize("M,H,I", [(3, 96, 48), (65, 256, 128), (300, 544, 208)])
def test_gated_strides_and_poisoned_padding(M, H, I):
    banner(f"gated strides M={M} H={H} I={I}")
    g = gen(5)
    x, w = randn(g, (M, H)), randn(g, (2 * I, H), 0.1)
    y = bi.bi_gated_linear_bf16(x, w.t())
    xp, _ = padded(x, 40)
    wp, _ = padded(w, 8)
    op, obuf = padded(torch.zeros((M, I), dtype=BF, device="cuda"), 24, 7.0)
    same(bi.bi_gated_linear_bf16(xp, wp.t(), out=op), y, "padded")
    assert (obuf[M:] == 7.0).all() and (obuf[:, I:] == 7.0).all()
    # a row that is all NaN or infinite stays its own
    x2 = x.clone()
    x2[M - 1] = float("nan")
    y2 = bi.bi_gated_linear_bf16(x2, w.t())
    same(y2[:M - 1], y[:M - 1], "neighbours of a NaN row")
    assert torch.isnan(y2[M - 1]).all()


# ------------------------------------------------------------------ backward

BWD = [(1, 32, 32), (1, 544, 64), (7, 96, 64), (31, 64, 96), (32, 128, 128), (33, 208, 160), (65, 272, 288), (130, 512, 96),
       (300, 2048, 768), (333, 1040, 544), (1000, 256, 512), (2050, 144, 96)]           # M, N, K


# sizes that reach every pair of tile shapes in one launch, and two launches
BWD_SHAPES = [(1, 272, 2784), (1, 272, 4192), (1, 80, 4128), (89, 80, 4128), (1, 272, 3424), (1, 400, 4192), (133, 496, 4128),
              (226, 1712, 4000), (1304, 1552, 3360), (135, 4016, 2016), (41, 3728, 3552), (235, 4048, 3872), (1442, 432, 2400),
              (2569, 144, 4128), (807, 816, 4256), (996, 3184, 3616), (4100, 48, 8160),
              (84, 1440, 672), (29, 1984, 96), (17, 2064, 544), (5, 8208, 32), (2, 2864, 4000),
              (33, 80, 2752), (134, 736, 1632), (69, 480, 1632), (65, 528, 2496), (551, 3488, 768)]


@pytest.mark.parametrize("M,N,K", BWD + BWD_SHAPES)
def test_linear_bwd_exact_on_integers(M, N, K):
    """Small integers: every product and sum is exact, so is the fp32 result."""
    banner(f"linear_bwd ints M={M} N={N} K={K}")
    g = gen(M + N + K)
    dy, x, w = ints(g, (M, N), -3, 3), ints(g, (M, K), -3, 3), ints(g, (N, K), -3, 3)
    dx, dw, db = bi.bi_linear_bf16_bwd(dy, x, w.t(), dw_dtype=torch.float32)
    same(dx + 0.0, ref.mm(dy, w).to(BF) + 0.0, "dx")
    same(dw + 0.0, ref.mm(dy.t().contiguous(), x).float(), "dw")
    same(db + 0.0, dy.double().sum(0).float(), "db")
    same(bi.bi_linear_bf16_bwd(dy, x, w.t())[1] + 0.0, ref.mm(dy.t().contiguous(), x).to(BF), "dw bf16")
    # each gradient alone takes its own shape
    same(bi.bi_linear_bf16_bwd(dy, None, w.t(), need_dw=False, need_db=False)[0], dx, "dx alone")
    same(bi.bi_linear_bf16_bwd(dy, x, None, need_dx=False, need_db=False, dw_dtype=torch.float32)[1], dw, "dw alone")
    same(bi.bi_linear_bf16_bwd(dy, None, None, need_dx=False, need_dw=False)[2], db, "db alone")


@pytest.mark.parametrize("M,N,K", [(1, 528, 512), (16, 4096, 4096), (333, 2048, 768), (700, 80, 64), (1000, 1040, 1024),
                                   (1031, 2064, 2080), (4100, 272, 32)])
def test_linear_bwd_column_sums(M, N, K):
    """db by dw's tiles and by workgroups of its own, beside both gradients, one
    and none; small integers, so that every order of adding is exact."""
    banner(f"linear_bwd sums M={M} N={N} K={K}")
    g = gen(M + N + K)
    dy, x, w = ints(g, (M, N), -3, 3), ints(g, (M, K), -3, 3), ints(g, (N, K), -3, 3)
    want = dy.double().sum(0).float()
    for kw in (dict(), dict(need_dx=False), dict(need_dw=False), dict(need_dx=False, need_dw=False),
               dict(dw_dtype=torch.float32)):
        same(bi.bi_linear_bf16_bwd(dy, x, w.t(), **kw)[2] + 0.0, want, f"db {kw}")


@pytest.mark.parametrize("M,N,K", BWD)
def test_linear_bwd_against_64_bits(M, N, K):
    banner(f"linear_bwd M={M} N={N} K={K}")
    g = gen(M + N + K)
    dy, x, w = randn(g, (M, N), 0.01), randn(g, (M, K)), randn(g, (N, K), 0.1)
    dyp, xp, wp = padded(dy)[0], padded(x, 16)[0], padded(w, 24)[0]
    dx, dw, db = bi.bi_linear_bf16_bwd(dyp, xp, wp.t(), dw_dtype=torch.float32)
    want = ref.mm(dy, w)
    within(dx, want, ref.stored(ref.sum_bound(dy, w, N), want, BF), "dx")
    t = dy.t().contiguous()
    want = ref.mm(t, x)
    within(dw, want, ref.stored(ref.sum_bound(t, x, M), want, torch.float32), "dw")
    want = dy.double().sum(0)
    within(db, want, (M + 1) * ref.HALF_F32 * dy.double().abs().sum(0) + ref.TINY, "db")
    dx2, dw2, db2 = bi.bi_linear_bf16_bwd(dy, x, w.t(), dw_dtype=torch.float32)
    same(dx, dx2), same(dw, dw2), same(db, db2)


def test_linear_bwd_rows_do_not_depend_on_the_batch():
    g = gen(3)
    for N, K in ((96, 64), (1040, 544), (4096, 768)):
        dy, w = randn(g, (640, N)), randn(g, (N, K), 0.1)
        full = bi.bi_linear_bf16_bwd(dy, None, w.t(), need_dw=False, need_db=False)[0]
        for M in MS:
            banner(f"dx invariance M={M} N={N} K={K}")
            for at in {0, 640 - M}:
                dx, dw, db = bi.bi_linear_bf16_bwd(dy[at:at + M], None, w.t(), need_dw=False, need_db=False)
                assert dw is None and db is None
                same(dx, full[at:at + M], f"M={M} at {at}")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("M,H,I", [(1, 32, 16), (5, 96, 48), (33, 256, 128), (200, 2048, 768), (513, 544, 208)])
def test_gated_bwd_against_64_bits(M, H, I, gate):
    banner(f"gated_bwd M={M} H={H} I={I} gate={gate}")
    g = gen(M + H + I)
    dy, x, w = randn(g, (M, I), 0.01), randn(g, (M, H)), randn(g, (2 * I, H), 0.05)
    h = randn(g, (M, 2 * I), 2.0)
    dx, dw = bi.bi_gated_linear_bf16_bwd(dy, x, w.t(), h, gate, dw_dtype=torch.float32)
    wx, ww, ex, ew = ref.gated_bwd(dy, x, w, h, gate)
    within(dx, wx, ref.stored(ex, wx, BF), "dx")
    within(dw, ww, ref.stored(ew, ww, torch.float32), "dw")
    # one gradient alone, padded inputs, and the bf16 weight gradient: the same values
    dyp, xp, wp, hp = padded(dy)[0], padded(x)[0], padded(w)[0], padded(h)[0]
    same(bi.bi_gated_linear_bf16_bwd(dyp, None, wp.t(), hp, gate, need_dw=False)[0], dx, "dx alone")
    same(bi.bi_gated_linear_bf16_bwd(dyp, xp, None, hp, gate, need_dx=False)[1], dw.to(BF), "dw alone, bf16")


@pytest.mark.parametrize("gate", GATES)
def test_gated_bwd_elementwise_part(gate):
    """With an identity weight, dx is dh itself: the activation's derivative over
    its range, rounded twice (dh, then dx of one product)."""
    I = 64
    g = torch.linspace(-20, 20, 8 * I, device="cuda").reshape(8, I).to(BF)
    u = randn(gen(1), (8, I))
    h = torch.cat((g, u), dim=1)
    dy = randn(gen(2), (8, I))
    eye = torch.eye(2 * I, dtype=BF, device="cuda")
    dx, _ = bi.bi_gated_linear_bf16_bwd(dy, None, eye.t(), h, gate, need_dw=False)
    want = ref.gate_bwd(dy, h, gate)
    slack = torch.cat((dy.double().abs() * u.double().abs() * (g.double().abs() + 1), dy.double().abs() * g.double().abs()), 1)
    within(dx, want, ref.HALF_BF16 * want.abs() + 2 * ref.ACT_REL * slack + 1e-30, "dh")


@pytest.mark.parametrize("gate", GATES)
def test_gated_bwd_large_projections(gate):
    """Projections whose square or cube passes fp32's range: act' is 1 or 0 there."""
    I = 64
    vals = [1e10, 1e13, 1e19, 2e19, 1e20, 1e25, 1e30, 3e38]
    g = torch.tensor(vals + [-v for v in vals], dtype=BF, device="cuda").repeat(2, I // 16)
    h = torch.cat((g, torch.full_like(g, 2.0)), dim=1)
    dy = torch.ones_like(g)
    eye = torch.eye(2 * I, dtype=BF, device="cuda")
    dx, _ = bi.bi_gated_linear_bf16_bwd(dy, None, eye.t(), h, gate, need_dw=False)
    same(dx, ref.gate_bwd(dy, h, gate).to(BF) + 0.0, "dh")


def test_gated_gradients_against_differences():
    """The layer's own forward pass, differenced: sum(y * dy) along random
    directions of x and w, in steps large enough for bf16 y."""
    M, H, I = 16, 256, 128
    g = gen(11)
    x, w = randn(g, (M, H), 1.0), randn(g, (2 * I, H), 1 / 16)
    dy = randn(g, (M, I))
    _, h = bi.bi_gated_linear_bf16(x, w.t(), 0, save_h=True)
    dx, dw = bi.bi_gated_linear_bf16_bwd(dy, x, w.t(), h, 0, dw_dtype=torch.float32)
    # along the gradient itself, so that the difference is large against y's rounding:
    # y's error is at most 2^-8 |y| per element, and they add at random signs or worse
    for which, grad in (("x", dx.double()), ("w", dw.double())):
        base = (x if which == "x" else w).double()
        step = 0.05 * base.norm() / grad.norm()
        a, b = (base + step * grad).to(BF), (base - step * grad).to(BF)
        move = a.double() - b.double()                      # what the rounding left of the step
        ya = bi.bi_gated_linear_bf16(a if which == "x" else x, (a if which == "w" else w).t(), 0).double()
        yb = bi.bi_gated_linear_bf16(b if which == "x" else x, (b if which == "w" else w).t(), 0).double()
        got, want = float(((ya - yb) * dy.double()).sum()), float((move * grad).sum())
        noise = 2.0 ** -8 * float(((ya.abs() + yb.abs()) * dy.double().abs()).sum())
        assert noise < 0.2 * want, (which, noise, want)
        # third-order terms: |step|^2 of a smooth layer, bounded by 5 percent at this step
        assert abs(got - want) <= noise + 0.05 * want, (which, got, want, noise)


def test_empty_batches():
    H, I = 64, 32
    w = torch.ones((2 * I, H), dtype=BF, device="cuda")
    x0 = torch.empty((0, H), dtype=BF, device="cuda")
    y, h = bi.bi_gated_linear_bf16(x0, w.t(), save_h=True)
    assert y.shape == (0, I) and h.shape == (0, 2 * I)
    dx, dw = bi.bi_gated_linear_bf16_bwd(y, x0, w.t(), h, dw_dtype=torch.float32)
    assert dx.shape == (0, H) and dw.shape == (2 * I, H) and not dw.any()
    dx, dw, db = bi.bi_linear_bf16_bwd(h, x0, w.t())
    assert dx.shape == (0, H) and not dw.any() and not db.any() and db.shape == (2 * I,)
    q, s = bi.bi_quantize_mxfp4(x0)
    assert q.shape == (0, H // 2) and s.shape == (0, H // 32)
    wq, ws = bi.bi_quantize_mxfp4(w)
    assert bi.bi_linear_mxfp4(q, s, wq, ws).shape == (0, 2 * I)
    assert bi.bi_dequantize_mxfp4(q, s).shape == (0, H)


# --------------------------------------------------------------------- MXFP4


def mx_check(x):
    q, s = bi.bi_quantize_mxfp4(x)
    code, sc = ref.mx_quantize(x)
    assert torch.equal(s.cpu().long(), sc.long()), "scales"
    assert torch.equal(ref.unpack(q), code), "codes"
    vals = ref.mx_values(code, sc)
    for dt in (BF, torch.float32):
        got = bi.bi_dequantize_mxfp4(q, s, dt).cpu()
        same(torch.nan_to_num(got, nan=77.0), torch.nan_to_num(vals.to(dt), nan=77.0), f"values {dt}")


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (16, 4096), (129, 544), (1000, 256)])
def test_quantize(M, K, dtype):
    banner(f"quantize M={M} K={K} {dtype}")
    g = gen(M + K)
    x = randn(g, (M, K), 1.0, torch.float32) * torch.exp(4 * torch.randn((M, 1), generator=g, device="cuda"))
    mx_check(x.to(dtype))
    mx_check(padded(x.to(dtype), 16 if dtype == BF else 8)[0])


def test_quantize_ties_specials_and_range():
    # every midpoint and its neighbours under several scales, both signs
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.999]
    row = []
    for m in mids:
        row += [m, m * (1 + 2 ** -20), m * (1 - 2 ** -20)]
    row = (row + [4.0, 0.0])[:32]
    row[31] = 4.5                                             # the block's scale is 1
    base = torch.tensor([row], dtype=torch.float32)
    rows = [base * s * 2.0 ** e for s in (1, -1) for e in (-140, -126, -120, -60, 0, 60, 120)]
    mx_check(torch.cat(rows).cuda())
    z = torch.zeros((6, 64), dtype=torch.float32)
    z[0, 3] = float("inf")
    z[1, 40] = float("nan")
    z[2, 5] = -float("inf")
    z[2, 6] = 1.0
    z[3, 0] = 2.0 ** -149                                     # the smallest subnormal alone
    z[4, 33] = 3.4e38
    z[5, 1] = -0.0
    mx_check(z.cuda())
    zb = z.to(BF)
    zb[4, 33] = 3.3e38
    mx_check(zb.cuda())


MX = [(1, 16, 32), (1, 48, 96), (5, 32, 128), (16, 256, 544), (17, 272, 1024), (64, 64, 160), (65, 528, 416), (130, 1040, 256),
      (300, 768, 2048), (1, 4096, 4096), (1030, 512, 672), (17, 6160, 32), (33, 5392, 32), (258, 6288, 32), (258, 6288, 416),
      (915, 8720, 32), (915, 8720, 160), (700, 8720, 672), (900, 8720, 1184), (1030, 2064, 1184)]    # M, N, K


@pytest.mark.parametrize("M,N,K", MX)
def test_mxfp4_exact(M, N, K):
    """Codes under scales 1 and 2: products are multiples of 1/4 below 144, sums exact in fp32."""
    banner(f"mxfp4 exact M={M} N={N} K={K}")
    g = gen(M + N + K)
    ops = []
    for rows in (M, N):
        code = torch.randint(0, 16, (rows, K), generator=g, device="cuda").cpu()
        s = torch.randint(127, 129, (rows, K // 32), generator=g, device="cuda").cpu()
        pad = torch.full((rows, (K // 32 + 3) // 4 * 4), 255, dtype=torch.uint8)       # past K: must not matter
        pad[:, :K // 32] = s
        ops += [ref.pack(code).cuda(), pad.cuda()[:, :K // 32], ref.mx_values(code, s).cuda()]
    xq, xs, xv, wq, ws, wv = ops
    bias = ints(g, (N,), -5, 5, torch.float32)
    want = torch.mm(xv, wv.t().contiguous())
    y = bi.bi_linear_mxfp4(xq, xs, wq, ws, out_dtype=torch.float32)
    same(y + 0.0, want.float() + 0.0, "fp32")
    same(bi.bi_linear_mxfp4(xq, xs, wq, ws, bias) + 0.0, (want + bias).to(BF) + 0.0, "bf16 with bias")
    # each row alone, and padded operands
    for m in {0, M // 2, M - 1}:
        same(bi.bi_linear_mxfp4(xq[m:m + 1], xs[m:m + 1], wq, ws, out_dtype=torch.float32), y[m:m + 1], f"row {m}")
    xqp, wqp = padded(xq, 16, 255)[0], padded(wq, 32, 255)[0]
    same(bi.bi_linear_mxfp4(xqp, xs, wqp, ws, out_dtype=torch.float32), y, "padded")


@pytest.mark.parametrize("N,K", [(272, 544), (1024, 2048), (4096, 1536)])
def test_mxfp4_against_64_bits_and_across_batches(N, K):
    g = gen(N)
    x, w = randn(g, (640, K)), randn(g, (N, K), 0.05)
    xq, xs = bi.bi_quantize_mxfp4(x)
    wq, ws = bi.bi_quantize_mxfp4(w)
    full = bi.bi_linear_mxfp4(xq, xs, wq, ws, out_dtype=torch.float32)
    xv, wv = bi.bi_dequantize_mxfp4(xq, xs, torch.float32), bi.bi_dequantize_mxfp4(wq, ws, torch.float32)
    wvt = wv.t().contiguous()
    want = ref.mm(xv, wvt)
    within(full, want, ref.stored(ref.sum_bound(xv, wvt, K), want, torch.float32), "y")
    for M in MS:
        banner(f"mxfp4 invariance M={M} N={N} K={K}")
        for at in {0, 640 - M}:
            same(bi.bi_linear_mxfp4(xq[at:at + M], xs[at:at + M], wq, ws, out_dtype=torch.float32), full[at:at + M], f"M={M}")


def test_mxfp4_nan_blocks():
    """A NaN block makes its row (of x) or its column (of w) NaN and nothing else."""
    g = gen(4)
    x, w = randn(g, (20, 256)), randn(g, (48, 256))
    y = bi.bi_linear_mxfp4(*bi.bi_quantize_mxfp4(x), *bi.bi_quantize_mxfp4(w))
    x[7, 100] = float("nan")
    w[33, 200] = float("inf")
    z = bi.bi_linear_mxfp4(*bi.bi_quantize_mxfp4(x), *bi.bi_quantize_mxfp4(w))
    bad = torch.zeros((20, 48), dtype=torch.bool, device="cuda")
    bad[7, :] = True
    bad[:, 33] = True
    assert torch.equal(torch.isnan(z), bad)
    same(torch.where(bad, torch.zeros_like(z), z), torch.where(bad, torch.zeros_like(y), y))


# -------------------------------------------------- streams, graphs, a whole layer


def far(t, pitch):
    """t's values in rows `pitch` elements apart; the buffer passes 4 GiB."""
    assert t.shape[0] * pitch * t.element_size() > 1 << 32
    buf = torch.empty((t.shape[0], pitch), dtype=t.dtype, device="cuda")
    out = buf[:, :t.shape[1]]
    out.copy_(t)
    return out


@pytest.mark.parametrize("M,H,I", [(300, 96, 304), (300, 96, 3536), (515, 672, 8752)])
def test_offsets_past_32_bits_gated(M, H, I):
    """Rows as far apart as the calls take them: the same bits as packed ones."""
    banner(f"far rows gated M={M} H={H} I={I}")
    g = gen(M)
    x, w, dy = randn(g, (M, H)), randn(g, (2 * I, H), 0.1), randn(g, (M, I))
    y, h = bi.bi_gated_linear_bf16(x, w.t(), save_h=True)
    pitch = (1 << 23) - 1024                                        # 255 rows and the last row's end: below 4 GiB
    xf = far(x, pitch)
    yf = far(torch.zeros_like(y), pitch)
    bi.bi_gated_linear_bf16(xf, w.t(), out=yf)
    same(yf, y, "x, y")
    del yf
    wp = ((1 << 32) // (I + 256) // 2 - H) // 8 * 8
    if 2 * I * wp * 2 > 1 << 32:
        same(bi.bi_gated_linear_bf16(x, far(w, wp).t()), y, "w")
    dx, dw = bi.bi_gated_linear_bf16_bwd(dy, x, w.t(), h)
    dxf, dwf = bi.bi_gated_linear_bf16_bwd(far(dy, pitch), xf, w.t(), far(h, pitch))
    same(dxf, dx, "dx")
    same(dwf, dw, "dw")


def test_offsets_past_32_bits_linear_bwd():
    M, N, K = 300, 272, 288
    g = gen(3)
    dy, x, w = randn(g, (M, N)), randn(g, (M, K)), randn(g, (N, K))
    pitch = (1 << 23) - 1024
    want = bi.bi_linear_bf16_bwd(dy, x, w.t())
    got = bi.bi_linear_bf16_bwd(far(dy, pitch), far(x, pitch), far(w, pitch).t())
    for a, b, what in zip(got, want, ("dx", "dw", "db")):
        same(a, b, what)


@pytest.mark.parametrize("M,N,K", [(300, 272, 96), (300, 3536, 2080)])
def test_offsets_past_32_bits_mxfp4(M, N, K):
    g = gen(4)
    x, w = randn(g, (M, K)), randn(g, (N, K))
    q, s = bi.bi_quantize_mxfp4(x)
    wq, ws = bi.bi_quantize_mxfp4(w)
    pitch = (1 << 24) - 2048                                        # bytes
    xf = far(x, pitch // 2)
    qf, sf = bi.bi_quantize_mxfp4(xf)
    same(qf, q, "codes")
    same(sf, s, "scales")
    y = bi.bi_linear_mxfp4(q, s, wq, ws)
    same(bi.bi_linear_mxfp4(far(q, pitch), far(s, pitch), wq, ws, out=far(torch.zeros_like(y), pitch)), y, "y")
    same(bi.bi_dequantize_mxfp4(far(q, pitch), far(s, pitch)), bi.bi_dequantize_mxfp4(q, s), "values")


def test_other_stream_and_shared_weights():
    g = gen(8)
    x, w = randn(g, (100, 256)), randn(g, (256, 256), 0.1)
    y = bi.bi_gated_linear_bf16(x, w.t())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y2 = bi.bi_gated_linear_bf16(x, w.t())
        dx2, dw2, db2 = bi.bi_linear_bf16_bwd(x, x, w.t())
    s.synchronize()
    same(y, y2)
    for a, b in zip((dx2, dw2, db2), bi.bi_linear_bf16_bwd(x, x, w.t())):
        same(a, b)


def train_layer(x, w13, w2, dout):
    """One feed-forward layer forward and backward through the public calls."""
    a, h = bi.bi_gated_linear_bf16(x, w13.t(), save_h=True)
    out = bi.bi_linear_bf16(a, w2.t())
    da, dw2, _ = bi.bi_linear_bf16_bwd(dout, a, w2.t(), need_db=False)
    dx, dw13 = bi.bi_gated_linear_bf16_bwd(da, x, w13.t(), h)
    return out, dx, dw13, dw2


def serve_layer(x, q13, q2, I):
    """The same layer from 4-bit weights."""
    h = bi.bi_linear_mxfp4(*bi.bi_quantize_mxfp4(x), *q13)
    a = (torch.nn.functional.silu(h[:, :I].float()) * h[:, I:].float()).to(BF)
    return bi.bi_linear_mxfp4(*bi.bi_quantize_mxfp4(a), *q2)


def layer(seed, M=70, H=256, I=160):
    g = gen(seed)
    return randn(g, (M, H)), randn(g, (2 * I, H), 1 / 16), randn(g, (H, I), 1 / 12), randn(g, (M, H), 0.1)


def test_a_layer_trained_and_served():
    x, w13, w2, dout = layer(21)
    M, I = x.shape[0], w2.shape[1]
    out, dx, dw13, dw2 = train_layer(x, w13, w2, dout)
    # the same graph by torch in 64 bits; the bounds compound, so hold the 2-norms to
    # the roundings in each path: a and out (2), da, dh and the gradient (3) at 2^-8 each
    leaves = [t.double().requires_grad_() for t in (x, w13, w2)]
    hh = leaves[0] @ leaves[1].t()
    o = (ref.act(hh[:, :I], 0)[0] * hh[:, I:]) @ leaves[2].t()
    o.backward(dout.double())
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(out, o.detach()) < 2 * ref.HALF_BF16
    for got, leaf, n in ((dx, leaves[0], 4), (dw13, leaves[1], 4), (dw2, leaves[2], 2)):
        assert rel(got, leaf.grad) < n * ref.HALF_BF16
    # served in 4 bits: rows do not depend on the batch
    q13, q2 = bi.bi_quantize_mxfp4(w13), bi.bi_quantize_mxfp4(w2)
    served = serve_layer(x, q13, q2, I)
    for m in (0, 33, M - 1):
        same(serve_layer(x[m:m + 1], q13, q2, I), served[m:m + 1], f"row {m}")


def test_two_graphs_replayed_between_eager_work():
    """Two captures of the layer, replayed several times in turn with eager calls
    between: every replay equals the eager result on the inputs of the moment."""
    ins = [layer(31), layer(32, M=33)]
    q = [(bi.bi_quantize_mxfp4(t[1]), bi.bi_quantize_mxfp4(t[2])) for t in ins]
    both = lambda k: train_layer(*ins[k]) + (serve_layer(ins[k][0], *q[k], ins[k][2].shape[1]),)
    for k in (0, 1):
        both(k)
    torch.cuda.synchronize()
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for k in (0, 1):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            outs.append(both(k))
        graphs.append(gr)
    for rep in range(4):
        for k in (0, 1):
            ins[k][0].copy_(randn(gen(100 * rep + k), tuple(ins[k][0].shape)))
        graphs[rep % 2].replay()
        graphs[1 - rep % 2].replay()
        for k in (0, 1):
            for a, b in zip(outs[k], both(k)):
                same(a, b, f"replay {rep}, graph {k}")
        torch.cuda.synchronize()


def test_results_repeat():
    g = gen(77)
    dy, x, w = randn(g, (777, 1040)), randn(g, (777, 544)), randn(g, (1040, 544))
    first = bi.bi_linear_bf16_bwd(dy, x, w.t(), dw_dtype=torch.float32)
    for _ in range(5):
        for a, b in zip(first, bi.bi_linear_bf16_bwd(dy, x, w.t(), dw_dtype=torch.float32)):
            same(a, b)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 40])
def test_gated_projections_whose_sigmoid_is_subnormal(gate, scale):
    """act is still a normal fp32 number where its sigmoid is below fp32's normal
    range.  Projections are the inputs (one product each), u is `scale`.  Values of
    act below 2^-127 and of act' below 2^-125 may count as zero; above, relative bounds."""
    H = I = 64
    lo, hi, step = ((-92.5, -77.0, 0.5), (-10.75, -9.8125, 0.0625))[gate]
    vals = torch.arange(lo, hi + step / 2, step, dtype=torch.float64)[:32]
    w = torch.zeros((2 * I, H), dtype=BF, device="cuda")
    w[:32, :32] = torch.eye(32, dtype=BF, device="cuda")
    w[I:, 32] = scale
    x = torch.zeros((40, H), dtype=BF, device="cuda")
    x[:, :len(vals)] = vals.to(BF).cuda()
    assert torch.equal(x[0, :len(vals)].double().cpu(), vals), "the values are bf16 numbers"
    x[:, 32] = 1.0
    a, da = ref.act(x[:, :32].double(), gate)
    y, h = bi.bi_gated_linear_bf16(x, w.t(), gate, save_h=True)
    # bf16 steps below 2^-126 are 2^-133
    within(y[:, :32], a * scale, (ref.HALF_BF16 + ref.ACT_REL) * a.abs() * scale + 2.0 ** -127 * scale + 2.0 ** -134, "y")
    # dh by an identity weight, dy as large as u: both halves, rounded twice
    dy = torch.full((40, I), 2.0 ** 20, dtype=BF, device="cuda")
    eye = torch.eye(2 * I, dtype=BF, device="cuda")
    dx, _ = bi.bi_gated_linear_bf16_bwd(dy, None, eye.t(), h, gate, need_dw=False)
    wg, wu = da * scale * 2.0 ** 20, a * 2.0 ** 20
    g = x[:, :32].double()
    within(dx[:, :32], wg, ref.HALF_BF16 * wg.abs() + 2 * ref.ACT_REL * wg.abs() + 2.0 ** -125 * scale * 2.0 ** 20, "dh gate")
    within(dx[:, I:I + 32], wu, ref.HALF_BF16 * wu.abs() + 2 * ref.ACT_REL * wu.abs() + 2.0 ** -127 * 2.0 ** 20, "dh up")


@pytest.mark.parametrize("rows,K", [(1, 32), (1, 96), (3, 96), (5, 544)])
def test_dequantize_scales_that_end_inside_a_word(rows, K):
    """Dequantisation reads single scale bytes: the last row may end at its last
    one.  The product reads words and refuses such scales."""
    q, s = bi.bi_quantize_mxfp4(randn(gen(rows + K), (rows, K)))
    pitch, kb = s.stride(0), K // 32
    tight = torch.empty((rows - 1) * pitch + kb, dtype=torch.uint8, device="cuda")
    st = tight.as_strided((rows, kb), (pitch, 1))
    st.copy_(s)
    for dt in (BF, torch.float32):
        same(bi.bi_dequantize_mxfp4(q, st, dt), bi.bi_dequantize_mxfp4(q, s, dt))
    wq, ws = bi.bi_quantize_mxfp4(randn(gen(1), (16, K)))
    with pytest.raises(ValueError, match="32-bit words"):
        bi.bi_linear_mxfp4(q, st, wq, ws)
