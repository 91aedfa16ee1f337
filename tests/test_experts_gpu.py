"""Products grouped by expert, forward and backward, and 8-bit products on the GPU
against 64-bit forms."""
import pytest

torch = pytest.importorskip("torch")

from tests import experts_ref as ref
from tests import experts_shapes as shapes
from tests import ffn_ref
from tests.gpu_util import banner

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bi():
    import deterministic_persistent_gemm_amd as m
    return m


def ints(shape, seed, lo=-2, hi=2):
    """Small integers: every sum of products is exact in fp32."""
    return torch.randint(lo, hi + 1, shape, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


def normal(shape, seed, dtype=BF, std=1.0):
    return (std * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def ends_of(counts):
    return torch.cumsum(torch.tensor(counts), 0).cuda()


def forward_ref(x, w, ends):
    """y in binary64; rows of no expert are NaN."""
    xd, wd = x.double().cpu(), w.double().cpu()
    y = torch.full((x.shape[0], w.shape[1]), float("nan"), dtype=torch.float64)
    for e, (a, b) in enumerate(ref.spans(ends.tolist(), x.shape[0])):
        y[a:b] = xd[a:b] @ wd[e].t()
    return y


def same_rows(got, want):
    """Equal where the reference has a value."""
    has = ~torch.isnan(want[:, 0])
    assert torch.equal(got.cpu()[has], want[has].to(got.dtype))


# rows per expert: none at the ends and between, one, around tile heights, one expert
SPLITS = [[0, 1, 0, 0, 5, 17, 0], [16, 15, 33, 64, 65], [300, 0, 7], [1], [0, 0, 0], [130, 1, 1, 259, 0, 31]]
# an odd number of tiles, k with a ragged slice
SIZES = [(16, 32), (48, 96), (144, 288), (272, 64)]


@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("counts", SPLITS, ids=lambda c: "-".join(map(str, c)))
def test_grouped_forward_is_exact_on_integers(bi, counts, N, K):
    T, E = sum(counts), len(counts)
    for tail in (0, 9):
        banner(f"grouped {counts} N={N} K={K} tail={tail}")
        x, w, ends = ints((T + tail, K), 1), ints((E, N, K), 2), ends_of(counts)
        want = forward_ref(x, w, ends)
        for dt in (BF, F32):
            out = torch.full((T + tail, N), 7.0, dtype=dt, device="cuda")
            assert bi.bi_grouped_linear_bf16(x, w, ends, out=out) is out
            same_rows(out, want)
            assert (out[T:] == 7.0).all()
            same_rows(bi.bi_grouped_linear_bf16(x, w, ends, out_dtype=dt), want)


@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("counts", SPLITS, ids=lambda c: "-".join(map(str, c)))
def test_grouped_backward_is_exact_on_integers(bi, counts, N, K):
    T, E = sum(counts), len(counts)
    for tail in (0, 5):
        banner(f"grouped backward {counts} N={N} K={K} tail={tail}")
        dy, x, w, ends = ints((T + tail, N), 3), ints((T + tail, K), 1), ints((E, N, K), 2), ends_of(counts)
        want_dx = forward_ref(dy, w.transpose(1, 2), ends)
        want_dw = torch.zeros((E, N, K), dtype=torch.float64)
        for e, (a, b) in enumerate(ref.spans(ends.tolist(), T)):
            want_dw[e] = dy[a:b].double().cpu().t() @ x[a:b].double().cpu()
        for dt in (BF, F32):
            own = torch.full((T + tail, K), 7.0, dtype=BF, device="cuda")
            dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, dw_dtype=dt, out_dx=own)
            assert dx is own and dw.dtype == dt
            same_rows(dx, want_dx)
            assert (dx[T:] == 7.0).all()
            assert torch.equal(dw.cpu(), want_dw.to(dt))
        only, none = bi.bi_grouped_linear_bf16_bwd(dy, None, w, ends, need_dw=False)
        assert none is None
        same_rows(only, want_dx)
        none, only = bi.bi_grouped_linear_bf16_bwd(dy, x, None, ends, need_dx=False)
        assert none is None and torch.equal(only.cpu(), want_dw.to(BF))


def test_grouped_values_within_their_bounds(bi):
    counts, N, K = [37, 0, 411, 2, 150], 352, 736
    T, E, ends = sum(counts), len(counts), ends_of(counts)
    x, w, dy = normal((T, K), 1), normal((E, N, K), 2, std=K ** -0.5), normal((T, N), 3, std=0.01)
    y = bi.bi_grouped_linear_bf16(x, w, ends)
    y32 = bi.bi_grouped_linear_bf16(x, w, ends, out_dtype=F32)
    dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends)
    _, dw32 = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, need_dx=False, dw_dtype=F32)
    for e, (a, b) in enumerate(ref.spans(ends.tolist(), T)):
        xe, we, de = x[a:b].cpu(), w[e].cpu(), dy[a:b].cpu()
        for got, p, q, k in ((y[a:b], xe, we.t(), K), (y32[a:b], xe, we.t(), K), (dx[a:b], de, we, N), (dw[e], de.t(), xe, b - a),
                             (dw32[e], de.t(), xe, b - a)):
            want = ffn_ref.mm(p, q)
            bound = ffn_ref.stored(ffn_ref.sum_bound(p, q, k), want, got.dtype)
            assert ((got.double().cpu() - want).abs() <= bound).all()


def test_grouped_rows_do_not_depend_on_the_batch(bi):
    """A row's bits: alone, in other splits, beside other experts."""
    E, N, K = 5, 208, 480
    counts = [700, 3, 0, 290, 64]
    T, ends = sum(counts), ends_of(counts)
    x, w, dy = normal((T, K), 1), normal((E, N, K), 2), normal((T, N), 3)
    xq, xs = bi.bi_quantize_int8(x)
    wq, ws = (t.reshape(E, N, -1).squeeze(2) for t in bi.bi_quantize_int8(w.reshape(E * N, K)))
    y = bi.bi_grouped_linear_bf16(x, w, ends)
    y8 = bi.bi_grouped_linear_int8(xq, xs, wq, ws, ends)
    dx, _ = bi.bi_grouped_linear_bf16_bwd(dy, None, w, ends, need_dw=False)
    for e, (a, b) in enumerate(ref.spans(ends.tolist(), T)):
        for s in (slice(a, min(a + 1, b)), slice(a + (b - a) // 2, b), slice(max(a, b - 17), b)):
            n = s.stop - s.start
            if n <= 0:
                continue
            alone = ends_of([0] * e + [n] + [0] * (E - e - 1))
            assert torch.equal(bi.bi_grouped_linear_bf16(x[s], w, alone), y[s])
            assert torch.equal(bi.bi_grouped_linear_int8(xq[s], xs[s], wq, ws, alone), y8[s])
            assert torch.equal(bi.bi_grouped_linear_bf16_bwd(dy[s], None, w, alone, need_dw=False)[0], dx[s])
            # the same layer with one expert, and as a plain 8-bit product
            assert torch.equal(bi.bi_grouped_linear_bf16(x[s], w[e:e + 1], ends_of([n])), y[s])
            assert torch.equal(bi.bi_linear_int8(xq[s], xs[s], wq[e], ws[e]), y8[s])
            # and the gradient a linear layer gives
            assert torch.equal(bi.bi_linear_bf16_bwd(dy[s], None, w[e].t(), need_dw=False, need_db=False)[0], dx[s])


def test_many_experts(bi):
    """More experts than a wave has lanes, most of them without rows."""
    for E in (64, 65, 128, 1024):
        banner(f"grouped E={E}")
        g = torch.Generator().manual_seed(E)
        counts = [int(c) for c in torch.randint(0, 40, (E,), generator=g) * (torch.rand(E, generator=g) < 0.3)]
        T, N, K = sum(counts), 32, 64
        x, w, dy, ends = ints((T, K), 1), ints((E, N, K), 2), ints((T, N), 3), ends_of(counts)
        same_rows(bi.bi_grouped_linear_bf16(x, w, ends), forward_ref(x, w, ends))
        dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, dw_dtype=F32)
        same_rows(dx, forward_ref(dy, w.transpose(1, 2), ends))
        for e, (a, b) in enumerate(ref.spans(ends.tolist(), T)):
            if e % 13 == 0 or b > a:
                assert torch.equal(dw[e].double().cpu(), dy[a:b].double().cpu().t() @ x[a:b].double().cpu())


@pytest.mark.parametrize("raw", [[3, 1, 9, 9], [-5, 4, 2, 100], [50, 0, 0, 0], [1 << 40, -(1 << 40), 7, 8], [0, 0, 0, -1]], ids=str)
def test_ends_of_any_values_stay_in_range(bi, raw):
    """Not ascending, negative or past the rows: the running maximum within 0 .. T."""
    T, N, K, E = 20, 48, 64, 4
    x, w, dy, ends = ints((T, K), 1), ints((E, N, K), 2), ints((T, N), 3), torch.tensor(raw).cuda()
    want = forward_ref(x, w, ends)
    out = torch.full((T + 4, N), 7.0, dtype=BF, device="cuda")
    bi.bi_grouped_linear_bf16(x, w, ends, out=out[:T])
    same_rows(out[:T], want)
    last = ref.spans(raw, T)[-1][1]
    assert (out[last:] == 7.0).all()
    _, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, need_dx=False, dw_dtype=F32)
    for e, (a, b) in enumerate(ref.spans(raw, T)):
        assert torch.equal(dw[e].double().cpu(), dy[a:b].double().cpu().t() @ x[a:b].double().cpu())


def test_layouts(bi):
    """Pitches, experts apart, one weight for all, rows out of a wider matrix."""
    counts, N, K = [20, 0, 45], 80, 160
    T, E, ends = sum(counts), 3, ends_of(counts)
    xb, wb, db = ints((T, K + 40), 1), ints((E, N + 3, K + 24), 2), ints((T, N + 16), 3)
    x, w, dy = xb[:, 8:8 + K], wb[:, 1:1 + N, 16:16 + K], db[:, :N]
    out = torch.full((T, N + 32), 7.0, dtype=BF, device="cuda")
    bi.bi_grouped_linear_bf16(x, w, ends, out=out[:, 16:16 + N])
    same_rows(out[:, 16:16 + N].contiguous(), forward_ref(x, w, ends))
    assert (out[:, :16] == 7.0).all() and (out[:, 16 + N:] == 7.0).all()
    dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends)
    same_rows(dx, forward_ref(dy, w.transpose(1, 2), ends))
    one = w[:1].expand(E, N, K)
    same_rows(bi.bi_grouped_linear_bf16(x, one, ends), forward_ref(x, one, ends))
    # an expert's columns of a [N, E K] matrix: experts closer together than their rows
    side = ints((N, E * K), 4).view(N, E, K).transpose(0, 1)
    same_rows(bi.bi_grouped_linear_bf16(x, side, ends), forward_ref(x, side, ends))


def test_no_rows_at_all(bi):
    w = ints((3, 32, 64), 1)
    e0 = torch.zeros(3, dtype=torch.int64, device="cuda")
    x, dy = torch.empty((0, 64), dtype=BF, device="cuda"), torch.empty((0, 32), dtype=BF, device="cuda")
    assert bi.bi_grouped_linear_bf16(x, w, e0).shape == (0, 32)
    dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, e0)
    assert dx.shape == (0, 64) and dw.shape == (3, 32, 64) and not dw.any()
    q, s = bi.bi_quantize_int8(x)
    assert q.shape == (0, 64) and s.shape == (0,)
    wq, ws = w.to(torch.int8), torch.ones((3, 32), device="cuda")
    assert bi.bi_grouped_linear_int8(q, s, wq, ws, e0).shape == (0, 32)
    assert bi.bi_linear_int8(q, s, wq[0], ws[0]).shape == (0, 32)


def test_nan_stays_in_its_expert(bi):
    """An expert's infinities and NaNs, and those of rows without expert."""
    counts, N, K = [18, 20, 3], 64, 96
    T, ends = sum(counts), ends_of(counts)
    x, w, dy = ints((T + 6, K), 1), ints((3, N, K), 2), ints((T + 6, N), 3)
    clean_y = bi.bi_grouped_linear_bf16(x, w, ends)[:T].clone()
    clean_dx, clean_dw = (t.clone() for t in bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends))
    for t in (x, dy):
        t[T:] = float("nan")
        t[18, 3] = float("nan")
        t[30, 1] = float("inf")
    y = bi.bi_grouped_linear_bf16(x, w, ends)
    dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends)
    keep = torch.ones(T, dtype=torch.bool)
    keep[[18, 30]] = False
    assert torch.equal(y[:T][keep], clean_y[keep]) and torch.equal(dx[:T][keep], clean_dx[:T][keep])
    assert torch.equal(dw[0], clean_dw[0]) and torch.equal(dw[2], clean_dw[2])
    assert torch.isnan(y[18]).all() and torch.isnan(dw[1][:, 3]).all()


# ------------------------------------------------------------------ 8-bit integers


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("K", [32, 64, 2016, 2048, 2080, 4096, 4128, 8192, 8224, 20000])
def test_quantize(bi, K, dtype):
    for rows in (1, 5, 300):
        g = torch.Generator().manual_seed(K + rows)
        x = (torch.randn((rows, K + 8), generator=g) * torch.exp(2 * torch.randn((rows, 1), generator=g))).to(dtype).cuda()[:, :K]
        q, s = bi.bi_quantize_int8(x)
        qd, sd = ref.codes(x)
        assert torch.equal(s.cpu(), sd) and torch.equal(q.cpu(), qd)


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("K", [96, 480, 512, 544, 768, 1024, 1056])
def test_quantize_a_wave_to_a_row(bi, K, dtype):
    """Rows on both sides of the lengths that one wave takes, some workgroups' last rows
    missing, more of them than workgroups are launched for; a row of NaN beside others."""
    for rows in (2, 3, 9001):
        x = normal((rows, K), K + rows, dtype=dtype)
        x[rows // 2, K // 2] = float("nan")
        q, s = bi.bi_quantize_int8(x)
        qd, sd = ref.codes(x)
        keep = torch.arange(rows) != rows // 2
        assert torch.equal(s.cpu()[keep], sd[keep]) and torch.isnan(s[rows // 2])
        assert torch.equal(q.cpu(), qd)


def test_quantize_on_the_border(bi):
    """Halfway points and their neighbours, by one fp32 step either way, under scales
    that are not powers of two; tiny, huge, empty and non-finite rows."""
    tops = torch.cat((torch.tensor([127.0, 1.0, 3.0, 0.1, 1e30, 1e-30, 2.0 ** -121, 1.0000001 * 2.0 ** -119, 3.3e38, 1e-40]),
                      torch.rand(500, generator=torch.Generator().manual_seed(1)) * 10))
    x = torch.zeros((len(tops), 1024), dtype=F32)
    half = torch.arange(-127, 127).double() + 0.5
    for i, top in enumerate(tops):
        s = torch.clamp(top * torch.tensor(1.0 / 127.0), min=2.0 ** -126)
        at = (half * s.double()).float()
        at = at[at.abs() <= top]
        n = len(at)
        x[i, :n] = at
        x[i, n:2 * n] = torch.nextafter(at, torch.tensor(float("inf")))
        x[i, 2 * n:3 * n] = torch.nextafter(at, torch.tensor(float("-inf")))
        x[i] = x[i].clamp(-float(top), float(top))
        x[i, -1] = top
    x = torch.cat((x, torch.zeros((4, 1024))))
    x[-3, 7], x[-2, 9], x[-1, 1] = float("inf"), float("nan"), float("-inf")
    q, s = bi.bi_quantize_int8(x.cuda())
    qd, sd = ref.codes(x)
    assert torch.equal(s.cpu()[:-3], sd[:-3]) and torch.isnan(s[-3:]).all()
    assert torch.equal(q.cpu(), qd)


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
def test_quantize_beside_the_quotients_scale(bi, dtype):
    """Scales are max|x| / 127 or one step less, codes within half a scale of their values,
    and where they are not the quotient's codes the value lies next to halfway."""
    top = 1 + torch.arange(1280, dtype=torch.float64) / 1280
    at = torch.cat((torch.tensor([1.0, 0.5, -0.5], dtype=torch.float64), torch.linspace(-1, 1, 61, dtype=torch.float64)))
    x = (top[:, None] * at).to(dtype)
    q, s = (t.cpu() for t in bi.bi_quantize_int8(x.cuda()))
    xd, sd = x.double(), s.double()[:, None]
    sq = (xd.abs().amax(1) / 127).float()
    step = s.view(torch.int32) - sq.view(torch.int32)
    assert step.min() == -1 and step.max() == 0
    assert ((q.double() * sd - xd).abs() <= 0.5 * sd).all()
    v = xd / sq.double()[:, None]
    far = (v - torch.floor(v) - 0.5).abs() > 127 * 2.0 ** -23
    assert (q.double() == torch.round(v))[far].all() and (q.double() - torch.round(v)).abs().max() == 1


@pytest.mark.parametrize("M,N,K", [(1, 16, 32), (3, 48, 96), (17, 80, 64), (33, 272, 416), (70, 144, 1056), (130, 400, 224),
                                   (300, 528, 160), (515, 784, 352), (5, 2064, 8224)])
def test_int8_product_bit_for_bit(bi, M, N, K):
    g = torch.Generator().manual_seed(M)
    xq = torch.randint(-128, 128, (M, K + 16), generator=g).to(torch.int8).cuda()[:, :K]
    wq = torch.randint(-128, 128, (N, K), generator=g).to(torch.int8).cuda()
    xs, ws = torch.rand(M, generator=g).cuda() * 0.1, torch.rand(N, generator=g).cuda() * 0.01
    bias = torch.randn(N, generator=g).cuda()
    for b in (None, bias):
        for dt in (BF, F32):
            banner(f"int8 M={M} N={N} K={K} {dt}")
            assert torch.equal(bi.bi_linear_int8(xq, xs, wq, ws, b, out_dtype=dt).cpu(), ref.linear_int8(xq, xs, wq, ws, b, dt))


def test_int8_extremes(bi):
    """The largest sums, and scales of any value."""
    K = 131040
    x = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((16, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one = torch.ones(16, device="cuda")
    y = bi.bi_linear_int8(x, one[:2].clone(), w, one, out_dtype=F32)
    assert torch.equal(y.cpu(), ref.linear_int8(x, one[:2], w, one, None, F32))
    xs = torch.tensor([float("nan"), 2.0 ** -126], device="cuda")
    y = bi.bi_linear_int8(x, xs, w, one, out_dtype=F32)
    assert torch.isnan(y[0]).all() and torch.equal(y[1].cpu(), ref.linear_int8(x, xs, w, one, None, F32)[1])


@pytest.mark.parametrize("counts", SPLITS, ids=lambda c: "-".join(map(str, c)))
def test_grouped_int8_bit_for_bit(bi, counts):
    T, E = sum(counts), len(counts)
    for (N, K), tail in zip(SIZES, (0, 3, 9, 0)):
        banner(f"grouped int8 {counts} N={N} K={K}")
        g = torch.Generator().manual_seed(N)
        xq = torch.randint(-128, 128, (T + tail, K), generator=g).to(torch.int8).cuda()
        wq = torch.randint(-128, 128, (E, N, K + 32), generator=g).to(torch.int8).cuda()[:, :, :K]
        xs, ws = torch.rand(T + tail, generator=g).cuda(), torch.rand((E, N + 4), generator=g).cuda()[:, :N]
        ends = ends_of(counts)
        for dt in (BF, F32):
            out = torch.full((T + tail, N), 7.0, dtype=dt, device="cuda")
            bi.bi_grouped_linear_int8(xq, xs, wq, ws, ends, out=out)
            for e, (a, b) in enumerate(ref.spans(ends.tolist(), T)):
                assert torch.equal(out[a:b].cpu(), ref.linear_int8(xq[a:b], xs[a:b], wq[e], ws[e], None, dt))
            assert (out[T:] == 7.0).all()


def test_int8_is_near_the_product_it_stands_for(bi):
    """Quantised activations and weights against the unquantised product: each
    operand is within half a scale of its value, every sum of products within what
    that adds up to."""
    M, N, K = 60, 96, 512
    x, w = normal((M, K), 1), normal((N, K), 2, F32, K ** -0.5)
    (xq, xs), (wq, ws) = bi.bi_quantize_int8(x), bi.bi_quantize_int8(w)
    y = bi.bi_linear_int8(xq, xs, wq, ws, out_dtype=F32).double().cpu()
    xd, wd = x.double().cpu(), w.double().cpu()
    ex, ew = 0.5 * xs.double().cpu()[:, None], 0.5 * ws.double().cpu()
    bound = ex * wd.abs().sum(1) + xd.abs().sum(1, keepdim=True) * ew + K * ex * ew
    want = xd @ wd.t()
    assert ((y - want).abs() <= bound * (1 + 1e-6) + 4 * ref.U * want.abs()).all()


# -------------------------------------------------- every tile shape past its ring


@pytest.mark.parametrize("M,N,K", shapes.INT8)
def test_int8_tile_shapes(bi, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    xq, wq = (torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8) for s in ((M, K), (N, K)))
    xs, ws, b = (torch.rand(n, generator=g, device="cuda") for n in (M, N, N))
    acc = torch.mm(xq.double(), wq.double().t()).float()
    want = acc * xs[:, None] * ws + b
    for dt in (BF, F32):
        banner(f"int8 shapes {M} {N} {K} {dt}")
        assert torch.equal(bi.bi_linear_int8(xq, xs, wq, ws, b, out_dtype=dt), want.to(dt))


@pytest.mark.parametrize("T,E,N,K", shapes.GROUPED)
def test_grouped_tile_shapes(bi, T, E, N, K):
    counts = shapes.counts(T, E)
    x, w, ends = ints((T, K), 1), ints((E, N, K), 2), ends_of(counts)
    xq, wq = x.to(torch.int8), w.to(torch.int8)
    xs, ws = torch.rand(T, device="cuda"), torch.rand((E, N), device="cuda")
    want = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    scale = torch.zeros((T, N), device="cuda")
    for e, (a, b) in enumerate(ref.spans(ends.tolist(), T)):
        want[a:b] = x[a:b].double() @ w[e].double().t()
        scale[a:b] = ws[e]
    for dt in (BF, F32):
        banner(f"grouped shapes {T} {E} {N} {K} {dt}")
        assert torch.equal(bi.bi_grouped_linear_bf16(x, w, ends, out_dtype=dt), want.to(dt))
        y8 = bi.bi_grouped_linear_int8(xq, xs, wq, ws, ends, out_dtype=dt)
        assert torch.equal(y8, (want.float() * xs[:, None] * scale).to(dt))


@pytest.mark.parametrize("T,E,N,K", shapes.GROUPED_BWD)
def test_grouped_backward_tile_shapes(bi, T, E, N, K):
    counts = shapes.counts(T, E)
    x, w, dy, ends = ints((T, K), 1), ints((E, N, K), 2), ints((T, N), 3), ends_of(counts)
    want_dx = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    want_dw = torch.zeros((E, N, K), dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(ref.spans(ends.tolist(), T)):
        want_dx[a:b] = dy[a:b].double() @ w[e].double()
        want_dw[e] = dy[a:b].double().t().contiguous() @ x[a:b].double()
    for dt in (BF, F32):
        for dx_too, dw_too in ((True, True), (True, False), (False, True)):
            banner(f"grouped backward shapes {T} {E} {N} {K} {dt} {dx_too} {dw_too}")
            dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, need_dx=dx_too, need_dw=dw_too, dw_dtype=dt)
            assert dx is None or torch.equal(dx, want_dx.to(BF))
            assert dw is None or torch.equal(dw, want_dw.to(dt))


def _skewed(T, E, kind):
    if kind == "one":
        return [0] * (E // 2) + [T] + [0] * (E - E // 2 - 1)
    if kind == "last":
        return [0] * (E - 1) + [T]
    if kind == "few":                                   # many more experts without rows than with
        c = [T // 7 if e % (E // 7 + 1) == 3 else 0 for e in range(E)]
        c[0] += T - sum(c)
        return c
    return shapes.counts(T, E)


@pytest.mark.parametrize("kind", ["half", "one", "last", "few"])
@pytest.mark.parametrize("T,E,N,K", [(9000, 40, 768, 1024), (3001, 300, 1024, 1024), (9000, 40, 1008, 1504)])
def test_largest_weight_gradient_tiles(bi, T, E, N, K, kind):
    """Several tiles to a workgroup, whole and ragged ones, with experts without rows
    between, before and behind them."""
    assert bi.grouped_tile(bi.BI_GROUPED_DW_ALONE, T, E, N, K)["rows"] == 256
    x, w, dy, ends = ints((T, K), 1), ints((E, N, K), 2), ints((T, N), 3), ends_of(_skewed(T, E, kind))
    want_dx = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    want = torch.zeros((E, N, K), dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(ref.spans(ends.tolist(), T)):
        if b > a:
            want_dx[a:b] = dy[a:b].double() @ w[e].double()
            want[e] = dy[a:b].double().t().contiguous() @ x[a:b].double()
    for dt in (BF, F32):
        banner(f"largest dw {T} {E} {N} {K} {kind} {dt}")
        for _ in range(3):
            assert torch.equal(bi.bi_grouped_linear_bf16_bwd(dy, x, None, ends, need_dx=False, dw_dtype=dt)[1], want.to(dt))
            dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, dw_dtype=dt)
            assert torch.equal(dw, want.to(dt)) and torch.equal(dx, want_dx.to(BF))


def test_operands_past_4_gib(bi):
    """Rows, experts and outputs whose offsets pass 32 bits."""
    T, E, N, K = 70000, 2, 64, 32768                       # x: 4.6e9 bytes in bf16
    x = torch.zeros((T, K), dtype=BF, device="cuda")
    w = torch.zeros((E, N, K), dtype=BF, device="cuda")
    probe = ints((16, K), 1)
    w[0], w[1] = ints((N, K), 2), ints((N, K), 3)
    x[-16:] = probe
    ends = ends_of([T - 16, 16])
    banner("grouped rows past 4 GiB")
    y = bi.bi_grouped_linear_bf16(x, w, ends, out_dtype=F32)
    assert torch.equal(y[-16:].double(), probe.double() @ w[1].double().t())
    assert not y[:-16].any()
    dy = torch.zeros((T, N), dtype=BF, device="cuda")
    dy[-16:] = ints((16, N), 4)
    dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, dw_dtype=F32)
    assert torch.equal(dx[-16:].double(), (dy[-16:].double() @ w[1].double()).to(BF).double()) and not dx[:-16].any()
    assert torch.equal(dw[1].double(), dy[-16:].double().t().contiguous() @ probe.double()) and not dw[0].any()
    banner("8-bit rows past 4 GiB")
    del dx, dw
    xq = torch.zeros((140000, K), dtype=torch.int8, device="cuda")
    xq[-16:] = probe.to(torch.int8)
    xs, ws = torch.ones(140000, device="cuda"), torch.ones(N, device="cuda")
    y = bi.bi_linear_int8(xq, xs, w[1].to(torch.int8), ws, out_dtype=F32)
    assert torch.equal(y[-16:].double(), probe.double() @ w[1].double().t()) and not y[:-16].any()
    q, s = bi.bi_quantize_int8(x)
    assert torch.equal(q[-16:].float(), torch.round(probe.float() / s[-16:, None])) and not q[:-16].any()
    banner("layer norm rows past 4 GiB")
    z = torch.zeros((280000, 8192), dtype=BF, device="cuda")
    z[-4:] = normal((4, 8192), 5)
    n, m, r = bi.bi_layer_norm(z, save_stats=True)
    assert torch.equal(n[-4:], bi.bi_layer_norm(z[-4:].clone())) and not n[:-4].any()
    assert torch.equal(bi.bi_layer_norm_bwd(z, z, m, r)[0][-4:], bi.bi_layer_norm_bwd(z[-4:].clone(), z[-4:].clone(), m[-4:].clone(), r[-4:].clone())[0])


# ---------------------------------------------------------------- a run of them


def test_an_expert_block_trained_and_served(bi):
    """Norm, routed rows, both products of gated experts and all gradients, against
    the same block in binary64; then the same experts in 8 bits."""
    g = torch.Generator().manual_seed(11)
    M, H, E, I, k = 90, 128, 6, 64, 2
    x = normal((M, H), 1, F32)
    nw, nb = 1 + 0.1 * normal((H,), 2, F32), 0.1 * normal((H,), 3, F32)
    w13, w2 = normal((E, 2 * I, H), 4, std=H ** -0.5), normal((E, H, I), 5, std=I ** -0.5)
    dout = normal((M, H), 6, std=0.1)
    ids = torch.rand((M, E), generator=g).topk(k, dim=1).indices
    order = torch.argsort(ids.flatten(), stable=True)
    token = (order // k).cuda()
    ends = torch.cumsum(torch.bincount(ids.flatten(), minlength=E), 0).cuda()

    y, mean, rstd = bi.bi_layer_norm(x, nw, nb, out_dtype=BF, save_stats=True)
    rows = y[token].contiguous()
    h = bi.bi_grouped_linear_bf16(rows, w13, ends)
    hg, hu = h[:, :I].float(), h[:, I:].float()
    act = (torch.nn.functional.silu(hg) * hu).to(BF)
    out = torch.zeros((M, H), device="cuda").index_add_(0, token, bi.bi_grouped_linear_bf16(act, w2, ends, out_dtype=F32))
    # backward
    drow = dout[token].contiguous()
    dact, dw2 = bi.bi_grouped_linear_bf16_bwd(drow, act, w2, ends, dw_dtype=F32)
    sg = torch.sigmoid(hg)
    dh = torch.cat((dact.float() * hu * (sg + hg * sg * (1 - sg)), dact.float() * hg * sg), 1).to(BF)
    drows, dw13 = bi.bi_grouped_linear_bf16_bwd(dh, rows, w13, ends, dw_dtype=F32)
    dy = torch.zeros((M, H), device="cuda").index_add_(0, token, drows.float())
    dx, dnw, dnb = bi.bi_layer_norm_bwd(dy, x, mean, rstd, nw)

    # the same in binary64 with autograd on the CPU
    p = [t.double().cpu().requires_grad_() for t in (x, nw, nb, w13, w2)]
    X, NW, NB, W13, W2 = p
    Y = (X - X.mean(1, keepdim=True)) * (X.var(1, unbiased=False, keepdim=True) + 1e-5) ** -0.5 * NW + NB
    tok, parts = token.cpu(), []
    for e, (a, b) in enumerate(ref.spans(ends.tolist(), M * k)):
        hh = Y[tok[a:b]] @ W13[e].t()
        parts.append((torch.nn.functional.silu(hh[:, :I]) * hh[:, I:]) @ W2[e].t())
    OUT = torch.zeros((M, H), dtype=torch.float64).index_add(0, tok, torch.cat(parts))
    OUT.backward(dout.double().cpu())
    # bf16 storage points in a row: the norm's output, h, act, and in the backward
    # pass dact, dh, drows: at most six roundings of 2^-9 rms each (2^-8 at most) plus
    # second order, on terms that add up like independent ones
    for got, want in ((out, OUT.detach()), (dw2, W2.grad), (dw13, W13.grad), (dx, X.grad), (dnw, NW.grad), (dnb, NB.grad)):
        err = (got.double().cpu() - want).norm() / want.norm()
        assert err < 6 * 2.0 ** -8, float(err)

    # served in 8 bits: the steps on the GPU equal the definition's, step by step
    w13q, w13s = (t.reshape(E, 2 * I, -1).squeeze(2) for t in bi.bi_quantize_int8(w13.reshape(-1, H)))
    q, s = bi.bi_quantize_int8(rows)
    h8 = bi.bi_grouped_linear_int8(q, s, w13q, w13s, ends)
    for e, (a, b) in enumerate(ref.spans(ends.tolist(), M * k)):
        assert torch.equal(h8[a:b].cpu(), ref.linear_int8(q[a:b], s[a:b], w13q[e], w13s[e], None, BF))


def test_graph_replays_and_streams(bi):
    """One capture serves any split of its rows: the ends are read at replay."""
    T, E, N, K = 120, 4, 96, 160
    x, w, dy = normal((T, K), 1), normal((E, N, K), 2), normal((T, N), 3)
    wq, ws = (t.reshape(E, N, -1).squeeze(2) for t in bi.bi_quantize_int8(w.reshape(-1, K)))
    ends = ends_of([30, 30, 30, 30])
    buf = {k: torch.zeros(s, dtype=BF, device="cuda") for k, s in (("y", (T, N)), ("y8", (T, N)), ("dx", (T, K)))}

    def step(b):
        q, s = bi.bi_quantize_int8(x)
        _, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, out_dx=b["dx"])
        return [bi.bi_grouped_linear_bf16(x, w, ends, out=b["y"]), bi.bi_grouped_linear_int8(q, s, wq, ws, ends, out=b["y8"]),
                b["dx"], dw, bi.bi_linear_int8(q, s, wq[0], ws[0])]

    want = [t.clone() for t in step(buf)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = step({k: torch.zeros_like(v) for k, v in buf.items()})
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(buf)
    for counts in ([30, 30, 30, 30], [0, 120, 0, 0], [1, 2, 3, 4], [60, 0, 0, 60], [0, 0, 0, 0]):
        ends.copy_(ends_of(counts))
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for t in out:
            t.zero_()
        eager = step({k: torch.zeros_like(v) for k, v in buf.items()})
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), counts


def test_refusals_on_the_gpu(bi):
    x, w, ends, dy = ints((8, 64), 1), ints((2, 32, 64), 2), ends_of([3, 5]), ints((8, 32), 3)
    i8 = torch.int8
    q, s, wq, ws = x.to(i8), torch.ones(8, device="cuda"), w.to(i8), torch.ones((2, 32), device="cuda")
    for call in (lambda: bi.bi_grouped_linear_bf16(x, w, ends[:1]), lambda: bi.bi_grouped_linear_bf16(x, w, ends.cpu()),
                 lambda: bi.bi_grouped_linear_bf16(x, w.transpose(1, 2), ends), lambda: bi.bi_grouped_linear_bf16(x[:, :32], w, ends),
                 lambda: bi.bi_grouped_linear_bf16(x, w, ends, out=dy[:4]), lambda: bi.bi_grouped_linear_bf16(x.cpu(), w, ends),
                 lambda: bi.bi_grouped_linear_bf16(x, w.cpu(), ends), lambda: bi.bi_grouped_linear_bf16(x, torch.empty((2, 33, 64))[:, :32].to(x), ends[::2]),
                 lambda: bi.bi_grouped_linear_bf16_bwd(dy, x[:5], w, ends), lambda: bi.bi_grouped_linear_bf16_bwd(dy, x, w[:1], ends),
                 lambda: bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, out_dx=x[:4]),
                 lambda: bi.bi_linear_int8(q, s[:4], wq[0], ws[0]), lambda: bi.bi_linear_int8(q, s, wq[0], ws[0, :16]),
                 lambda: bi.bi_linear_int8(q, s, wq[0][:, :32], ws[0]), lambda: bi.bi_linear_int8(q, s, wq[0], ws[0], bias=s),
                 lambda: bi.bi_grouped_linear_int8(q, s, wq, ws[:1], ends), lambda: bi.bi_grouped_linear_int8(q, s, wq, ws.t().contiguous().t(), ends)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bi.bi_grouped_linear_bf16(x, w, ends.int()), lambda: bi.bi_grouped_linear_bf16(x, w.float(), ends),
                 lambda: bi.bi_linear_int8(q.to(torch.uint8), s, wq[0], ws[0]), lambda: bi.bi_linear_int8(q, s.double(), wq[0], ws[0])):
        with pytest.raises(TypeError):
            call()


def test_outputs_over_operands_are_refused_and_beside_them_taken(bi):
    """Columns of one matrix: an output beside its operand, and over it."""
    T, N, K, ends = 70, 64, 64, ends_of([30, 0, 40])
    w, dy = ints((3, N, K), 2), ints((T, N), 3)
    wide = torch.cat((ints((T, K), 1), torch.full((T, 2 * N), 7.0, dtype=BF, device="cuda")), 1)
    x, keep = wide[:, :K], wide[:, :K].clone()
    q, s = bi.bi_quantize_int8(keep)
    wq, ws = (t.reshape(3, N, -1).squeeze(2) for t in bi.bi_quantize_int8(w.reshape(-1, K)))
    for call in (lambda: bi.bi_grouped_linear_bf16(x, w, ends, out=x), lambda: bi.bi_grouped_linear_bf16(x, w, ends, out=wide[:, 32:96]),
                 lambda: bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, out_dx=dy), lambda: bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, out_dx=x),
                 lambda: bi.bi_layer_norm(x, out=wide[:, 8:8 + K]),
                 lambda: bi.bi_linear_int8(q[:2], s[:2], wq[0], ws[0], out=q.view(BF).view(-1)[:2 * N].view(2, N)),
                 lambda: bi.bi_grouped_linear_int8(q[:2], s[:2], wq, ws, ends, out=q.view(BF).view(-1)[:2 * N].view(2, N))):
        with pytest.raises(ValueError, match="overlap"):
            call()
    bi.bi_grouped_linear_bf16(x, w, ends, out=wide[:, K:K + N])
    same_rows(wide[:, K:K + N].contiguous(), forward_ref(keep, w, ends))
    bi.bi_grouped_linear_bf16_bwd(wide[:, K:K + N], None, w, ends, need_dw=False, out_dx=wide[:, K + N:])
    same_rows(wide[:, K + N:].contiguous(), forward_ref(wide[:, K:K + N].contiguous(), w.transpose(1, 2), ends).to(BF).double())
    assert torch.equal(x, keep)


@pytest.mark.parametrize("E", [1, 63, 129, 160, 256, 257, 512])
def test_experts_to_a_lane(bi, E):
    """1, 2, 4 and 16 experts to a lane of the wave that finds a workgroup's rows, at both
    ends of each: forward, dx, dw alone and together, 8 bits, uneven rows."""
    g = torch.Generator().manual_seed(E)
    counts = [int(c) for c in torch.randint(0, 50, (E,), generator=g) * (torch.rand(E, generator=g) < 0.6)]
    counts[0], counts[-1] = 3, 70
    T, N, K, ends = sum(counts), 48, 64, ends_of(counts)
    x, w, dy = ints((T, K), 1), ints((E, N, K), 2), ints((T, N), 3)
    xs, ws = torch.rand(T, generator=g).cuda(), torch.rand((E, N), generator=g).cuda()
    want, want_dx = forward_ref(x, w, ends), forward_ref(dy, w.transpose(1, 2), ends)
    want_dw = torch.zeros((E, N, K), dtype=torch.float64)
    want8 = torch.zeros((T, N))
    for e, (a, b) in enumerate(ref.spans(ends.tolist(), T)):
        want_dw[e] = dy[a:b].double().cpu().t() @ x[a:b].double().cpu()
        want8[a:b] = ref.linear_int8(x[a:b].to(torch.int8), xs[a:b], w[e].to(torch.int8), ws[e], None, F32)
    banner(f"grouped E={E}")
    same_rows(bi.bi_grouped_linear_bf16(x, w, ends, out_dtype=F32), want)
    assert torch.equal(bi.bi_grouped_linear_int8(x.to(torch.int8), xs, w.to(torch.int8), ws, ends, out_dtype=F32).cpu(), want8)
    for dx_too, dw_too in ((True, True), (True, False), (False, True)):
        dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, need_dx=dx_too, need_dw=dw_too, dw_dtype=F32)
        assert dx is None or same_rows(dx, want_dx) is None
        assert dw is None or torch.equal(dw.double().cpu(), want_dw)


def _some_experts(ends, T):
    """The experts with the most rows, the first and the last that have any."""
    spans = ref.spans(ends.tolist(), T)
    some = [e for e, (a, b) in enumerate(spans) if b > a]
    big = sorted(some, key=lambda e: spans[e][0] - spans[e][1])[:2]
    return [(e, *spans[e]) for e in sorted({*big, some[0], some[-1]})]


def _some_rows(a, b):
    """Rows at the expert's ends and around tile heights, as short slices."""
    at = {a, (a + b) // 2, b - 1, *(a + h for h in (15, 63, 127, 255) if a + h < b)}
    return [slice(i, min(i + 2, b)) for i in sorted(at)]


@pytest.mark.parametrize("T,E,N,K", shapes.GROUPED)
def test_rows_do_not_depend_on_the_tile(bi, T, E, N, K):
    """Random values, whose sums round at every step, through every tile shape: rows of y
    have the bits of the same rows alone, which take the smallest shapes."""
    ends = ends_of(shapes.counts(T, E))
    x, w = normal((T, K), 1), normal((E, N, K), 2, std=K ** -0.5)
    for dt in (BF, F32):
        banner(f"rows of tiles {T} {E} {N} {K} {dt}")
        y = bi.bi_grouped_linear_bf16(x, w, ends, out_dtype=dt)
        for e, a, b in _some_experts(ends, T):
            for s in _some_rows(a, b):
                assert torch.equal(bi.bi_grouped_linear_bf16(x[s], w[e:e + 1], ends_of([s.stop - s.start]), out_dtype=dt), y[s])


def _check_backward_bits(bi, dy, x, w, ends):
    """Both gradients from one call and from one each; rows of dx and experts of dw alone."""
    T, E = len(x), len(w)
    alone_dx, _ = bi.bi_grouped_linear_bf16_bwd(dy, None, w, ends, need_dw=False)
    last = int(ends[-1])
    for dt in (BF, F32):
        _, alone_dw = bi.bi_grouped_linear_bf16_bwd(dy, x, None, ends, need_dx=False, dw_dtype=dt)
        for _ in range(2):
            dx, dw = bi.bi_grouped_linear_bf16_bwd(dy, x, w, ends, dw_dtype=dt)
            assert torch.equal(dx[:last], alone_dx[:last]) and torch.equal(dw, alone_dw)
        for e, a, b in _some_experts(ends, T):
            one = bi.bi_grouped_linear_bf16_bwd(dy[a:b], x[a:b], None, ends_of([b - a]), need_dx=False, dw_dtype=dt)[1]
            assert torch.equal(one[0], dw[e])
    for e, a, b in _some_experts(ends, T):
        for s in _some_rows(a, b):
            few = bi.bi_grouped_linear_bf16_bwd(dy[s], None, w[e:e + 1], ends_of([s.stop - s.start]), need_dw=False)[0]
            assert torch.equal(few, alone_dx[s])


@pytest.mark.parametrize("T,E,N,K", shapes.GROUPED_BWD)
def test_gradients_do_not_depend_on_the_tile(bi, T, E, N, K):
    banner(f"gradients of tiles {T} {E} {N} {K}")
    ends = ends_of(shapes.counts(T, E))
    _check_backward_bits(bi, normal((T, N), 3), normal((T, K), 1), normal((E, N, K), 2), ends)


@pytest.mark.parametrize("kind", ["half", "one", "few"])
@pytest.mark.parametrize("T,E,N,K", [(9000, 40, 768, 1024), (3001, 300, 1024, 1024), (9000, 40, 1008, 1504)])
def test_gradients_of_the_largest_tiles_do_not_depend_on_the_tile(bi, T, E, N, K, kind):
    banner(f"gradients of the largest tiles {T} {E} {N} {K} {kind}")
    assert bi.grouped_tile(bi.BI_GROUPED_DW_ALONE, T, E, N, K)["rows"] == 256
    g = torch.Generator(device="cuda").manual_seed(T)
    dy, x, w = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((T, N), (T, K), (E, N, K)))
    _check_backward_bits(bi, dy, x, w, ends_of(_skewed(T, E, kind)))
