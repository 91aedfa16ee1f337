"""Layer norm and its backward pass on the GPU against 64-bit forms."""
import pytest

torch = pytest.importorskip("torch")

from tests import experts_ref as ref
from tests.gpu_util import banner

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bi():
    import deterministic_persistent_gemm_amd as m
    return m


def rows(M, H, seed, dtype, shift=0.3, pad=0):
    """M rows off zero with channels of unlike size, at a pitch of H + pad."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, H + pad), generator=g) * torch.exp(0.5 * torch.randn((1, H + pad), generator=g)) + shift * torch.randn((M, 1), generator=g)
    return x.to(dtype).cuda()[:, :H]


def vec(H, seed, mean=0.0):
    return (mean + 0.1 * torch.randn(H, generator=torch.Generator().manual_seed(seed))).cuda()


def within(got, want, bound, what):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} outside, worst {float((err / bound).nan_to_num(1e9).max()):.3f} of the bound"


# every team size and chunk count, and their edges
HS = [8, 256, 504, 512, 520, 2048, 2056, 4088, 4096, 4104, 8192, 8200, 16384]


@pytest.mark.parametrize("x_dtype,y_dtype", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)], ids=str)
@pytest.mark.parametrize("H", HS)
def test_forward(bi, H, x_dtype, y_dtype):
    for M, pad, affine in ((1, 0, True), (7, 8, False), (33, 16, True)):
        banner(f"layer norm M={M} H={H} {x_dtype} -> {y_dtype}")
        x = rows(M, H, H + M, x_dtype, pad=pad)
        w, b = (vec(H, 1, 1.0), vec(H, 2)) if affine else (None, None)
        y, m, r = bi.bi_layer_norm(x, w, b, 1e-5, out_dtype=y_dtype, save_stats=True)
        assert y.dtype == y_dtype and m.dtype == r.dtype == F32
        yd, md, rd, ey, em, er = ref.norm(x, w, b, 1e-5, y_dtype)
        within(y, yd, ey, "y")
        within(m, md, em + 1e-37, "mean")
        within(r, rd, er, "rstd")
        assert torch.equal(bi.bi_layer_norm(x, w, b, 1e-5, out_dtype=y_dtype), y)


def test_more_rows_than_one_launch_keeps_busy(bi):
    """Workgroups that take several rows each, with a ragged last round."""
    for M, H in ((9001, 264), (5003, 1032)):
        banner(f"layer norm M={M} H={H}")
        x, w, b = rows(M, H, M, BF), vec(H, 1, 1.0), vec(H, 2)
        y, m, r = bi.bi_layer_norm(x, w, b, save_stats=True)
        yd, md, rd, ey, em, er = ref.norm(x, w, b, 1e-5, BF)
        within(y, yd, ey, "y")
        within(m, md, em, "mean")
        within(r, rd, er, "rstd")


@pytest.mark.parametrize("H", [512, 1000, 4096, 6000, 12288])
def test_rows_do_not_depend_on_the_batch(bi, H):
    x, dy, w, b = rows(3000, H, 5, BF), rows(3000, H, 6, BF), vec(H, 1, 1.0), vec(H, 2)
    y, m, r = bi.bi_layer_norm(x, w, b, save_stats=True)
    dx, _, _ = bi.bi_layer_norm_bwd(dy, x, m, r, w)
    for at, n in ((0, 1), (17, 1), (2999, 1), (100, 33), (1000, 1025)):
        s = slice(at, at + n)
        ys, ms, rs = bi.bi_layer_norm(x[s], w, b, save_stats=True)
        assert torch.equal(ys, y[s]) and torch.equal(ms, m[s]) and torch.equal(rs, r[s])
        assert torch.equal(bi.bi_layer_norm_bwd(dy[s], x[s], m[s].clone(), r[s].clone(), w)[0], dx[s])
        # nor on which outputs are wanted
        assert torch.equal(bi.bi_layer_norm_bwd(dy[s], x[s], m[s].clone(), r[s].clone(), w, need_dw=False, need_db=False)[0], dx[s])


@pytest.mark.parametrize("d_dtype,x_dtype", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)], ids=str)
@pytest.mark.parametrize("H", HS)
def test_backward(bi, H, d_dtype, x_dtype):
    for M, pad, affine in ((1, 0, True), (19, 8, False), (300, 16, True)):
        banner(f"layer norm backward M={M} H={H} {d_dtype} {x_dtype}")
        x, dy = rows(M, H, H + M, x_dtype, pad=pad), rows(M, H, 7 + M, d_dtype, pad=2 * pad)
        w = vec(H, 3, 1.0) if affine else None
        _, m, r = bi.bi_layer_norm(x, w, None, save_stats=True)
        dx, dw, db = bi.bi_layer_norm_bwd(dy, x, m, r, w)
        assert dx.dtype == x_dtype and dw.dtype == db.dtype == F32
        dxd, dwd, dbd, ex, ew, eb = ref.norm_bwd(dy, x, m, r, w, x_dtype)
        within(dx, dxd, ex, "dx")
        within(dw, dwd, ew, "dw")
        within(db, dbd, eb, "db")


def test_backward_over_many_rows(bi):
    for M, H in ((1024, 264), (1025, 264), (5001, 520), (4100, 2048), (8500, 256)):
        banner(f"layer norm backward M={M} H={H}")
        x, dy, w = rows(M, H, 1, BF), rows(M, H, 2, BF), vec(H, 3, 1.0)
        _, m, r = bi.bi_layer_norm(x, w, None, save_stats=True)
        got = bi.bi_layer_norm_bwd(dy, x, m, r, w)
        dxd, dwd, dbd, ex, ew, eb = ref.norm_bwd(dy, x, m, r, w, BF)
        for t, d, e, what in zip(got, (dxd, dwd, dbd), (ex, ew, eb), ("dx", "dw", "db")):
            within(t, d, e, what)
        again = bi.bi_layer_norm_bwd(dy, x, m, r, w)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_each_output_alone(bi):
    M, H = 77, 1032
    x, dy, w = rows(M, H, 1, BF), rows(M, H, 2, F32), vec(H, 3, 1.0)
    _, m, r = bi.bi_layer_norm(x, w, None, save_stats=True)
    full = bi.bi_layer_norm_bwd(dy, x, m, r, w)
    for i in range(3):
        want = [j == i for j in range(3)]
        got = bi.bi_layer_norm_bwd(dy, x, m, r, w, need_dx=want[0], need_dw=want[1], need_db=want[2])
        assert [t is not None for t in got] == want and torch.equal(got[i], full[i])


def test_no_rows(bi):
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    assert bi.bi_layer_norm(x).shape == (0, 64)
    s = torch.empty(0, dtype=F32, device="cuda")
    dx, dw, db = bi.bi_layer_norm_bwd(x, x, s, s)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_rows_of_extreme_values(bi):
    H = 264
    x = torch.zeros((8, H), dtype=F32, device="cuda")
    x[1] = 5.0                                              # no variance: y = b
    x[2, 3] = float("inf")
    x[3, 100] = float("nan")
    x[4] = torch.arange(H, device="cuda") * 1e-30           # variance far below eps
    x[5] = 1e4 + 1e-2 * (torch.arange(H, device="cuda") % 2)  # a mean far from the spread
    x[6] = rows(1, H, 1, F32)[0]
    x[7] = 1e18 * rows(1, H, 2, F32)[0]
    b = vec(H, 2)
    y, m, r = bi.bi_layer_norm(x, None, b, save_stats=True)
    ok = torch.tensor([0, 1, 4, 5, 6, 7])
    yd, md, rd, ey, em, er = ref.norm(x[ok], None, b, 1e-5, F32)
    within(y[ok], yd, ey, "y")
    within(m[ok], md, em + 1e-37, "mean")
    assert torch.equal(y[0], b) and torch.equal(y[1], b)
    assert torch.isnan(y[2]).any() and torch.isnan(y[3]).all()      # and no other row
    dx, _, _ = bi.bi_layer_norm_bwd(torch.ones_like(x), x, m, r)
    assert torch.isfinite(dx[ok]).all() and torch.isnan(dx[3]).all()


def test_outputs_in_place_and_untouched_surroundings(bi):
    M, H = 21, 72
    x, w = rows(M, H, 1, BF), vec(H, 1, 1.0)
    want = bi.bi_layer_norm(x, w)
    buf = torch.full((M + 2, H + 24), 7.0, dtype=BF, device="cuda")
    assert bi.bi_layer_norm(x, w, out=buf[1:-1, 8:8 + H]).data_ptr() == buf[1:-1, 8:8 + H].data_ptr()
    assert torch.equal(buf[1:-1, 8:8 + H], want)
    buf[1:-1, 8:8 + H] = 7.0
    assert (buf == 7.0).all()
    y = x.contiguous().clone()
    bi.bi_layer_norm(y, w, out=y)
    assert torch.equal(y, want)


def test_refusals_on_the_gpu(bi):
    x = rows(4, 64, 1, BF)
    s = torch.zeros(4, device="cuda")
    many, ms = rows(5000, 64, 1, BF), torch.zeros(5000, device="cuda")        # enough rows to need a workspace
    for call in (lambda: bi.bi_layer_norm(x, vec(32, 1)), lambda: bi.bi_layer_norm(x, vec(64, 1).cpu()),
                 lambda: bi.bi_layer_norm(x, vec(128, 1)[::2]), lambda: bi.bi_layer_norm(x, vec(72, 1)[1:65]),
                 lambda: bi.bi_layer_norm(x, out=x[:3]), lambda: bi.bi_layer_norm(x.t().contiguous().t()),
                 lambda: bi.bi_layer_norm_bwd(x, x[:3], s, s), lambda: bi.bi_layer_norm_bwd(x, x, s[:3], s),
                 lambda: bi.bi_layer_norm_bwd(x, x.cpu(), s, s),
                 lambda: bi.bi_layer_norm_bwd(many, many, ms, ms, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bi.bi_layer_norm(x, vec(64, 1).to(BF)), lambda: bi.bi_layer_norm_bwd(x, x, s.double(), s)):
        with pytest.raises(TypeError):
            call()
    for eps in (-1.0, float("nan")):
        with pytest.raises(bi.BIError):
            bi.bi_layer_norm(x, eps=eps)


def test_graph_replays_and_streams(bi):
    M, H = 300, 2056
    x, dy, w, b = rows(M, H, 1, BF), rows(M, H, 2, BF), vec(H, 1, 1.0), vec(H, 2)

    def step():
        y, m, r = bi.bi_layer_norm(x, w, b, save_stats=True)
        return (y, m, r) + bi.bi_layer_norm_bwd(dy, x, m, r, w)

    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(3):
        for t in out:
            t.zero_()
        keep = x.clone()
        x.mul_(1 + i)
        eager = [t.clone() for t in step()]
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
        x.copy_(keep)


@pytest.mark.parametrize("M", [1025, 3000])
def test_partials_in_graphs_and_on_two_streams(bi, M):
    """The backward pass whose partials go through a workspace: captured and replayed among
    eager calls, and two of them under way on two streams at once."""
    H = 2056
    w, b = vec(H, 1, 1.0), vec(H, 2)
    ins = [(rows(M, H, i, BF), rows(M, H, 10 + i, F32)) for i in range(2)]

    def step(x, dy):
        y, m, r = bi.bi_layer_norm(x, w, b, save_stats=True)
        return (y, m, r) + bi.bi_layer_norm_bwd(dy, x, m, r, w)

    want = [[t.clone() for t in step(*i)] for i in ins]
    assert bi.lib().bi_layer_norm_bwd_workspace_size(M, H) > 0 and not torch.equal(want[0][4], want[1][4])
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(step(*ins[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for run in got[k] for a, b in zip(run, want[k]))
    x, dy = (t.clone() for t in ins[0])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(step(x, dy))
    for i in (0, 1, 0):
        x.copy_(ins[i][0])
        dy.copy_(ins[i][1])
        for g, out in zip(graphs, outs):
            for t in out:
                t.zero_()
            g.replay()
            step(*ins[1 - i])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
