"""The feed-forward operators on the host: what the C entry points and the
binding refuse, workspace sizes, and the 64-bit references against differences
and hand-worked values.  Nothing here needs a GPU."""
import pytest

torch = pytest.importorskip("torch")

from tests import ffn_ref as ref

bi = pytest.importorskip("deterministic_persistent_gemm_amd")
L = bi.lib()
P = 0x10000          # aligned, never dereferenced by validation
BIG = 1 << 62


def gated(x=P, ldx=64, w=P, ldw=64, gate=0, y=P, ldy=32, h=P, ldh=64, M=4, I=32, H=64):
    return L.bi_gated_linear_bf16(x, ldx, w, ldw, gate, y, ldy, h, ldh, M, I, H, None)


def gated_bwd(dy=P, lddy=32, x=P, ldx=64, w=P, ldw=64, h=P, ldh=64, gate=0, dx=P, lddx=64, dw=P, dt=1, lddw=64, M=4, I=32, H=64,
              ws=P, n=1 << 20):
    return L.bi_gated_linear_bf16_bwd(dy, lddy, x, ldx, w, ldw, h, ldh, gate, dx, lddx, dw, dt, lddw, M, I, H, ws, n, None)


def linear_bwd(dy=P, lddy=32, x=P, ldx=64, w=P, ldw=64, dx=P, lddx=64, dw=P, dt=1, lddw=64, db=P, M=4, N=32, K=64):
    return L.bi_linear_bf16_bwd(dy, lddy, x, ldx, w, ldw, dx, lddx, dw, dt, lddw, db, M, N, K, None)


def quantize(x=P, dt=1, ldx=64, q=P, ldq=32, s=P, lds=4, rows=4, K=64):
    return L.bi_quantize_mxfp4(x, dt, ldx, q, ldq, s, lds, rows, K, None)


def dequantize(q=P, ldq=32, s=P, lds=4, y=P, dt=1, ldy=64, rows=4, K=64):
    return L.bi_dequantize_mxfp4(q, ldq, s, lds, y, dt, ldy, rows, K, None)


def mx(xq=P, ldxq=32, xs=P, ldxs=4, wq=P, ldwq=32, ws=P, ldws=4, b=P, y=P, dt=1, ldy=32, M=4, N=32, K=64):
    return L.bi_linear_mxfp4(xq, ldxq, xs, ldxs, wq, ldwq, ws, ldws, b, y, dt, ldy, M, N, K, None)


INVALID = [
    (gated, dict(gate=2)), (gated, dict(gate=-1)), (gated, dict(x=None)), (gated, dict(w=None)), (gated, dict(y=None)),
    (gated, dict(x=P + 8)), (gated, dict(h=P + 2)), (gated, dict(ldx=56)), (gated, dict(ldx=68)), (gated, dict(ldw=63)),
    (gated, dict(ldy=24)), (gated, dict(ldh=56)), (gated, dict(M=-1)), (gated, dict(I=-16)), (gated, dict(ldx=BIG)),
    (gated_bwd, dict(dy=None)), (gated_bwd, dict(h=None)), (gated_bwd, dict(x=None)), (gated_bwd, dict(w=None)),
    (gated_bwd, dict(gate=7)), (gated_bwd, dict(dt=2)), (gated_bwd, dict(lddw=60)), (gated_bwd, dict(lddx=32)),
    (gated_bwd, dict(dw=P + 4)), (gated_bwd, dict(ldh=32)), (gated_bwd, dict(M=0, dw=P + 4)),
    (linear_bwd, dict(dy=None)), (linear_bwd, dict(x=None)), (linear_bwd, dict(w=None)), (linear_bwd, dict(db=P + 4)),
    (linear_bwd, dict(dt=5)), (linear_bwd, dict(lddy=31)), (linear_bwd, dict(K=-32)), (linear_bwd, dict(M=0, lddw=8)),
    (quantize, dict(x=None)), (quantize, dict(q=None)), (quantize, dict(s=None)), (quantize, dict(s=P + 2)), (quantize, dict(lds=3)),
    (quantize, dict(lds=1)), (quantize, dict(ldq=40)), (quantize, dict(ldq=16)), (quantize, dict(dt=3)), (quantize, dict(ldx=66)),
    (dequantize, dict(y=None)), (dequantize, dict(ldy=32)), (dequantize, dict(dt=-1)), (dequantize, dict(q=P + 1)),
    (mx, dict(xq=None)), (mx, dict(xs=None)), (mx, dict(wq=None)), (mx, dict(ws=None)), (mx, dict(b=P + 4)), (mx, dict(y=P + 2)),
    (mx, dict(ldxs=6)), (mx, dict(ldwq=24)), (mx, dict(ldy=16)), (mx, dict(dt=9)), (mx, dict(M=-3)),
]


@pytest.mark.parametrize("fn,kw", INVALID, ids=lambda v: v.__name__ if callable(v) else "-".join(map(str, v)))
def test_invalid_arguments(fn, kw):
    assert fn(**kw) == bi.BI_EINVAL


UNSUPPORTED = [
    (gated, dict(I=24)), (gated, dict(I=0)), (gated, dict(H=48)), (gated, dict(H=0)), (gated, dict(M=(1 << 30) + 1)),
    (gated, dict(ldw=1 << 30, ldx=64)), (gated, dict(ldx=1 << 32)),
    (gated_bwd, dict(I=40)), (gated_bwd, dict(H=33)), (gated_bwd, dict(ldx=1 << 32)),
    (linear_bwd, dict(N=8)), (linear_bwd, dict(K=16)), (linear_bwd, dict(ldw=1 << 32)), (linear_bwd, dict(lddy=1 << 32)),
    (quantize, dict(K=48)), (dequantize, dict(K=16)), (mx, dict(K=80)), (mx, dict(N=8)), (mx, dict(ldxq=1 << 32)),
    (mx, dict(M=1 << 30, N=1 << 29, ldy=1 << 29)),
]


@pytest.mark.parametrize("fn,kw", UNSUPPORTED, ids=lambda v: v.__name__ if callable(v) else "-".join(map(str, v)))
def test_unsupported_sizes(fn, kw):
    assert fn(**kw) == bi.BI_EUNSUPPORTED


def test_more_workgroups_than_a_launch_holds():
    """2^32 threads and more are refused, not handed to the runtime."""
    M = 1 << 30
    assert gated(M=M, I=16, H=32) == bi.BI_EUNSUPPORTED
    assert mx(M=M, N=16, K=32, ldy=16) == bi.BI_EUNSUPPORTED
    assert linear_bwd(M=M, N=16, K=32, dw=None, db=None) == bi.BI_EUNSUPPORTED


def test_a_refused_backward_pass_enqueues_nothing():
    """The gated layer's too: its elementwise part is a launch of its own, which
    without a GPU would be a HIP error."""
    M = 1 << 30
    n = L.bi_gated_linear_bwd_workspace_size(M, 16)
    for kw in (dict(dw=None), dict()):
        assert gated_bwd(M=M, I=16, H=32, n=n, **kw) == bi.BI_EUNSUPPORTED


def test_nothing_to_do():
    assert gated(M=0, x=None, y=None) == bi.BI_OK
    assert gated_bwd(dx=None, dw=None) == bi.BI_OK
    assert gated_bwd(M=0, dw=None, ws=None, n=0) == bi.BI_OK
    assert linear_bwd(dx=None, dw=None, db=None) == bi.BI_OK
    assert linear_bwd(M=0, dw=None, db=None) == bi.BI_OK
    assert quantize(rows=0, x=None) == dequantize(rows=0, q=None) == mx(M=0, xq=None) == bi.BI_OK


def test_workspace_sizes_and_refusals():
    need = L.bi_gated_linear_bwd_workspace_size(4, 32)
    assert need == bi.WS_COUNTER_BYTES + 4 * 64 * 2
    assert gated_bwd(ws=None) == gated_bwd(n=need - 1) == gated_bwd(ws=P + 8) == bi.BI_EWORKSPACE
    for args in ((0, 32), (-1, 32), (4, 24), (4, 0)):
        assert L.bi_gated_linear_bwd_workspace_size(*args) == 0
    assert L.bi_gated_linear_bwd_workspace_size(1 << 30, 1 << 20) == bi.WS_COUNTER_BYTES + (1 << 52)   # past 32 bits


# ------------------------------------------------------------------- the binding


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_before_it_enqueues():
    x, w = cpu(4, 64), cpu(64, 64)
    for call in (lambda: bi.bi_gated_linear_bf16(x, w.t()),                         # not on a GPU
                 lambda: bi.bi_gated_linear_bf16(x, cpu(33, 64).t()),               # odd number of weight rows
                 lambda: bi.bi_gated_linear_bf16(x, cpu(48, 64).t()),               # I = 24
                 lambda: bi.bi_gated_linear_bf16(cpu(4, 48), cpu(64, 48).t()),      # H = 48
                 lambda: bi.bi_gated_linear_bf16(cpu(64), w.t()),
                 lambda: bi.bi_linear_bf16_bwd(x, None, w.t()),                     # dw without x
                 lambda: bi.bi_linear_bf16_bwd(x, x, None),                         # dx without w
                 lambda: bi.bi_gated_linear_bf16_bwd(x, None, w.t(), x),
                 lambda: bi.bi_gated_linear_bf16_bwd(x, cpu(64), None, x, need_dx=False),       # 1-D x
                 lambda: bi.bi_gated_linear_bf16_bwd(x, x, cpu(64), x),                         # 1-D w
                 lambda: bi.bi_linear_bf16_bwd(x, cpu(64), None, need_dx=False),
                 lambda: bi.bi_linear_bf16_bwd(x, x, cpu(64)),
                 lambda: bi.bi_quantize_mxfp4(cpu(4, 48)),
                 lambda: bi.bi_quantize_mxfp4(cpu(64)),
                 lambda: bi.bi_linear_mxfp4(cpu(4, 32, dtype=torch.uint8), cpu(4, 2, dtype=torch.uint8),
                                            cpu(16, 16, dtype=torch.uint8), cpu(16, 1, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bi.bi_quantize_mxfp4(cpu(4, 64, dtype=torch.float16)),
                 lambda: bi.bi_linear_bf16_bwd(x, x, w.t(), dw_dtype=torch.float16),
                 lambda: bi.bi_gated_linear_bf16(x.float(), w.t()),
                 lambda: bi.bi_dequantize_mxfp4(cpu(4, 32, dtype=torch.uint8), cpu(4, 2, dtype=torch.uint8), torch.float64)):
        with pytest.raises(TypeError):
            call()


# ----------------------------------------------------------------- the references


@pytest.mark.parametrize("gate", [0, 1])
def test_activation_derivative_against_differences(gate):
    g = torch.linspace(-12, 12, 4001, dtype=torch.float64)
    e = 1e-5
    diff = (ref.act(g + e, gate)[0] - ref.act(g - e, gate)[0]) / (2 * e)
    # central differences: e^2 / 6 of a third derivative below 2, and cancellation of 1e-16 * 12 / e
    assert torch.allclose(ref.act(g, gate)[1], diff, rtol=0, atol=1e-9)
    assert ref.act(g, gate)[1].abs().max() < ref.ACT_SLOPE


@pytest.mark.parametrize("gate", [0, 1])
def test_gated_backward_reference_against_differences(gate):
    g = torch.Generator().manual_seed(gate)
    M, H, I = 3, 4, 5
    x, w, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((M, H), (2 * I, H), (M, I)))

    def value(x, w):
        h = x @ w.t()
        return float((ref.act(h[:, :I], gate)[0] * h[:, I:] * dy).sum())

    dx, dw, _, _ = ref.gated_bwd(dy, x, w, x @ w.t(), gate)
    e = 1e-6
    for t, grad in ((x, dx), (w, dw)):
        for i in range(t.numel()):
            keep = float(t.view(-1)[i])
            t.view(-1)[i] = keep + e
            up = value(x, w)
            t.view(-1)[i] = keep - e
            down = value(x, w)
            t.view(-1)[i] = keep
            assert abs((up - down) / (2 * e) - float(grad.view(-1)[i])) < 1e-7


def test_quantize_reference_by_hand():
    x = torch.zeros((3, 32), dtype=torch.float32)
    x[0, :9] = torch.tensor([7.9, 5.0, -5.01, 0.25, 0.2501, -0.75, 1.25, 2.5, -3.5])    # scale 1
    x[1, :3] = torch.tensor([3.0, 0.125, -0.374])                                      # scale 1/2
    code, s = ref.mx_quantize(x)
    assert s[:, 0].tolist() == [127, 126, 0]
    assert code[0, :9].tolist() == [7, 6, 15, 0, 1, 10, 2, 4, 14]
    assert code[1, :3].tolist() == [7, 0, 9]                                           # 6, 0.25 (a tie, to 0), -0.748
    assert not code[2].any()
    assert ref.mx_values(code, s)[0, :9].tolist() == [6.0, 4.0, -6.0, 0.0, 0.5, -1.0, 1.0, 2.0, -4.0]
    assert torch.equal(ref.unpack(ref.pack(code)), code)
