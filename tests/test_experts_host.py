"""Layer norm, products grouped by expert and 8-bit products on the host: what
the C entry points and the binding refuse, workspace sizes, and the 64-bit
references against differences and hand-worked values.  Nothing here needs a GPU."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from tests import experts_ref as ref
from tests import experts_shapes as shapes

bi = pytest.importorskip("deterministic_persistent_gemm_amd")
from deterministic_persistent_gemm_amd import _build
L = bi.lib()
P = 0x10000          # aligned, never dereferenced by validation
BIG = 1 << 62


def norm(x=P, xt=1, ldx=64, w=P, b=P, eps=1e-5, y=P, yt=1, ldy=64, mean=P, rstd=P, M=4, H=64):
    return L.bi_layer_norm(x, xt, ldx, w, b, eps, y, yt, ldy, mean, rstd, M, H, None)


def norm_bwd(dy=P, dt=1, lddy=64, x=P, xt=1, ldx=64, mean=P, rstd=P, w=P, dx=P, lddx=64, dw=P, db=P, M=4, H=64, ws=P, n=1 << 24):
    return L.bi_layer_norm_bwd(dy, dt, lddy, x, xt, ldx, mean, rstd, w, dx, lddx, dw, db, M, H, ws, n, None)


def grouped(x=P, ldx=64, w=P, ldw=64, sw=2048, ends=P, E=4, y=P, yt=1, ldy=32, T=4, N=32, K=64):
    return L.bi_grouped_linear_bf16(x, ldx, w, ldw, sw, ends, E, y, yt, ldy, T, N, K, None)


def grouped_bwd(dy=P, lddy=32, x=P, ldx=64, w=P, ldw=64, sw=2048, ends=P, E=4, dx=P, lddx=64, dw=P, dt=1, lddw=64, sdw=2048,
                T=4, N=32, K=64):
    return L.bi_grouped_linear_bf16_bwd(dy, lddy, x, ldx, w, ldw, sw, ends, E, dx, lddx, dw, dt, lddw, sdw, T, N, K, None)


def quantize(x=P, dt=1, ldx=64, q=P, ldq=64, s=P, rows=4, K=64):
    return L.bi_quantize_int8(x, dt, ldx, q, ldq, s, rows, K, None)


def int8(xq=P, ldxq=64, xs=P, wq=P, ldwq=64, ws=P, b=P, y=P, dt=1, ldy=32, M=4, N=32, K=64):
    return L.bi_linear_int8(xq, ldxq, xs, wq, ldwq, ws, b, y, dt, ldy, M, N, K, None)


def grouped_int8(xq=P, ldxq=64, xs=P, wq=P, ldwq=64, sw=2048, ws=P, ss=32, ends=P, E=4, y=P, dt=1, ldy=32, T=4, N=32, K=64):
    return L.bi_grouped_linear_int8(xq, ldxq, xs, wq, ldwq, sw, ws, ss, ends, E, y, dt, ldy, T, N, K, None)


INVALID = [
    (norm, dict(x=None)), (norm, dict(y=None)), (norm, dict(x=P + 8)), (norm, dict(w=P + 4)), (norm, dict(b=P + 8)),
    (norm, dict(mean=P + 2)), (norm, dict(rstd=P + 1)), (norm, dict(ldx=56)), (norm, dict(ldx=68)), (norm, dict(ldy=63)),
    (norm, dict(xt=2)), (norm, dict(yt=-1)), (norm, dict(eps=-1e-9)), (norm, dict(eps=float("nan"))), (norm, dict(eps=float("inf"))),
    (norm, dict(M=-1)), (norm, dict(H=-8)), (norm, dict(M=0, eps=-1.0)),
    (norm_bwd, dict(dy=None)), (norm_bwd, dict(x=None)), (norm_bwd, dict(mean=None)), (norm_bwd, dict(rstd=None)),
    (norm_bwd, dict(rstd=P + 2)), (norm_bwd, dict(dx=P + 8)), (norm_bwd, dict(dw=P + 4)), (norm_bwd, dict(db=P + 4)),
    (norm_bwd, dict(lddx=60)), (norm_bwd, dict(lddy=32)), (norm_bwd, dict(dt=3)), (norm_bwd, dict(xt=3)), (norm_bwd, dict(w=P + 4)),
    (norm_bwd, dict(M=0, dw=P + 4)),
    (grouped, dict(x=None)), (grouped, dict(w=None)), (grouped, dict(ends=None)), (grouped, dict(ends=P + 4)), (grouped, dict(y=None)),
    (grouped, dict(sw=-8)), (grouped, dict(sw=2044)), (grouped, dict(sw=BIG)), (grouped, dict(ldx=63)), (grouped, dict(ldw=56)),
    (grouped, dict(ldy=16)), (grouped, dict(yt=2)), (grouped, dict(T=-1)), (grouped, dict(E=-1)), (grouped, dict(x=P + 2)),
    (grouped_bwd, dict(dy=None)), (grouped_bwd, dict(x=None)), (grouped_bwd, dict(w=None)), (grouped_bwd, dict(ends=None)),
    (grouped_bwd, dict(sw=4)), (grouped_bwd, dict(sdw=2040)), (grouped_bwd, dict(sdw=2050)), (grouped_bwd, dict(dt=7)),
    (grouped_bwd, dict(lddx=56)), (grouped_bwd, dict(lddw=32)), (grouped_bwd, dict(lddy=8)), (grouped_bwd, dict(T=0, dw=P + 4)),
    (grouped_bwd, dict(T=0, ends=None)), (grouped_bwd, dict(dx=P + 8)),
    (quantize, dict(x=None)), (quantize, dict(q=None)), (quantize, dict(s=None)), (quantize, dict(s=P + 2)), (quantize, dict(q=P + 8)),
    (quantize, dict(ldq=72)), (quantize, dict(ldq=48)), (quantize, dict(dt=4)), (quantize, dict(ldx=60)), (quantize, dict(rows=-2)),
    (int8, dict(xq=None)), (int8, dict(xs=None)), (int8, dict(wq=None)), (int8, dict(ws=None)), (int8, dict(ws=P + 4)),
    (int8, dict(xs=P + 2)), (int8, dict(b=P + 4)), (int8, dict(y=P + 8)), (int8, dict(ldxq=72)), (int8, dict(ldwq=32)),
    (int8, dict(ldy=24)), (int8, dict(dt=2)), (int8, dict(M=-1)),
    (grouped_int8, dict(xq=None)), (grouped_int8, dict(xs=None)), (grouped_int8, dict(ws=None)), (grouped_int8, dict(ends=None)),
    (grouped_int8, dict(sw=2056)), (grouped_int8, dict(ss=30)), (grouped_int8, dict(ss=-4)), (grouped_int8, dict(ldy=8)),
    (grouped_int8, dict(dt=2)), (grouped_int8, dict(E=-4)),
]


def ids(v):
    return v.__name__ if callable(v) else "-".join(map(str, v))


@pytest.mark.parametrize("fn,kw", INVALID, ids=ids)
def test_invalid_arguments(fn, kw):
    assert fn(**kw) == bi.BI_EINVAL


def test_expert_strides_that_pass_64_bits():
    """(N - 1) lddw + K past 2^63 is not taken for a small number; the least stride is."""
    assert grouped_bwd(dx=None, N=1 << 28, lddy=1 << 28, lddw=1 << 36, sdw=1 << 20) == bi.BI_EINVAL
    assert grouped_bwd(dx=None, N=(1 << 28) + 16, lddy=(1 << 28) + 16, lddw=1 << 39, sdw=1 << 39) == bi.BI_EINVAL
    least = 31 * 72 + 64
    for sdw in (least - 8, least):
        for dt in (0, 1):
            # an input that is refused later: only the stride tells the two calls apart
            got = grouped_bwd(E=4, lddw=72, sdw=sdw, dt=dt, lddy=1 << 32)
            assert got == (bi.BI_EINVAL if sdw < least else bi.BI_EUNSUPPORTED)


UNSUPPORTED = [
    (norm, dict(H=60)), (norm, dict(H=0)), (norm, dict(H=16392, ldx=16392, ldy=16392)), (norm, dict(M=(1 << 30) + 1)),
    (norm_bwd, dict(H=4)), (norm_bwd, dict(H=16392)),
    (grouped, dict(E=0)), (grouped, dict(E=1025)), (grouped, dict(N=24)), (grouped, dict(K=48)), (grouped, dict(N=0)),
    (grouped, dict(T=(1 << 30) + 1)), (grouped, dict(ldx=1 << 32)), (grouped, dict(ldw=1 << 32)),
    (grouped_bwd, dict(E=0)), (grouped_bwd, dict(E=2000)), (grouped_bwd, dict(N=8)), (grouped_bwd, dict(K=16)),
    (grouped_bwd, dict(ldw=1 << 32)), (grouped_bwd, dict(ldx=1 << 32)), (grouped_bwd, dict(lddy=1 << 32)),
    (quantize, dict(K=48)), (int8, dict(K=80)), (int8, dict(N=8)), (int8, dict(ldxq=1 << 32)),
    (int8, dict(K=131072, ldxq=131072, ldwq=131072)), (grouped_int8, dict(K=131072, ldxq=131072, ldwq=131072)),
    (grouped_int8, dict(E=0)), (grouped_int8, dict(E=1025)), (grouped_int8, dict(ldwq=1 << 32)),
]


@pytest.mark.parametrize("fn,kw", UNSUPPORTED, ids=ids)
def test_unsupported_sizes(fn, kw):
    assert fn(**kw) == bi.BI_EUNSUPPORTED


def test_more_workgroups_than_a_launch_holds():
    T = 1 << 30
    assert int8(M=T, N=16, K=32, ldy=16) == bi.BI_EUNSUPPORTED
    # 2^22 row tiles and more even of the largest shape, four columns of them
    assert grouped(T=T, N=1024, E=1024, ldy=1024) == bi.BI_EUNSUPPORTED
    assert grouped_int8(T=T, N=1024, E=1024, ldy=1024) == bi.BI_EUNSUPPORTED
    assert grouped_bwd(T=T, N=32, K=1024, ldx=1024, ldw=1024, lddx=1024, dw=None) == bi.BI_EUNSUPPORTED
    # dw alone: 2^32 tiles of 256 x 256
    n = 1 << 19
    assert grouped_bwd(dx=None, E=1024, N=n, K=n, lddy=n, ldx=n, lddw=n, sdw=n * n) == bi.BI_EUNSUPPORTED
    # ... and beside a dx that would fit: nothing is enqueued, which without a GPU would be a HIP error
    assert grouped_bwd(E=1024, N=n, K=n, lddy=n, ldx=n, ldw=n, lddx=n, lddw=n, sdw=n * n) == bi.BI_EUNSUPPORTED


def test_nothing_to_do():
    assert norm(M=0, x=None, y=None) == bi.BI_OK
    assert norm_bwd(dx=None, dw=None, db=None) == norm_bwd(M=0, dw=None, db=None, ws=None) == bi.BI_OK
    assert grouped(T=0, x=None, ends=None) == grouped_int8(T=0, xq=None, ends=None) == bi.BI_OK
    assert grouped_bwd(dx=None, dw=None) == grouped_bwd(T=0, dw=None, ends=None) == bi.BI_OK
    assert quantize(rows=0, x=None) == int8(M=0, xq=None) == bi.BI_OK


def test_workspace_sizes_and_refusals():
    need = L.bi_layer_norm_bwd_workspace_size(5000, 64)
    assert need > bi.WS_COUNTER_BYTES and (need - bi.WS_COUNTER_BYTES) % (2 * 64 * 4) == 0
    assert norm_bwd(M=5000, ws=None) == norm_bwd(M=5000, n=need - 1) == norm_bwd(M=5000, ws=P + 8) == bi.BI_EWORKSPACE
    assert norm_bwd(M=5000, dw=None, n=need - 1) == bi.BI_EWORKSPACE
    # a few rows need none; nor do sizes that are refused
    for args in ((1, 64), (0, 64), (-1, 64), (5000, 60), (5000, 0), (5000, 16392)):
        assert L.bi_layer_norm_bwd_workspace_size(*args) == 0
    # it does not grow with the batch for ever
    assert L.bi_layer_norm_bwd_workspace_size(1 << 20, 4096) == L.bi_layer_norm_bwd_workspace_size(1 << 30, 4096)


def test_tile_query_refusals():
    out = (bi._I32 * 8)()
    tile = L.bi_lab_grouped_tile
    assert tile(6, 4, 4, 32, 64, 1, out) == tile(0, 0, 4, 32, 64, 1, out) == tile(0, 4, 4, 32, 64, 3, out) == bi.BI_EINVAL
    assert tile(0, 4, 4, 32, 64, 1, None) == bi.BI_EINVAL
    assert tile(0, 4, 4, 24, 64, 1, out) == tile(0, 4, 0, 32, 64, 1, out) == tile(0, 4, 1025, 32, 64, 1, out) == bi.BI_EUNSUPPORTED


# ------------------------------------------------------------------- the binding


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_before_it_enqueues():
    x, w, ends = cpu(4, 64), cpu(2, 32, 64), cpu(2, dtype=torch.int64)
    f, i8 = cpu(4, dtype=torch.float32), torch.int8
    for call in (lambda: bi.bi_layer_norm(x),                                          # not on a GPU
                 lambda: bi.bi_layer_norm(cpu(64)), lambda: bi.bi_layer_norm(cpu(4, 60)),
                 lambda: bi.bi_layer_norm(cpu(4, 16392)), lambda: bi.bi_layer_norm(cpu(4, 0)),
                 lambda: bi.bi_layer_norm_bwd(cpu(64), x, f, f), lambda: bi.bi_layer_norm_bwd(cpu(4, 12), cpu(4, 12), f, f),
                 lambda: bi.bi_grouped_linear_bf16(x, w, ends),
                 lambda: bi.bi_grouped_linear_bf16(x, cpu(32, 64), ends),              # 2-D w
                 lambda: bi.bi_grouped_linear_bf16(cpu(64), w, ends),
                 lambda: bi.bi_grouped_linear_bf16(x, cpu(0, 32, 64), ends),
                 lambda: bi.bi_grouped_linear_bf16(x, cpu(2, 24, 64), ends),
                 lambda: bi.bi_grouped_linear_bf16(cpu(4, 48), cpu(2, 32, 48), ends),
                 lambda: bi.bi_grouped_linear_bf16_bwd(x, None, cpu(2, 64, 32), ends),          # dw without x
                 lambda: bi.bi_grouped_linear_bf16_bwd(x, x, None, ends),                       # dx without w
                 lambda: bi.bi_grouped_linear_bf16_bwd(x, x, cpu(64, 32), ends),
                 lambda: bi.bi_grouped_linear_bf16_bwd(x, x, cpu(2, 64, 32), cpu(2, 1, dtype=torch.int64)),
                 lambda: bi.bi_quantize_int8(x), lambda: bi.bi_quantize_int8(cpu(64)), lambda: bi.bi_quantize_int8(cpu(4, 48)),
                 lambda: bi.bi_linear_int8(cpu(4, 64, dtype=i8), f, cpu(32, 64, dtype=i8), f),
                 lambda: bi.bi_linear_int8(cpu(64, dtype=i8), f, cpu(32, 64, dtype=i8), f),
                 lambda: bi.bi_linear_int8(cpu(1, 131072, dtype=i8), f, cpu(16, 131072, dtype=i8), f),
                 lambda: bi.bi_grouped_linear_int8(cpu(4, 64, dtype=i8), f, cpu(2, 32, 64, dtype=i8), f, ends),
                 lambda: bi.bi_grouped_linear_int8(cpu(4, 64, dtype=i8), f, cpu(32, 64, dtype=i8), f, ends)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bi.bi_layer_norm(cpu(4, 64, dtype=torch.float16)),
                 lambda: bi.bi_layer_norm(x, out_dtype=torch.float64),
                 lambda: bi.bi_layer_norm_bwd(cpu(4, 64, dtype=torch.float64), x, f, f),
                 lambda: bi.bi_grouped_linear_bf16_bwd(x, x, cpu(2, 64, 64), ends, dw_dtype=torch.float16),
                 lambda: bi.bi_grouped_linear_bf16(x.float(), w, ends),
                 lambda: bi.bi_quantize_int8(cpu(4, 64, dtype=torch.float16)),
                 lambda: bi.bi_linear_int8(cpu(4, 64, dtype=i8), f, cpu(32, 64, dtype=i8), f, out_dtype=torch.int32)):
        with pytest.raises(TypeError):
            call()


def test_overlap_of_an_output_and_an_operand():
    """Against the bytes themselves, in every place of a small buffer."""
    def bytes_of(p, rows, ld, width):
        return {p + i * ld + j for i in range(rows) for j in range(width)}

    def refused(*a):
        try:
            bi._apart(*a, "call", "out")
            return False
        except ValueError:
            return True

    for rows, ld, width, ldq, widthq in ((3, 10, 4, 10, 3), (4, 7, 7, 7, 2), (1, 10, 4, 6, 5), (2, 9, 1, 9, 8), (2, 9, 2, 9, 8)):
        mine = bytes_of(100, rows, ld, width)
        for q in range(50, 160):
            assert refused(rows, 100, ld, width, q, ldq, widthq) == bool(mine & bytes_of(q, rows, ldq, widthq))
    assert not refused(0, 0, 64, 64, 0, 64, 64)
    # other pitches: nothing that shares a byte passes
    for q in range(50, 160):
        if bytes_of(100, 3, 10, 4) & bytes_of(q, 3, 8, 3):
            assert refused(3, 100, 10, 4, q, 8, 3)


def test_outputs_over_operands_are_refused(monkeypatch):
    """The calls on host tensors that say they are on a GPU, up to the point of the launch."""
    calls = []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(bi, "_call", lambda fn, name, *a: calls.append(name))
    i8 = torch.int8
    x, w, ends = cpu(4, 64), cpu(2, 64, 64), cpu(2, dtype=torch.int64)
    q, s, wq, ws = cpu(4, 64, dtype=i8), cpu(4, dtype=torch.float32), cpu(2, 64, 64, dtype=i8), cpu(2, 64, dtype=torch.float32)
    wide, wide8 = cpu(4, 128), cpu(4, 256, dtype=i8)
    over8 = wide8.view(torch.bfloat16)
    for call in (lambda: bi.bi_grouped_linear_bf16(x, w, ends, out=x),
                 lambda: bi.bi_grouped_linear_bf16(wide[:, :64], w, ends, out=wide[:, 56:120]),
                 lambda: bi.bi_grouped_linear_bf16_bwd(x, cpu(4, 64), w, ends, out_dx=x),
                 lambda: bi.bi_grouped_linear_bf16_bwd(x, None, w, ends, need_dw=False, out_dx=x),
                 lambda: bi.bi_grouped_linear_bf16_bwd(cpu(4, 64), x, w, ends, out_dx=x),
                 lambda: bi.bi_linear_int8(wide8[:, :64], s, wq[0], ws[0], out=over8[:, :64]),
                 lambda: bi.bi_grouped_linear_int8(wide8[:, 64:128], s, wq, ws, ends, out=over8[:, 56:120]),
                 lambda: bi.bi_layer_norm(wide[:, :64], out=wide[:, 32:96]),
                 lambda: bi.bi_layer_norm(x[:3], out=x[1:])):
        calls.clear()
        with pytest.raises(ValueError, match="overlap"):
            call()
    calls.clear()
    bi.bi_layer_norm(x, out=x)
    bi.bi_layer_norm(wide[:, :64], out=wide[:, 64:])
    bi.bi_grouped_linear_bf16(wide[:, :64], w, ends, out=wide[:, 64:])
    bi.bi_grouped_linear_bf16_bwd(wide[:, :64], cpu(4, 64), w, ends, out_dx=wide[:, 64:])
    bi.bi_grouped_linear_bf16_bwd(x, wide[:, :64], w, ends, need_dw=False, out_dx=wide[:, :64])      # x is not read
    bi.bi_linear_int8(wide8[:, :64], s, wq[0], ws[0], out=over8[:, 64:])
    bi.bi_grouped_linear_int8(wide8[:, 128:192], s, wq, ws, ends, out=over8[:, :64])
    assert len(calls) == 7


def test_import_beside_a_torch_without_gpu_support():
    """Recipe and workspace queries and refusals need no GPU entries of torch."""
    run = subprocess.run([sys.executable, "-c", """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import deterministic_persistent_gemm_amd as bi
assert bi.lib().bi_layer_norm_bwd_workspace_size(5000, 64) > 0
assert bi.grouped_tile(bi.BI_GROUPED_BF16, 4, 4, 32, 64)["rows"] >= 16
try:
    bi.bi_layer_norm(torch.zeros((4, 64)))
except ValueError:
    print("refused")
"""], capture_output=True, text=True, timeout=300, cwd=_build.ROOT)
    assert run.returncode == 0 and run.stdout.split() == ["refused"], run.stderr


# ----------------------------------------------------------------- the references


def test_norm_reference_against_differences():
    g = torch.Generator().manual_seed(0)
    M, H, eps = 3, 8, 1e-5
    x, w, b, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((M, H), (H,), (H,), (M, H)))

    def value():
        return float((ref.norm(x, w, b, eps, torch.float32)[0] * dy).sum())

    _, m, r, *_ = ref.norm(x, w, b, eps, torch.float32)
    dx, dw, db, *_ = ref.norm_bwd(dy, x, m, r, w, torch.float32)
    e = 1e-6
    for t, grad in ((x, dx), (w, dw), (b, db)):
        for i in range(t.numel()):
            keep = float(t.view(-1)[i])
            t.view(-1)[i] = keep + e
            up = value()
            t.view(-1)[i] = keep - e
            down = value()
            t.view(-1)[i] = keep
            assert abs((up - down) / (2 * e) - float(grad.view(-1)[i])) < 1e-7


def test_codes_by_hand():
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, 2.500001, -0.49999, 126.5, -127.0],        # scale 1
                      [0.0] * 8,
                      [1.0, float("inf"), 0, 0, 0, 0, 0, 0],
                      [2.0 ** -140, 0, 0, 0, 0, 0, 0, 0]])                                # far below the least scale
    q, s = ref.codes(x)
    assert q[0].tolist() == [127, 0, 2, -2, 3, 0, 126, -127] and s[0] == 1.0
    assert not q[1].any() and s[1] == 2.0 ** -126
    assert not q[2].any() and torch.isnan(s[2])
    assert not q[3].any() and s[3] == 2.0 ** -126


def test_scales_beside_the_quotient():
    """max|x| times fp32's 1/127 is max|x| / 127 rounded once or the number next below,
    for every fp32 mantissa; codes differ by one at most, and only next to halfway points,
    and either is within half a scale of its value."""
    top = 1 + torch.arange(1 << 23, dtype=torch.float64) / (1 << 23)
    step = (top.float() * torch.tensor(1.0 / 127.0)).view(torch.int32) - (top / 127).float().view(torch.int32)
    assert step.min() == -1 and step.max() == 0
    m = 1 + torch.arange(128, dtype=torch.float64) / 128
    x = m[:, None] * torch.cat((torch.tensor([1.0, 0.5, -0.5], dtype=torch.float64), torch.linspace(-1, 1, 61, dtype=torch.float64)))
    x = x.to(torch.bfloat16)
    q, s = ref.codes(x)
    sq = (x.double().abs().amax(1) / 127).float()
    v = x.double() / sq.double()[:, None]
    other = torch.round(v)
    assert int((s != sq).sum()) == 6 and ((s.view(torch.int32) - sq.view(torch.int32)) >= -1).all()
    assert ((q.double() * s.double()[:, None] - x.double()).abs() <= 0.5 * s.double()[:, None]).all()
    far = (v - torch.floor(v) - 0.5).abs() > 127 * 2.0 ** -23
    assert (q.double() == other)[far].all() and (q.double() - other).abs().max() == 1
    assert (q[s != sq, 1] == 64).all() and (other[s != sq, 1] == 63).all()


def test_spans_of_any_ends():
    assert ref.spans([2, 2, 5], 6) == [(0, 2), (2, 2), (2, 5)]
    assert ref.spans([3, 1, -7, 99], 6) == [(0, 3), (3, 3), (3, 3), (3, 6)]


# ------------------------------------------------------------------ the tile shapes


def steady(t, k):
    """At least two stages past the ring."""
    return -(-k // t["slice_k"]) >= (t["ring_stages"] + 1) * t["stage_slices"] + 1


def test_every_int8_shape_is_tested_past_its_ring():
    seen = set()
    for M, N, K in shapes.INT8:
        for dt in (bi.BI_BF16, bi.BI_F32):
            t = bi.ffn_tile(bi.BI_FFN_INT8, M, N, K, dt)
            if steady(t, K):
                seen.add((t["shape"], dt))
    assert seen == {(i, dt) for i in range(9) for dt in (bi.BI_BF16, bi.BI_F32)}


@pytest.mark.parametrize("op,n,sizes", [
    (bi.BI_GROUPED_BF16, 7, shapes.GROUPED), (bi.BI_GROUPED_INT8, 7, shapes.GROUPED),
    (bi.BI_GROUPED_DX, 6, shapes.GROUPED_BWD), (bi.BI_GROUPED_DX_ALONE, 6, shapes.GROUPED_BWD),
    (bi.BI_GROUPED_DW, 3, shapes.GROUPED_BWD), (bi.BI_GROUPED_DW_ALONE, 3, shapes.GROUPED_BWD)],
    ids=["bf16", "int8", "dx", "dx-alone", "dw", "dw-alone"])
def test_every_grouped_shape_is_tested_past_its_ring(op, n, sizes):
    dx, dw = op in (bi.BI_GROUPED_DX, bi.BI_GROUPED_DX_ALONE), op in (bi.BI_GROUPED_DW, bi.BI_GROUPED_DW_ALONE)
    dts = (bi.BI_BF16,) if dx else (bi.BI_BF16, bi.BI_F32)
    seen = set()
    for T, E, N, K in sizes:
        for dt in dts:
            t = bi.grouped_tile(op, T, E, N, K, dt)
            if steady(t, N if dx else max(shapes.counts(T, E)) if dw else K):
                seen.add((t["shape"], dt))
    assert seen == {(i, dt) for i in range(n) for dt in dts}


def test_counts_add_up():
    for T, E, _, _ in shapes.GROUPED + shapes.GROUPED_BWD:
        c = shapes.counts(T, E)
        assert len(c) == E and sum(c) == T and min(c) >= 0


PAIRS = """
#include "bi_grouped.hip"
#include <cstdio>
namespace bi { int device_cu_count() { return 256; } }
int main()
{
    bi::TileArgs a{}, b{};
    a.N = b.M = b.N = 512;
    const bi::GroupArgs q{nullptr, 4, 300, 0, 0};
    const int dx = bi::kNumDxShapes - 1, dw = bi::kNumDwShapes - 1;
    for (int i = 0; i < dx; ++i)
        printf("%d\\n", bi::run_both(a, q, i, b, q, dw, nullptr) == hipErrorInvalidConfiguration);
    for (int i = 0; i < dw; ++i)
        printf("%d\\n", bi::run_both(a, q, dx, b, q, i, nullptr) == hipErrorInvalidConfiguration);
}
"""


def test_a_pair_of_gradient_tiles_without_a_kernel_is_refused(tmp_path):
    """The largest tiles of one gradient beside smaller ones of the other: no kernel is built
    for them in one launch, and asking for it must not look like a launch.  The host
    half of the source alone, run without a GPU."""
    if not os.path.exists(_build.HIPCC):
        pytest.skip("no hipcc")
    src, exe = tmp_path / "pairs.hip", tmp_path / "pairs"
    src.write_text(PAIRS)
    subprocess.run([_build.HIPCC, "--offload-host-only", "-fuse-cuid=none", f"--offload-arch={_build.ARCH}", "-O0", "-std=c++17",
                    "-I", _build.INCLUDE, "-I", _build.CSRC, "-x", "hip", str(src), "-Wl,--defsym=__hip_fatbin=main", "-o", str(exe)],
                   check=True, timeout=300)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60,
                         env=dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1"))
    assert got.stdout.split() == ["1"] * 7
