"""Every tile shape of the feed-forward products in its steady state: sizes from
ffn_shapes.py, inputs on which every sum is exact, so that a wrong ring slot,
scale group or ragged edge shows as a wrong value."""
import pytest

torch = pytest.importorskip("torch")

from tests import ffn_ref as ref
from tests import ffn_shapes
from tests.gpu_util import banner
from tests.test_ffn_gpu import gen, ints, padded, same, within

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("deterministic_persistent_gemm_amd")
BF = torch.bfloat16


@pytest.mark.parametrize("M,I,H", ffn_shapes.GATED)
def test_gated(M, I, H):
    banner(f"gated steady M={M} I={I} H={H}")
    g = gen(M + H + I)
    x, w = ints(g, (M, H), -3, 3), ints(g, (2 * I, H), -2, 2)
    xp, wp = padded(x)[0], padded(w)[0]
    wh = ref.mm(x, w.t().contiguous())
    for gate in (0, 1):
        y, h = bi.bi_gated_linear_bf16(xp, wp.t(), gate, save_h=True)
        same(h + 0.0, wh.to(BF) + 0.0, f"h, gate {gate}")
        wy = ref.act(wh[:, :I], gate)[0] * wh[:, I:]
        within(y, wy, (ref.HALF_BF16 + ref.ACT_REL) * (1 + ref.HALF_BF16) * wy.abs() + ref.TINY, f"y, gate {gate}")
        same(bi.bi_gated_linear_bf16(x[M - 1:], w.t(), gate), y[M - 1:], f"the last row alone, gate {gate}")


@pytest.mark.parametrize("M,N,K", ffn_shapes.MXFP4)
def test_mxfp4(M, N, K):
    """Codes under scales 1 and 2: products are multiples of 1/4 below 144, so sums
    of up to 2^24 / (4 * 144) = 29127 of them are exact in fp32."""
    banner(f"mxfp4 steady M={M} N={N} K={K}")
    g = gen(M + N + K)
    ops = []
    for rows in (M, N):
        code = torch.randint(0, 16, (rows, K), generator=g, device="cuda").cpu()
        s = torch.randint(127, 129, (rows, K // 32), generator=g, device="cuda").cpu()
        pad = torch.full((rows, (K // 32 + 3) // 4 * 4), 255, dtype=torch.uint8)       # past K: must not matter
        pad[:, :K // 32] = s
        ops += [padded(ref.pack(code).cuda(), 16, 255)[0], pad.cuda()[:, :K // 32], ref.mx_values(code, s).cuda()]
    xq, xs, xv, wq, ws, wv = ops
    bias = ints(g, (N,), -5, 5, torch.float32)
    want = torch.mm(xv, wv.t().contiguous())
    y = bi.bi_linear_mxfp4(xq, xs, wq, ws, out_dtype=torch.float32)
    same(y + 0.0, want.float() + 0.0, "fp32")
    same(bi.bi_linear_mxfp4(xq, xs, wq, ws, bias) + 0.0, (want + bias).to(BF) + 0.0, "bf16 with bias")
    same(bi.bi_linear_mxfp4(xq[M - 1:], xs[M - 1:], wq, ws, out_dtype=torch.float32), y[M - 1:], "the last row alone")


@pytest.mark.parametrize("M,N,K", ffn_shapes.LINEAR_BWD)
def test_linear_bwd(M, N, K):
    banner(f"linear_bwd steady M={M} N={N} K={K}")
    g = gen(M + N + K)
    dy, x, w = ints(g, (M, N), -3, 3), ints(g, (M, K), -3, 3), ints(g, (N, K), -3, 3)
    dyp, xp, wp = padded(dy)[0], padded(x, 16)[0], padded(w, 24)[0]
    wx, ww, wb = ref.mm(dy, w), ref.mm(dy.t().contiguous(), x), dy.double().sum(0)
    for dt in (BF, torch.float32):
        dx, dw, db = bi.bi_linear_bf16_bwd(dyp, xp, wp.t(), dw_dtype=dt)
        same(dx + 0.0, wx.to(BF) + 0.0, f"dx beside {dt}")
        same(dw + 0.0, ww.to(dt) + 0.0, f"dw {dt}")
        same(db + 0.0, wb.float() + 0.0, f"db beside {dt}")
