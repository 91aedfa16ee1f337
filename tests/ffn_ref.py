"""Plain 64-bit forms of the feed-forward operators and the error bounds their
kernels are held to.

Every bound is worked out from the arithmetic: a stored value is within half a
step of what was rounded (bf16 2^-8, fp32 2^-24, relative), and an fp32 sum of n
products, in whatever order and grouping, is within n 2^-24 (plus one rounding
per product) of the sum of the products' magnitudes.
"""
import math

import torch

HALF_BF16, HALF_F32 = 2.0 ** -8, 2.0 ** -24
C = math.sqrt(2.0 / math.pi)
# |act'| of either gate stays below this (gelu: 1.129, silu: 1.0998)
ACT_SLOPE = 1.13
# relative error of an fp32 activation: exp's argument carries a few roundings
# of a magnitude of at most 88 (beyond it the value is below fp32's range)
ACT_REL = 2.0 ** -14
TINY = 1e-30


def act(g, gate):
    """act(g) and act'(g); gate 0: silu, 1: gelu (tanh).  The tanh form's
    (1 + tanh z) / 2 is computed as the equal 1 / (1 + exp(-2 z)): in binary64
    1 + tanh z is off by 2^-53, which for z = -16 is a hundredth of its value."""
    if gate == 0:
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    z2 = 2 * C * (g + 0.044715 * g ** 3)
    s, up = torch.sigmoid(z2), torch.sigmoid(-z2)
    return g * s, s + g * s * up * 2 * C * (1 + 3 * 0.044715 * g * g)


def mm(a, b):
    return torch.mm(a.double(), b.double())


def sum_bound(a, b, k):
    """Bound of an fp32 sum of k products against the exact one."""
    return (k + 1) * HALF_F32 * torch.mm(a.double().abs(), b.double().abs())


def gated(x, w13, gate):
    I = w13.shape[0] // 2
    h = mm(x, w13.t().contiguous())
    a, _ = act(h[:, :I], gate)
    y = a * h[:, I:]
    eh = sum_bound(x, w13.t().contiguous(), x.shape[1])
    ey = (ACT_SLOPE * eh[:, :I] * (h[:, I:].abs() + eh[:, I:]) + a.abs() * eh[:, I:] + ACT_REL * y.abs())
    return y, h, ey + HALF_BF16 * (y.abs() + ey) + TINY, eh + HALF_BF16 * (h.abs() + eh) + TINY


def gate_bwd(dy, h, gate):
    I = h.shape[1] // 2
    g, u, d = h[:, :I].double(), h[:, I:].double(), dy.double()
    a, da = act(g, gate)
    return torch.cat((d * u * da, d * a), dim=1)


def gated_bwd(dy, x, w13, h, gate):
    """dx, dw and their bounds: dh is rounded to bf16 once, products are fp32 sums."""
    dh = gate_bwd(dy, h, gate)
    # act' is a difference of terms of magnitude up to |g| + 1: absolute error there
    g, u, d = h[:, :h.shape[1] // 2].double(), h[:, h.shape[1] // 2:].double(), dy.double()
    edh = torch.cat((d.abs() * u.abs() * (g.abs() + 1) * ACT_REL, d.abs() * g.abs() * ACT_REL), dim=1)
    edh = edh + HALF_BF16 * (dh.abs() + edh) + TINY
    w, xd = w13.double(), x.double()
    dx = torch.mm(dh, w)
    edx = torch.mm(edh, w.abs()) + (dh.shape[1] + 1) * HALF_F32 * torch.mm(dh.abs() + edh, w.abs())
    dht = dh.t().contiguous()
    dw = torch.mm(dht, xd)
    edw = torch.mm(edh.t().contiguous(), xd.abs()) + (dh.shape[0] + 1) * HALF_F32 * torch.mm((dh.abs() + edh).t().contiguous(), xd.abs())
    return dx, dw, edx, edw


def stored(err, val, dtype):
    """A bound before rounding, after the value is stored as dtype."""
    return err + (HALF_BF16 if dtype == torch.bfloat16 else HALF_F32) * (val.abs() + err) + TINY


VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def mx_quantize(x):
    """Codes (unpacked, [M, K]) and scale bytes by the definition, in binary64:
    the nearest value by distance, ties to the even code."""
    M, K = x.shape
    b = x.double().cpu().reshape(M, K // 32, 32)
    top = b.abs().amax(dim=2)
    bad = ~torch.isfinite(b).all(dim=2)
    ex = torch.frexp(torch.where(bad, torch.ones_like(top), top)).exponent - 1
    s = torch.where((top == 0) & ~bad, torch.full_like(ex, 0), (ex - 2 + 127).clamp(min=0))
    a = b.abs() * torch.exp2((127 - s).double())[:, :, None]
    code = torch.zeros(b.shape, dtype=torch.int64)
    dist = a.clone()
    for k in (2, 4, 6, 1, 3, 5, 7):
        d = (a - VALUES[k]).abs()
        code = torch.where(d < dist, k, code)
        dist = torch.minimum(d, dist)
    code = code + 8 * torch.signbit(b).long()
    code = torch.where(bad[:, :, None], 0, code)
    s = torch.where(bad, 255, s)
    return code.reshape(M, K), s


def mx_values(code, s):
    """The values [M, K] in binary64; NaN blocks are NaN."""
    t = torch.tensor(VALUES + tuple(-v for v in VALUES), dtype=torch.float64)
    M, K = code.shape
    v = t[code.cpu().long()].reshape(M, K // 32, 32)
    sc = torch.where(s.cpu() == 255, torch.full(s.shape, float("nan"), dtype=torch.float64),
                     torch.exp2(s.cpu().double() - 127))
    return (v * sc[:, :, None]).reshape(M, K)


def unpack(q):
    q = q.cpu().long()
    return torch.stack((q & 15, q >> 4), dim=2).reshape(q.shape[0], -1)


def pack(code):
    c = code.to(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()
