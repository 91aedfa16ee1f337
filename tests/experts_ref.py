"""Plain 64-bit forms of the layer norm, the products grouped by expert and the
8-bit products, and the error bounds their kernels are held to.

Every bound is worked out from the arithmetic.  U = 2^-24 is half an fp32 step.
A sum of values through a tree of additions of depth D is off by at most D U
times the sum of their magnitudes; the norm's row sums have a depth of at most 16
(a thread's values) + 6 (a wave's lanes) + 16 (the waves) = 38.
"""
import torch

from tests.ffn_ref import stored

U = 2.0 ** -24
ROW_DEPTH = 38


def norm(x, w, b, eps, out_dtype):
    """y, mean, rstd and their bounds."""
    x = x.double().cpu()
    H = x.shape[1]
    w = torch.ones(H, dtype=torch.float64) if w is None else w.double().cpu()
    b = torch.zeros(H, dtype=torch.float64) if b is None else b.double().cpu()
    m = x.mean(dim=1, keepdim=True)
    d = x - m
    v = (d * d).mean(dim=1, keepdim=True)
    r = (v + eps) ** -0.5
    y = d * r * w + b
    # the mean: the sum's depth and the division; x - mean: that and its own rounding
    em = (ROW_DEPTH + 1) * U * x.abs().mean(dim=1, keepdim=True)
    ed = em + U * (d.abs() + em)
    # the variance: each square's error, its rounding, the sum's depth and the division
    ev = (2 * d.abs() * ed + ed * ed).mean(dim=1, keepdim=True) + (ROW_DEPTH + 2) * U * ((d.abs() + ed) ** 2).mean(dim=1, keepdim=True)
    # r: half the relative error of v + eps (its rounding included) and second order, a root, a division
    rel = ev / (v + eps) + U
    er = 0.5 * rel * (1 + 2 * rel) + 2 * U
    a = (d * r * w).abs()
    ey = a * (er + 2 * U) * (1 + er) + ed * r * (1 + er) * w.abs() + U * y.abs() + U * a
    return y, m[:, 0], r[:, 0], stored(ey, y, out_dtype), em[:, 0], (er * r)[:, 0]


def norm_bwd(dy, x, mean, rstd, w, x_dtype):
    """dx, dw, db at the given fp32 statistics, and their bounds."""
    dy, x = dy.double().cpu(), x.double().cpu()
    M, H = x.shape
    w = torch.ones(H, dtype=torch.float64) if w is None else w.double().cpu()
    m, r = mean.double().cpu()[:, None], rstd.double().cpu()[:, None]
    n = (x - m) * r
    g = dy * w
    c0, c1 = g.mean(dim=1, keepdim=True), (g * n).mean(dim=1, keepdim=True)
    dx = r * (g - (c0 + n * c1))
    k = 1 + 1e-3                                          # second-order terms
    en = 2 * U * n.abs() * k                              # a difference and a product
    eg = U * g.abs()
    e0 = (ROW_DEPTH + 2) * U * g.abs().mean(dim=1, keepdim=True) * k
    e1 = (ROW_DEPTH + 5) * U * (g * n).abs().mean(dim=1, keepdim=True) * k
    inner = eg + e0 + n.abs() * e1 + c1.abs() * en + 3 * U * (g.abs() + c0.abs() + (n * c1).abs())
    edx = r * inner * k + U * dx.abs()
    # many rows: a team's in order, 8 teams, 8 partials of a slice, 32 slices; up to 1024
    # rows: a 64th in order, 16 lanes, four sixteens
    depth = max(M // 256 + 1 + 8 + 8 + 32, min(M, 1024) // 64 + 1 + 16 + 4)
    t = dy * n
    edw = ((depth + 3) * U * t.abs()).sum(dim=0) * k
    edb = (depth * U * dy.abs()).sum(dim=0)
    return dx, t.sum(dim=0), dy.sum(dim=0), stored(edx, dx, x_dtype), edw + 1e-37, edb + 1e-37


def spans(ends, T):
    """Expert by expert first and last + 1 row: a running maximum, held to 0 .. T."""
    out, at = [], 0
    for v in ends:
        to = max(at, min(max(int(v), 0), T))
        out.append((at, to))
        at = to
    return out


def codes(x):
    """Codes and fp32 scales of the rows of x by the definition, in binary64."""
    x = x.double().cpu()
    bad = ~torch.isfinite(x).all(dim=1)
    top = torch.where(bad, torch.zeros(x.shape[0], dtype=torch.float64), x.abs().amax(dim=1))
    s = torch.clamp(top.float() * torch.tensor(1.0 / 127.0), min=2.0 ** -126)        # fp32's 1/127, one rounding
    q = torch.round(torch.where(bad[:, None], torch.zeros_like(x), x) / s.double()[:, None])      # torch.round: ties to even
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    return q.to(torch.int8), s


def linear_int8(xq, xs, wq, ws, bias, out_dtype):
    """The kernel's own sequence: the integer sum, then fp32 steps in order, all of
    them exactly as IEEE rounds them."""
    acc = torch.mm(xq.double().cpu(), wq.double().cpu().t().contiguous())       # below 2^53: exact
    v = acc.float() * xs.float().cpu()[:, None] * ws.float().cpu()
    if bias is not None:
        v = v + bias.cpu()
    return v.to(out_dtype)
