"""The feed-forward operators, case by case: the gated linear layer with its
backward pass, the backward pass of the plain linear layer, and 4-bit
microscaled (MXFP4) quantisation with the product of quantised operands.

A case is a dict of plain values.  ``prepare`` makes what a caller holds before
the call, ``run`` makes one pass -- the operators' plain form in elementary
torch operations, or, where ``own`` is true, the package's kernels -- and
``exact`` says what the outputs are in 64 bits.

Definitions (all rows are independent; R rounds to the stored type once):

gated         h = x W13^T (gate half, then up half);  y = R(act(h_g) * h_u)
              act = silu, or gelu in its tanh form; h is also stored, rounded
              to bf16, where a backward pass will follow
gated_bwd     dh = [dy * h_u * act'(h_g), dy * act(h_g)] of the stored h;
              dx = R(dh W13),  dw = R(dh^T x)
linear_bwd    dx = R(dy W),  dw = R(dy^T x),  db = sum of dy over the rows
quantize      blocks of 32 along a row share the power of two
              2^(floor(log2 max|x|) - 2); elements are x / scale rounded to the
              nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to even, saturating)
linear_mxfp4  y = R(X W^T + b) of the values that codes and scales stand for
"""
import math

import torch

own = False

SILU, GELU = "silu", "gelu_tanh"
_C = math.sqrt(2.0 / math.pi)


# ------------------------------------------------------------------- the cases


def listed():
    return [
        # one token through a small layer (an expert-sized block): pure latency
        dict(name="gated_m1_small", op="gated", M=1, H=2048, I=768, act=SILU, save=False),
        # a decode batch through a large layer: the weight is read once
        dict(name="gated_m16", op="gated", M=16, H=4096, I=12288, act=SILU, save=False),
        # a training micro-batch of ragged length, pre-activations kept
        dict(name="gated_m1000_train", op="gated", M=1000, H=4096, I=6144, act=GELU, save=True),
        # a long prompt through a large layer
        dict(name="gated_m4096", op="gated", M=4096, H=4096, I=12288, act=SILU, save=False),
        # the backward pass of a short batch through the small layer
        dict(name="gated_bwd_m200", op="gated_bwd", M=200, H=2048, I=768, act=GELU),
        # the backward pass of a full training micro-batch
        dict(name="gated_bwd_m4096", op="gated_bwd", M=4096, H=4096, I=12288, act=SILU),
        # a down projection's gradients, ragged batch, fp32 weight gradient
        dict(name="linear_bwd_m333", op="linear_bwd", M=333, N=2048, K=768, dw="float32"),
        # a square projection's gradients at a full micro-batch
        dict(name="linear_bwd_m4096", op="linear_bwd", M=4096, N=4096, K=4096, dw="bfloat16"),
        # activations of a decode batch, quantised in front of a product
        dict(name="quantize_m16", op="quantize", M=16, K=4096, x="bfloat16"),
        # a weight, quantised when a checkpoint is loaded
        dict(name="quantize_weight", op="quantize", M=12288, K=4096, x="bfloat16"),
        # one token through a 4-bit projection
        dict(name="mxfp4_m1", op="linear_mxfp4", M=1, N=4096, K=4096, bias=True, y="bfloat16"),
        # a long prompt through a large 4-bit projection
        dict(name="mxfp4_m4096", op="linear_mxfp4", M=4096, N=12288, K=4096, bias=False, y="bfloat16"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("gated", "gated_bwd", "linear_bwd", "quantize", "linear_mxfp4"))
    M = _log(rng, 1, 4096)
    if op in ("gated", "gated_bwd"):
        c = dict(op=op, M=M, H=_log(rng, 256, 4096, 32), I=_log(rng, 128, 12288, 16), act=rng.choice((SILU, GELU)))
        return dict(c, save=rng.random() < 0.5) if op == "gated" else c
    if op == "linear_bwd":
        return dict(op=op, M=M, N=_log(rng, 128, 8192, 16), K=_log(rng, 256, 4096, 32),
                    dw=rng.choice(("float32", "bfloat16")))
    if op == "quantize":
        return dict(op=op, M=_log(rng, 1, 12288), K=_log(rng, 256, 4096, 32), x=rng.choice(("float32", "bfloat16")))
    return dict(op=op, M=M, N=_log(rng, 128, 12288, 16), K=_log(rng, 256, 4096, 32), bias=rng.random() < 0.5,
                y=rng.choice(("float32", "bfloat16")))


# ---------------------------------------------------------- inputs and the work


def _randn(gen, shape, std, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    b16 = torch.bfloat16
    st = {"case": dict(case)}
    op, M = case["op"], case["M"]
    if op in ("gated", "gated_bwd"):
        H, I = case["H"], case["I"]
        st["x"] = _randn(gen, (M, H), 1.0, b16)                       # activations behind a norm
        st["w13"] = _randn(gen, (2 * I, H), 1.0 / math.sqrt(H), b16)  # nn.Linear weight
        if op == "gated_bwd":
            st["dy"] = _randn(gen, (M, I), 1e-2, b16)
            st["h"] = _randn(gen, (M, 2 * I), 1.0, b16)               # pre-activations that the forward pass kept
    elif op == "linear_bwd":
        N, K = case["N"], case["K"]
        st["dy"] = _randn(gen, (M, N), 1e-2, b16)
        st["x"] = _randn(gen, (M, K), 1.0, b16)
        st["w"] = _randn(gen, (N, K), 1.0 / math.sqrt(K), b16)
    elif op == "quantize":
        # channels of unlike size, as activations and weights have
        size = torch.exp(torch.randn((1, case["K"]), generator=gen, device="cuda"))
        st["x"] = (_randn(gen, (M, case["K"]), 1.0, torch.float32) * size).to(getattr(torch, case["x"]))
    else:
        N, K = case["N"], case["K"]
        for name, rows, std in (("x", M, 1.0), ("w", N, 1.0 / math.sqrt(K))):
            e, m = _mx_split(_randn(gen, (rows, K), std, torch.float32))
            code = _mx_code(m)
            st[name + "q"] = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
            # scales in rows of a whole number of 32-bit words, as the kernels read them
            kb = K // 32
            st[name + "s"] = torch.zeros((rows, (kb + 3) // 4 * 4), dtype=torch.uint8, device="cuda")[:, :kb]
            st[name + "s"].copy_(e)
        st["bias"] = _randn(gen, (N,), 0.1, torch.float32) if case["bias"] else None
    return st


def work(case):
    op, M = case["op"], case["M"]
    if op == "gated":
        H, I = case["H"], case["I"]
        return {"bytes": 2 * (M * H + 2 * I * H + M * I + (2 * M * I if case["save"] else 0)), "flops": 4 * M * H * I}
    if op == "gated_bwd":
        H, I = case["H"], case["I"]
        return {"bytes": 2 * (M * I + 2 * M * I + 2 * M * H + 4 * I * H), "flops": 8 * M * H * I}
    if op == "linear_bwd":
        N, K = case["N"], case["K"]
        dw = 4 if case["dw"] == "float32" else 2
        return {"bytes": 2 * (M * N + 2 * M * K + N * K) + dw * N * K + 4 * N, "flops": 4 * M * N * K}
    if op == "quantize":
        # quantised, and read back to bf16: the codes and scales are written and read
        K = case["K"]
        coded = M * K // 2 + M * K // 32
        return {"bytes": M * K * (4 if case["x"] == "float32" else 2) + 2 * coded + 2 * M * K, "flops": 4 * M * K}
    N, K = case["N"], case["K"]
    y = 4 if case["y"] == "float32" else 2
    return {"bytes": (M + N) * (K // 2 + K // 32) + y * M * N + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}


# --------------------------------------------------------------- the plain form


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _act(g, act):
    """act(g) and its derivative."""
    if act == SILU:
        s = _sigmoid(g)
        return g * s, s * (1.0 + g * (1.0 - s))
    s = _sigmoid(2.0 * _C * (g + 0.044715 * g * g * g))      # 0.5 (1 + tanh(z)) = sigmoid(2 z)
    return g * s, s + g * s * (1.0 - s) * (2.0 * _C) * (1.0 + 3 * 0.044715 * g * g)


def _mx_split(x):
    """Rows of fp32 in blocks of 32: the scale byte of each block and the
    elements over their scale."""
    M, K = x.shape
    b = x.reshape(M, K // 32, 32)
    top = (b.abs().amax(dim=2).view(torch.int32) >> 23) & 0xff          # exponent byte of the largest
    e = (top - 2).clamp(min=0)
    half = -(e - 127)                                                   # 2^-(e - 127), in two exact factors
    lo = half // 2
    m = b * torch.ldexp(torch.ones_like(lo, dtype=torch.float32), lo)[:, :, None]
    m = m * torch.ldexp(torch.ones_like(lo, dtype=torch.float32), half - lo)[:, :, None]
    return e.to(torch.uint8), m.reshape(M, K)


def _mx_code(m):
    """The 4-bit code (sign, 0..7) nearest to each value, ties to the even code."""
    a = m.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    # halfway points between neighbouring values; a tie goes up where the upper code is even
    for at, up_on_tie in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += ((a >= at) if up_on_tie else (a > at)).to(torch.uint8)
    return code | (torch.signbit(m).to(torch.uint8) << 3)


_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_tables = {}


def _table(device):
    if device not in _tables:
        _tables[device] = torch.tensor(_VALUES + tuple(-v for v in _VALUES), dtype=torch.float32, device=device)
    return _tables[device]


def _mx_values(code, e):
    """fp32 values of unpacked codes [M, K] under the scale bytes [M, K/32]."""
    M, K = code.shape
    v = _table(code.device)[code.to(torch.int64)].reshape(M, K // 32, 32)
    p = (e.to(torch.int32) - 127)
    lo = p // 2
    one = torch.ones_like(lo, dtype=torch.float32)
    return (v * torch.ldexp(one, lo)[:, :, None] * torch.ldexp(one, p - lo)[:, :, None]).reshape(M, K)


def _mx_unpack(q):
    return torch.stack((q & 15, q >> 4), dim=2).reshape(q.shape[0], -1)


def _plain(st):
    c = st["case"]
    op, b16 = c["op"], torch.bfloat16
    if op == "gated":
        h = torch.mm(st["x"].float(), st["w13"].float().t())
        y = (_act(h[:, :c["I"]], c["act"])[0] * h[:, c["I"]:]).to(b16)
        return {"y": y, "h": h.to(b16)} if c["save"] else {"y": y}
    if op == "gated_bwd":
        g, u, dy = st["h"][:, :c["I"]].float(), st["h"][:, c["I"]:].float(), st["dy"].float()
        a, da = _act(g, c["act"])
        dh = torch.cat((dy * u * da, dy * a), dim=1)
        return {"dx": torch.mm(dh, st["w13"].float()).to(b16), "dw": torch.mm(dh.t(), st["x"].float()).to(b16)}
    if op == "linear_bwd":
        dy = st["dy"].float()
        return {"dx": torch.mm(dy, st["w"].float()).to(b16),
                "dw": torch.mm(dy.t(), st["x"].float()).to(getattr(torch, c["dw"])), "db": dy.sum(dim=0)}
    if op == "quantize":
        e, m = _mx_split(st["x"].float())
        return {"values": _mx_values(_mx_code(m), e).to(b16), "scale": e}
    y = torch.mm(_mx_values(_mx_unpack(st["xq"]), st["xs"]), _mx_values(_mx_unpack(st["wq"]), st["ws"]).t())
    if st["bias"] is not None:
        y = y + st["bias"]
    return {"y": y.to(getattr(torch, c["y"]))}


# ------------------------------------------------------------ the package's calls


def _own(st):
    import deterministic_persistent_gemm_amd as bi

    c = st["case"]
    op = c["op"]
    if op in ("gated", "gated_bwd"):
        gate = bi.BI_GATE_SILU if c["act"] == SILU else bi.BI_GATE_GELU_TANH
    if op == "gated":
        if c["save"]:
            y, h = bi.bi_gated_linear_bf16(st["x"], st["w13"].t(), gate, save_h=True)
            return {"y": y, "h": h}
        return {"y": bi.bi_gated_linear_bf16(st["x"], st["w13"].t(), gate)}
    if op == "gated_bwd":
        dx, dw = bi.bi_gated_linear_bf16_bwd(st["dy"], st["x"], st["w13"].t(), st["h"], gate)
        return {"dx": dx, "dw": dw}
    if op == "linear_bwd":
        dx, dw, db = bi.bi_linear_bf16_bwd(st["dy"], st["x"], st["w"].t(), dw_dtype=getattr(torch, c["dw"]))
        return {"dx": dx, "dw": dw, "db": db}
    if op == "quantize":
        q, s = bi.bi_quantize_mxfp4(st["x"])
        return {"values": bi.bi_dequantize_mxfp4(q, s), "scale": s}
    return {"y": bi.bi_linear_mxfp4(st["xq"], st["xs"], st["wq"], st["ws"], st["bias"],
                                    out_dtype=getattr(torch, c["y"]))}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64-bit values


def _exact_act(g, act):
    """act and act' from their textbook forms in binary64."""
    if act == SILU:
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    t = torch.tanh(_C * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * _C * (1 + 3 * 0.044715 * g * g)


def _exact_values(q, e):
    """Values of packed codes by the format's fields: sign, two exponent bits
    (bias 1), one mantissa bit."""
    n = torch.empty((q.shape[0], q.shape[1] * 2), dtype=torch.int32, device=q.device)
    n[:, 0::2] = q.to(torch.int32) % 16
    n[:, 1::2] = q.to(torch.int32) // 16
    ex, ma = (n // 2) % 4, (n % 2).double()
    v = torch.where(ex == 0, 0.5 * ma, (1 + 0.5 * ma) * torch.exp2((ex - 1).double()))
    v = torch.where(n >= 8, -v, v)
    return v * torch.exp2(e.double() - 127).repeat_interleave(32, dim=1)


def _exact_quantized(x):
    """The nearest representable value by comparing distances, block by block."""
    M, K = x.shape
    b = x.double().reshape(M, K // 32, 32)
    top = torch.frexp(b.abs().amax(dim=2)).exponent - 1                  # floor(log2 max)
    e = torch.where(b.abs().amax(dim=2) == 0, torch.full_like(top, -127), (top - 2).clamp(min=-127))
    scale = torch.exp2(e.double())[:, :, None]
    a = b.abs() / scale
    best = torch.zeros_like(a)
    for k in (2, 4, 6, 1, 3, 5, 7):                                      # even codes first: they keep ties
        v = torch.full_like(a, _VALUES[k])
        best = torch.where((v - a).abs() < (best - a).abs(), v, best)
    return (torch.sign(b) * best * scale).reshape(M, K)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "gated":
        h = torch.mm(st["x"].double(), st["w13"].double().t())
        y = _exact_act(h[:, :case["I"]], case["act"])[0] * h[:, case["I"]:]
        return {"y": y, "h": h} if case["save"] else {"y": y}
    if op == "gated_bwd":
        g, u, dy = st["h"].double()[:, :case["I"]], st["h"].double()[:, case["I"]:], st["dy"].double()
        a, da = _exact_act(g, case["act"])
        dh = torch.cat((dy * u * da, dy * a), dim=1)
        return {"dx": torch.mm(dh, st["w13"].double()), "dw": torch.mm(dh.t().contiguous(), st["x"].double())}
    if op == "linear_bwd":
        dy = st["dy"].double()
        return {"dx": torch.mm(dy, st["w"].double()), "dw": torch.mm(dy.t().contiguous(), st["x"].double()),
                "db": dy.sum(dim=0)}
    if op == "quantize":
        return {"values": _exact_quantized(st["x"]), "scale": None}
    y = torch.mm(_exact_values(st["xq"], st["xs"]), _exact_values(st["wq"], st["ws"]).t())
    return {"y": y if st["bias"] is None else y + st["bias"].double()}
