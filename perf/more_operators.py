"""The operators of an expert block, case by case: layer norm with its backward
pass, products grouped by expert with theirs, and products of 8-bit integers
with a scale for each token and channel, plain and grouped.

A case is a dict of plain values.  ``prepare`` makes what a caller holds before
the call, ``run`` makes one pass -- the operators' plain form in elementary
torch operations, or, where ``own`` is true, the package's kernels -- and
``exact`` says what the outputs are in 64 bits.

Definitions (R rounds to the stored type once):

norm          m = mean(x), v = mean((x - m)^2), r = 1 / sqrt(v + eps) of a row;
              y = R((x - m) r w + b); m and r are stored in fp32 where a
              backward pass will follow
norm_bwd      with the stored m and r, n = (x - m) r and g = dy w:
              dx = R(r (g - mean(g) - n mean(g n))), dw = sum of dy n and
              db = sum of dy over the rows
grouped       rows ends[e-1] .. ends[e] - 1 of x belong to expert e (ends[-1]
              = 0): y = R(x W[e]^T) there; rows behind the last expert's are
              left as they are
grouped_bwd   dx = R(dy W[e]) and dw[e] = R(dy^T x) over the expert's rows
              (zero for an expert without rows)
int8          a row's scale is s = max(max|x| / 127, 2^-126) in fp32 and its codes
              x / s rounded to the nearest integer (ties to even);
              y = R(sum of code products * s_x[m] * s_w[n] + b[n])
grouped_int8  the same with the weight of each row's expert
"""
import math

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------- the cases


def listed():
    moe = dict(E=128, N=1536, K=2048)             # gate and up rows of an expert of 768, 8 of 128 a token
    return [
        # one token in front of its layer: pure latency
        dict(name="norm_m1", op="norm", M=1, H=4096, x="bfloat16", y="bfloat16", save=False),
        # a training batch from an fp32 residual stream, statistics kept
        dict(name="norm_m8192_train", op="norm", M=8192, H=4096, x="float32", y="bfloat16", save=True),
        # the backward pass of a short ragged batch
        dict(name="norm_bwd_m333", op="norm_bwd", M=333, H=2048, x="float32", y="bfloat16"),
        # the backward pass of a full training batch
        dict(name="norm_bwd_m8192", op="norm_bwd", M=8192, H=4096, x="bfloat16", y="bfloat16"),
        # one token's experts: eight weights of a row each
        dict(name="grouped_1token", op="grouped", tokens=1, topk=8, pad=0, skew=0.0, y="bfloat16", **moe),
        # a long prompt, some experts much more in demand than others
        dict(name="grouped_4096tokens", op="grouped", tokens=4096, topk=8, pad=0, skew=0.7, y="bfloat16", **moe),
        # a ragged micro-batch through few experts, fp32 weight gradients
        dict(name="grouped_bwd_333tokens", op="grouped_bwd", tokens=333, topk=2, skew=1.0, E=16, N=2048, K=768, dw="float32"),
        # a full training batch
        dict(name="grouped_bwd_4096tokens", op="grouped_bwd", tokens=4096, topk=8, skew=0.7, dw="bfloat16", **moe),
        # a decode batch through an 8-bit projection
        dict(name="int8_m16", op="int8", M=16, N=4096, K=4096, x="bfloat16", bias=True, y="bfloat16"),
        # a long prompt through a large 8-bit projection
        dict(name="int8_m4096", op="int8", M=4096, N=12288, K=4096, x="bfloat16", bias=False, y="bfloat16"),
        # a decode batch through 8-bit experts, padded to the rows its graph was captured with
        dict(name="grouped_int8_8tokens", op="grouped_int8", tokens=8, topk=8, pad=64, skew=0.0, y="bfloat16", **moe),
        # a prompt through 8-bit experts
        dict(name="grouped_int8_2000tokens", op="grouped_int8", tokens=2000, topk=8, pad=0, skew=0.7, y="bfloat16", **moe),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "grouped", "grouped_bwd", "int8", "grouped_int8"))
    f = lambda: rng.choice(("float32", "bfloat16"))
    if op in ("norm", "norm_bwd"):
        c = dict(op=op, M=_log(rng, 1, 8192), H=_log(rng, 256, 8192, 8), x=f(), y=f())
        return dict(c, save=rng.random() < 0.5) if op == "norm" else c
    if op == "int8":
        return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 128, 12288, 16), K=_log(rng, 256, 4096, 32), x=f(),
                    bias=rng.random() < 0.5, y=f())
    E = _log(rng, 2, 128)
    c = dict(op=op, tokens=_log(rng, 1, 2048), topk=rng.randint(1, min(8, E)), skew=rng.choice((0.0, 0.7, 1.5)), E=E,
             N=_log(rng, 128, 2048, 16), K=_log(rng, 256, 2048, 32))
    if op == "grouped_bwd":
        return dict(c, dw=f())
    return dict(c, pad=rng.choice((0, rng.randint(1, 100))), y=f())


# ---------------------------------------------------------- inputs and the work


def _randn(gen, shape, std, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _route(case, seed):
    """Rows of each expert: every token takes topk experts, popular ones more often."""
    gen = torch.Generator()
    gen.manual_seed(seed)
    want = torch.randn((1, case["E"]), generator=gen) * case["skew"]
    u = torch.rand((case["tokens"], case["E"]), generator=gen).clamp_(min=1e-20)
    ids = (want - torch.log(-torch.log(u))).topk(case["topk"], dim=1).indices
    return torch.bincount(ids.flatten(), minlength=case["E"])


def _codes(x):
    """Rows as 8-bit codes and fp32 scales."""
    s = (x.float().abs().amax(dim=-1) / 127.0).clamp(min=2.0 ** -126)
    return torch.round(x.double() / s.double()[..., None]).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    b16 = torch.bfloat16
    st = {"case": dict(case)}
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        M, H = case["M"], case["H"]
        # a residual stream: channels of unlike size, rows off zero
        size = torch.exp(0.5 * torch.randn((1, H), generator=gen, device="cuda"))
        x = _randn(gen, (M, H), 1.0, torch.float32) * size + _randn(gen, (M, 1), 0.3, torch.float32)
        st["x"] = x.to(getattr(torch, case["x"]))
        st["w"] = 1.0 + _randn(gen, (H,), 0.1, torch.float32)
        st["b"] = _randn(gen, (H,), 0.1, torch.float32)
        if op == "norm_bwd":
            st["dy"] = _randn(gen, (M, H), 1e-2, getattr(torch, case["y"]))
            d = st["x"].double()
            st["mean"] = d.mean(dim=1).float()
            st["rstd"] = (1.0 / torch.sqrt(d.var(dim=1, unbiased=False) + EPS)).float()
        return st
    if op == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        size = torch.exp(0.5 * torch.randn((1, K), generator=gen, device="cuda"))
        st["x"] = (_randn(gen, (M, K), 1.0, torch.float32) * size).to(getattr(torch, case["x"]))
        st["wq"], st["ws"] = _codes(_randn(gen, (N, K), 1.0 / math.sqrt(K), torch.float32))
        st["bias"] = _randn(gen, (N,), 0.1, torch.float32) if case["bias"] else None
        return st
    E, N, K = case["E"], case["N"], case["K"]
    count = _route(case, seed)
    st["rows"] = count.tolist()                                       # the plain form's loop over experts
    st["ends"] = torch.cumsum(count, 0).cuda()
    T = sum(st["rows"]) + case.get("pad", 0)
    st["x"] = _randn(gen, (T, K), 1.0, b16)                           # sorted by expert
    if op == "grouped_int8":
        st["wq"] = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
        st["ws"] = torch.empty((E, N), dtype=torch.float32, device="cuda")
        for e in range(E):
            st["wq"][e], st["ws"][e] = _codes(_randn(gen, (N, K), 1.0 / math.sqrt(K), torch.float32))
    else:
        st["w"] = _randn(gen, (E, N, K), 1.0 / math.sqrt(K), b16)
    if op == "grouped_bwd":
        st["dy"] = _randn(gen, (T, N), 1e-2, b16)
    else:
        # the caller's buffer: rows behind the last expert's stay what they are
        st["y"] = torch.zeros((T, N), dtype=getattr(torch, case["y"]), device="cuda")
    return st


def _size(name):
    return 4 if name == "float32" else 2


def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        M, H = case["M"], case["H"]
        x, y = _size(case["x"]), _size(case["y"])
        if op == "norm":
            return {"bytes": M * H * (x + y) + 8 * H + (8 * M if case["save"] else 0), "flops": 8 * M * H}
        return {"bytes": M * H * (2 * x + y) + 8 * M + 12 * H, "flops": 16 * M * H}
    if op == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * _size(case["x"]) + N * K + 4 * N + M * N * _size(case["y"]) + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    T, E, N, K = case["tokens"] * case["topk"], case["E"], case["N"], case["K"]
    active = round(E * (1.0 - (1.0 - case["topk"] / E) ** case["tokens"]))      # experts with rows, were all alike
    if op == "grouped_bwd":
        return {"bytes": 2 * T * (N + 2 * K) + 2 * active * N * K + E * N * K * _size(case["dw"]), "flops": 4 * T * N * K}
    w = 1 if op == "grouped_int8" else 2
    return {"bytes": 2 * T * K + w * active * N * K + T * N * _size(case["y"]), "flops": 2 * T * N * K}


# --------------------------------------------------------------- the plain form


def _groups(st):
    at = 0
    for e, n in enumerate(st["rows"]):
        yield e, at, at + n
        at += n


def _plain(st):
    c = st["case"]
    op, b16 = c["op"], torch.bfloat16
    if op == "norm":
        x = st["x"].float()
        m = x.mean(dim=1, keepdim=True)
        d = x - m
        r = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + EPS)
        y = (d * r * st["w"] + st["b"]).to(getattr(torch, c["y"]))
        return {"y": y, "mean": m[:, 0], "rstd": r[:, 0]} if c["save"] else {"y": y}
    if op == "norm_bwd":
        dy, r = st["dy"].float(), st["rstd"][:, None]
        n = (st["x"].float() - st["mean"][:, None]) * r
        g = dy * st["w"]
        dx = r * (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True))
        return {"dx": dx.to(st["x"].dtype), "dw": (dy * n).sum(dim=0), "db": dy.sum(dim=0)}
    if op == "int8":
        q, s = _codes(st["x"])
        y = torch.mm(q.float(), st["wq"].float().t()) * s[:, None] * st["ws"]
        if st["bias"] is not None:
            y = y + st["bias"]
        return {"y": y.to(getattr(torch, c["y"]))}
    if op == "grouped":
        y, x = st["y"], st["x"].float()
        for e, a, b in _groups(st):
            if b > a:
                y[a:b] = torch.mm(x[a:b], st["w"][e].float().t()).to(y.dtype)
        return {"y": y}
    if op == "grouped_int8":
        y = st["y"]
        q, s = _codes(st["x"])
        q = q.float()
        for e, a, b in _groups(st):
            if b > a:
                y[a:b] = (torch.mm(q[a:b], st["wq"][e].float().t()) * s[a:b, None] * st["ws"][e]).to(y.dtype)
        return {"y": y}
    dy, x = st["dy"].float(), st["x"].float()
    dx = torch.empty_like(st["x"])
    dw = torch.empty(st["w"].shape, dtype=getattr(torch, c["dw"]), device="cuda")
    for e, a, b in _groups(st):
        if b > a:
            dx[a:b] = torch.mm(dy[a:b], st["w"][e].float()).to(b16)
        dw[e] = torch.mm(dy[a:b].t(), x[a:b]).to(dw.dtype)
    return {"dx": dx, "dw": dw}


# ------------------------------------------------------------ the package's calls


def _own(st):
    import deterministic_persistent_gemm_amd as bi

    c = st["case"]
    op = c["op"]
    if op == "norm":
        r = bi.bi_layer_norm(st["x"], st["w"], st["b"], EPS, out_dtype=getattr(torch, c["y"]), save_stats=c["save"])
        return dict(zip(("y", "mean", "rstd"), r)) if c["save"] else {"y": r}
    if op == "norm_bwd":
        dx, dw, db = bi.bi_layer_norm_bwd(st["dy"], st["x"], st["mean"], st["rstd"], st["w"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "int8":
        xq, xs = bi.bi_quantize_int8(st["x"])
        return {"y": bi.bi_linear_int8(xq, xs, st["wq"], st["ws"], st["bias"], out_dtype=getattr(torch, c["y"]))}
    if op == "grouped":
        return {"y": bi.bi_grouped_linear_bf16(st["x"], st["w"], st["ends"], out=st["y"])}
    if op == "grouped_int8":
        xq, xs = bi.bi_quantize_int8(st["x"])
        return {"y": bi.bi_grouped_linear_int8(xq, xs, st["wq"], st["ws"], st["ends"], out=st["y"])}
    dx, dw = bi.bi_grouped_linear_bf16_bwd(st["dy"], st["x"], st["w"], st["ends"], dw_dtype=getattr(torch, c["dw"]))
    return {"dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64-bit values


def _exact_codes(x):
    """The codes' values and the scales by the definition: the nearest integer by
    its distance, the even one where two are as near."""
    top = x.double().abs().amax(dim=1)
    s = torch.where(top / 127.0 < 2.0 ** -126, torch.full_like(top, 2.0 ** -126), (top / 127.0).float().double())
    v = x.double() / s[:, None]
    low = torch.floor(v)
    up = (v - low > 0.5) | ((v - low == 0.5) & (torch.remainder(low, 2.0) == 1.0))
    return low + up.double(), s


def _span(ends, e):
    return (0 if e == 0 else int(ends[e - 1])), int(ends[e])


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = st["x"].double()
        m = x.sum(dim=1) / case["H"]
        var = ((x - m[:, None]) ** 2).sum(dim=1) / case["H"]
        r = (var + EPS) ** -0.5
        y = (x - m[:, None]) * r[:, None] * st["w"].double() + st["b"].double()
        return {"y": y, "mean": m, "rstd": r} if case["save"] else {"y": y}
    if op == "norm_bwd":
        # the Jacobian of the normalised row, (I - 1 1^T / H - n n^T / H) r, applied to dy w
        dy, r = st["dy"].double(), st["rstd"].double()[:, None]
        n = (st["x"].double() - st["mean"].double()[:, None]) * r
        g, H = dy * st["w"].double(), case["H"]
        dx = r * g - r / H * g.sum(dim=1, keepdim=True) - r / H * n * (g * n).sum(dim=1, keepdim=True)
        return {"dx": dx, "dw": torch.einsum("mh,mh->h", dy, n), "db": torch.einsum("mh->h", dy)}
    if op == "int8":
        q, s = _exact_codes(st["x"])
        y = torch.mm(q, st["wq"].double().t()) * (s[:, None] * st["ws"].double()[None, :])
        return {"y": y if st["bias"] is None else y + st["bias"].double()}
    ends = st["ends"].tolist()
    if op in ("grouped", "grouped_int8"):
        y = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
        if op == "grouped_int8":
            q, s = _exact_codes(st["x"])
        for e in range(case["E"]):
            a, b = _span(ends, e)
            if a == b:
                continue
            if op == "grouped":
                y[a:b] = torch.mm(st["x"][a:b].double(), st["w"][e].double().t())
            else:
                y[a:b] = torch.mm(q[a:b], st["wq"][e].double().t()) * (s[a:b, None] * st["ws"][e].double()[None, :])
        return {"y": y}
    dx = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(st["w"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        a, b = _span(ends, e)
        if a < b:
            d, x = st["dy"][a:b].double(), st["x"][a:b].double()
            dx[a:b] = torch.mm(d, st["w"][e].double())
            dw[e] = torch.mm(d.t().contiguous(), x)
    return {"dx": dx, "dw": dw}
