"""Measured cases of the MLP block's operators: LayerNorm forward and backward, the activation's cast-transpose
forward and backward, and the FP8 GEMM with bias, activation and residual.

`run` computes a case in plain torch (32-bit elementary operations, one rounding at the end) where `own` is false, and
through the framework's entry points where it is true.  `exact` is the definition in 64 bits.
"""

import torch

own = False

DEV = "cuda"
EPS = 1e-5
HP = {"f32": torch.float32, "bf16": torch.bfloat16}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}

OPS = ("layernorm", "layernorm_backward", "act", "act_backward", "gemm_residual")


# ------------------------------------------------------------------ cases


def listed():
    return [
        # a decoding step's norm: one token of the small model's width, all latency
        dict(name="ln-token", op="layernorm", rows=1, cols=768, dtype="bf16", out="bf16"),
        # the norm before a large FC1, the residual stream in bf16
        dict(name="ln-large", op="layernorm", rows=8192, cols=4096, dtype="bf16", out="bf16"),
        # its backward at the small model's size
        dict(name="lnb-small", op="layernorm_backward", rows=2048, cols=768, dtype="bf16", dy="bf16", dres=False),
        # an odd width and an odd number of rows, the stream and its gradient in fp32
        dict(name="lnb-odd-f32", op="layernorm_backward", rows=1537, cols=1251, dtype="f32", dy="f32", dres=True),
        # the large block's norm, with the residual branch's gradient joined in the same pass
        dict(name="lnb-large", op="layernorm_backward", rows=8192, cols=4096, dtype="bf16", dy="bf16", dres=True),
        # a wide blockwise FC1's GELU output, both copies for FC2 and its wgrad
        dict(name="act-gelu-tile", op="act", rows=4096, cols=7168, act="gelu", fmt="e4m3", gran="tile", dtype="bf16"),
        # the large SwiGLU FC1: gate and up interleaved, delayed scale
        dict(name="act-swiglu-large", op="act", rows=8192, cols=14336, act="swiglu", fmt="e4m3", gran="tensor",
             dtype="bf16"),
        # a ragged batch through a GELU layer's backward
        dict(name="actb-gelu-ragged", op="act_backward", rows=1531, cols=2310, act="gelu", fmt="e5m2", gran="tensor",
             dtype="bf16"),
        # blockwise recipe's SwiGLU backward
        dict(name="actb-swiglu-tile", op="act_backward", rows=4096, cols=7168, act="swiglu", fmt="e4m3", gran="tile",
             dtype="bf16"),
        # hybrid recipe's SwiGLU backward at the large FC1's size, with its bias gradient
        dict(name="actb-swiglu-large", op="act_backward", rows=8192, cols=14336, act="swiglu", fmt="e5m2",
             gran="tensor", dtype="bf16"),
        # one decoding step of a few sequences through the large down projection
        dict(name="gemm-tokens", op="gemm_residual", m=4, n=4096, k=7168, mode="tensor", fmt="e4m3", act="none",
             bias=True, dtype="bf16"),
        # the large down projection onto the residual stream
        dict(name="gemm-large", op="gemm_residual", m=8192, n=4096, k=7168, mode="tensor", fmt="e4m3", act="none",
             bias=True, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("layernorm", "layernorm_backward"):
        rows, cols = _spread(rng, 1, 8192), _spread(rng, 64, 8192)
        if rng.random() < 0.6:
            cols = max(64, cols // 8 * 8)
        rows = min(rows, (1 << 25) // cols)
        if op == "layernorm":
            return dict(op=op, rows=rows, cols=cols, dtype=dtype, out=rng.choice(("bf16", dtype)))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, dy=rng.choice(("bf16", dtype)), dres=rng.random() < 0.5)
    if op in ("act", "act_backward"):
        rows, cols = _spread(rng, 1, 8192), _spread(rng, 64, 14336)
        gran, act = rng.choice(("tensor", "tile")), rng.choice(("gelu", "swiglu"))
        if op == "act_backward" and rng.random() < 0.25:
            act = "none"
        if gran == "tile":
            unit = 256 if act == "swiglu" else 128
            rows, cols = -(-rows // 128) * 128, max(unit, cols // unit * unit)
        else:
            cols = cols // 2 * 2 if act == "swiglu" or rng.random() < 0.7 else cols
        return dict(op=op, rows=rows, cols=cols, act=act, fmt=rng.choice(("e4m3", "e5m2")), gran=gran, dtype=dtype)
    m, n, k = _spread(rng, 1, 8192), _spread(rng, 64, 14336), 128 * _spread(rng, 1, 56)
    mode, act = rng.choice(("tensor", "block", "mx")), rng.choice(("none", "none", "gelu", "swiglu"))
    n = min(n, (1 << 25) // m) // 4 * 4
    return dict(op=op, m=m, n=n, k=k, mode=mode, fmt=rng.choice(("e4m3", "e4m3", "e5m2")), act=act,
                bias=rng.random() < 0.7, dtype="bf16")


def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}
    if op == "gemm_residual":
        m, n, k = case["m"], case["n"], case["k"]
        out = n // 2 if case["act"] == "swiglu" else n
        return {"bytes": (m + n) * k + 2 * out * m * size[case["dtype"]], "flops": 2.0 * m * n * k}
    r, c = case["rows"], case["cols"]
    e = r * c
    x = size[case["dtype"]]
    if op == "layernorm":
        return {"bytes": e * (x + size[case["out"]]) + 8 * r + 8 * c, "flops": 8.0 * e}
    if op == "layernorm_backward":
        return {"bytes": e * (2 * x + size[case["dy"]] + (x if case["dres"] else 0)) + 8 * r + 12 * c,
                "flops": 14.0 * e}
    if op == "act":
        outs = e // 2 if case["act"] == "swiglu" else e
        scales = outs // 16 if case["gran"] == "tile" else 0
        return {"bytes": e * x + 2 * outs + scales, "flops": 20.0 * outs}
    dys = e // 2 if case["act"] == "swiglu" else e
    scales = e // 16 if case["gran"] == "tile" else 0
    return {"bytes": dys * x + (0 if case["act"] == "none" else e * x) + 2 * e + 4 * c + scales, "flops": 20.0 * e}


# ------------------------------------------------------------------ inputs


def _normal(g, shape, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def _codes(v, fmt):
    """fp32 -> FP8, saturating at the format's largest value, as uint8."""
    return v.clamp(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)


def _operand(g, rows, k, std, gran, fmt):
    """Quantised N(0, std) [rows][k]: (codes, scale_inv) in the layouts of the framework's quantizers."""
    v = _normal(g, (rows, k), std)
    if gran == "tensor":
        s = FMAX[fmt] / v.abs().amax()
        return _codes(v * s, fmt), (1 / s).reshape(1)
    if gran == "mx":
        run = v.view(rows, k // 32, 32)
        e = torch.ceil(torch.log2(run.abs().amax(2) / FMAX[fmt])).clamp(-126, 126)
        return (_codes(run * torch.exp2(-e)[..., None], fmt).view(rows, k),
                (e + 127).to(torch.uint8).t().contiguous())
    if gran == "tile":
        run = v.view(rows, k // 128, 128)
        s = FMAX[fmt] / run.abs().amax(2)
        return _codes(run * s[..., None], fmt).view(rows, k), (1 / s).t().contiguous()
    blocks = -(-rows // 128)
    padded = torch.zeros((blocks * 128, k), device=DEV)
    padded[:rows] = v
    run = padded.view(blocks, 128, k // 128, 128)
    s = FMAX[fmt] / run.abs().amax((1, 3))
    return _codes(run * s[:, None, :, None], fmt).view(-1, k)[:rows].contiguous(), 1 / s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, st = case["op"], dict(case)
    if op == "gemm_residual":
        m, n, k, mode = case["m"], case["n"], case["k"], case["mode"]
        st["A"], st["sa"] = _operand(g, m, k, 1.0, "tile" if mode == "block" else mode, case["fmt"])
        st["B"], st["sb"] = _operand(g, n, k, k ** -0.5, mode, "e4m3")
        out = n // 2 if case["act"] == "swiglu" else n
        st["bias"] = _normal(g, (n,), 0.1) if case["bias"] else None
        st["R"] = _normal(g, (m, out), 1.0, HP[case["dtype"]])
        return st
    r, c, t = case["rows"], case["cols"], HP[case["dtype"]]
    if op in ("layernorm", "layernorm_backward"):
        # a residual stream: rows of different scale and offset
        x = _normal(g, (r, c)) * (0.5 + torch.rand((r, 1), generator=g, device=DEV)) + _normal(g, (r, 1), 0.5)
        st["x"] = x.to(t)
        st["gamma"], st["beta"] = 1 + _normal(g, (c,), 0.1), _normal(g, (c,), 0.1)
        if op == "layernorm_backward":
            x = st["x"].double()
            mu = x.mean(1)
            st["mu"] = mu.float()
            st["rs"] = ((x - mu[:, None]).square().mean(1) + EPS).rsqrt().float()
            st["dY"] = _normal(g, (r, c), 1e-2, HP[case["dy"]])
            st["dR"] = _normal(g, (r, c), 1e-2, t) if case["dres"] else None
        return st
    st["pre"] = None if case["act"] == "none" else _normal(g, (r, c), 1.0, t)
    std = 1.0
    if op == "act_backward":
        std = 1e-3
        st["dY"] = _normal(g, (r, c // 2 if case["act"] == "swiglu" else c), std, t)
    # the delayed recipe's scale of the step before: an amax of about six deviations
    st["scale"] = torch.full((1,), FMAX[case["fmt"]] / (6 * std), device=DEV)
    st["slot"] = torch.zeros(1, device=DEV)
    return st


# ------------------------------------------------------------------ one pass


def _phi(v):
    return 0.5 * torch.special.erfc(v * -0.7071067811865476)


def _activation(pre, act):
    if act == "gelu":
        return pre * _phi(pre)
    gate, up = pre[:, 0::2], pre[:, 1::2]
    return gate / (1 + torch.exp(-gate)) * up


def _gradient(dy, pre, act):
    """d pre from d act(pre)."""
    if act == "none":
        return dy
    if act == "gelu":
        return dy * (_phi(pre) + pre * torch.exp(-0.5 * pre * pre) * 0.3989422804014327)
    gate, up = pre[:, 0::2], pre[:, 1::2]
    s = 1 / (1 + torch.exp(-gate))
    return torch.stack((dy * up * s * (1 + gate * (1 - s)), dy * gate * s), 2).flatten(1)


def _cast_both(v, st):
    """The FP8 copy of v, that of its transpose, and the amax or both copies' scales."""
    fmt = st["fmt"]
    if st["gran"] == "tensor":
        torch.maximum(st["slot"], v.abs().amax(), out=st["slot"])
        q = _codes(v * st["scale"], fmt)
        return q.view(F8[fmt]), q.t().contiguous().view(F8[fmt]), st["slot"]
    q, si = _cast_runs(v, fmt)
    qt, sit = _cast_runs(v.t(), fmt)
    return q, si, qt, sit


def _cast_runs(v, fmt):
    """One scale for each 128 along the rows of v: the codes and [cols / 128][rows] of 1 / scale."""
    run = v.reshape(v.shape[0], -1, 128)
    amax = run.abs().amax(2)
    s = torch.where(amax > 0, FMAX[fmt] / amax, 1.0)
    return _codes(run * s[..., None], fmt).view(v.shape).view(F8[fmt]), (1 / s).t().contiguous()


def _operand_values(codes, scale_inv, gran, fmt, t):
    """The values that an operand's codes stand for."""
    v = codes.view(F8[fmt]).to(t)
    rows, k = v.shape
    if gran == "tensor":
        return v * scale_inv.to(t)
    if gran == "mx":
        return (v.view(rows, -1, 32) * torch.exp2(scale_inv.t().to(t) - 127)[..., None]).view(rows, k)
    if gran == "tile":
        return (v.view(rows, -1, 128) * scale_inv.t().to(t)[..., None]).view(rows, k)
    wide = scale_inv.to(t).repeat_interleave(128, 0)[:rows]
    return (v.view(rows, -1, 128) * wide[..., None]).view(rows, k)


def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "layernorm":
        x = st["x"].float()
        mu = x.mean(1)
        rs = 1 / torch.sqrt((x - mu[:, None]).square().mean(1) + EPS)
        y = (x - mu[:, None]) * rs[:, None] * st["gamma"] + st["beta"]
        return y.to(HP[st["out"]]), mu, rs
    if op == "layernorm_backward":
        dy, rs = st["dY"].float(), st["rs"][:, None]
        xh = (st["x"].float() - st["mu"][:, None]) * rs
        g = dy * st["gamma"]
        dx = rs * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if st["dR"] is not None:
            dx = dx + st["dR"].float()
        return dx.to(st["x"].dtype), (dy * xh).sum(0), dy.sum(0)
    if op == "act":
        return _cast_both(_activation(st["pre"].float(), st["act"]), st)
    if op == "act_backward":
        pre = None if st["pre"] is None else st["pre"].float()
        d = _gradient(st["dY"].float(), pre, st["act"])
        return _cast_both(d, st) + (d.sum(0),)
    gran_a = "tile" if st["mode"] == "block" else st["mode"]
    a = _operand_values(st["A"], st["sa"], gran_a, st["fmt"], torch.float32)
    v = a @ _operand_values(st["B"], st["sb"], st["mode"], "e4m3", torch.float32).t()
    if st["bias"] is not None:
        v = v + st["bias"]
    if st["act"] != "none":
        v = _activation(v, st["act"])
    return (v + st["R"].float()).to(HP[st["dtype"]])


def _run_own(st):
    import scaled_quantize_gemm_amd as sq

    op = st["op"]
    if op == "layernorm":
        x = st["x"]
        mu, rs = torch.empty(2, x.shape[0], device=x.device).unbind(0)
        y = sq.fp8_layernorm(x, st["gamma"], st["beta"], EPS, sq.OUT_F32 if st["out"] == "f32" else sq.OUT_BF16,
                             mu=mu, rsigma=rs)
        return y, mu, rs
    if op == "layernorm_backward":
        return sq.fp8_layernorm_backward(st["dY"], st["x"], st["gamma"], st["mu"], st["rs"], dres=st["dR"])
    act = {"none": sq.FP8_ACT_NONE, "gelu": sq.FP8_ACT_GELU, "swiglu": sq.FP8_ACT_SWIGLU}[st["act"]]
    fmt = sq.FP8_E5M2 if st["fmt"] == "e5m2" else sq.FP8_E4M3
    if op == "gemm_residual":
        ga, gb = {"tensor": (sq.FP8_SCALE_TENSOR, sq.FP8_SCALE_TENSOR), "mx": (sq.FP8_SCALE_MX_1x32,) * 2,
                  "block": (sq.FP8_SCALE_TILE_1x128, sq.FP8_SCALE_BLOCK_128x128)}[st["mode"]]
        return sq.fp8_gemm_residual(st["A"], fmt, st["sa"], ga, st["B"], sq.FP8_E4M3, st["sb"], gb, st["R"],
                                    sq.OUT_F32 if st["dtype"] == "f32" else sq.OUT_BF16, bias=st["bias"], act=act)
    tensor = st["gran"] == "tensor"
    scaling = (dict(granularity=sq.FP8_SCALE_TENSOR, scale=st["scale"], amax_slot=st["slot"]) if tensor
               else dict(granularity=sq.FP8_SCALE_TILE_1x128))
    if op == "act":
        q, si, qt, sit = sq.fp8_act_cast_transpose(st["pre"], act, fmt, **scaling)
        more = ()
    else:
        q, si, qt, sit, dbias = sq.fp8_act_backward(st["dY"], st["pre"], act, fmt, **scaling)
        more = (dbias,)
    q, qt = q.view(F8[st["fmt"]]), qt.view(F8[st["fmt"]])
    return ((q, qt, st["slot"]) if tensor else (q, si, qt, sit)) + more


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "layernorm":
        x = st["x"].double()
        d = x - x.mean(dim=-1, keepdim=True)
        rs = (d.pow(2).mean(dim=-1, keepdim=True) + EPS).pow(-0.5)
        y = torch.addcmul(st["beta"].double(), d * rs, st["gamma"].double())
        return y, x.mean(dim=-1), rs.flatten()
    if op == "layernorm_backward":
        # the derivative with mu and rs as functions of x, at the given values of both
        rs, dy, c = st["rs"].double(), st["dY"].double(), case["cols"]
        n = torch.einsum("rc,r->rc", st["x"].double() - st["mu"].double().unsqueeze(1), rs)
        w = dy * st["gamma"].double()
        inner = w * c - w.sum(1, keepdim=True) - n * (w * n).sum(1, keepdim=True)
        dx = inner * (rs / c).unsqueeze(1)
        return (dx if st["dR"] is None else dx + st["dR"].double()), (n * dy).sum(0), dy.sum(0)
    if op in ("act", "act_backward"):
        h = _exact_act(case, st)
        if case["gran"] == "tensor":
            q = _on_grid(h * st["scale"].double(), case["fmt"])
            out = (q, q.t().contiguous(), h.abs().max().reshape(1))
        else:
            out = _exact_runs(h, case["fmt"]) + _exact_runs(h.t().contiguous(), case["fmt"])
        return out + ((h.sum(0),) if op == "act_backward" else ())
    return _exact_gemm(case, st)


def _exact_act(case, st):
    """act(pre), or its gradient times dY where the state has one, in 64 bits."""
    dy = st["dY"].double() if "dY" in st else None
    if case["act"] == "none":
        return dy
    p = st["pre"].double()
    if case["act"] == "gelu":
        cdf = (1 + torch.erf(p / 2 ** 0.5)) / 2
        return p * cdf if dy is None else dy * cdf + dy * p * torch.exp(-p.pow(2) / 2) / (2 * torch.pi) ** 0.5
    gate, up = p.unflatten(1, (-1, 2)).unbind(2)
    s = torch.sigmoid(gate)
    if dy is None:
        return gate * s * up
    out = torch.empty_like(p)
    out[:, ::2] = dy * up * (s + gate * s * torch.sigmoid(-gate))
    out[:, 1::2] = dy * s * gate
    return out


def _on_grid(v, fmt):
    """v on the format's grid, saturating: to the nearest multiple of its binade's step, ties to the even one."""
    bits, least = {"e4m3": (3, -6), "e5m2": (2, -14)}[fmt]
    binade = (torch.frexp(v).exponent - 1).clamp(min=least)
    step = torch.ldexp(torch.ones_like(v), binade - bits)
    return (torch.round(v / step) * step).clamp(-FMAX[fmt], FMAX[fmt])


def _exact_runs(h, fmt):
    """Codes' values under each column run's scale, and 1 / scale by column run."""
    amax = h.unflatten(1, (-1, 128)).abs().max(dim=2).values
    codes = _on_grid(h / amax.repeat_interleave(128, dim=1) * FMAX[fmt], fmt)
    return codes, (amax / FMAX[fmt]).t().contiguous()


def _exact_gemm(case, st):
    def values(codes, scale, fmt, run, by_row):
        v = codes.view(F8[fmt]).double()
        if run is None:
            return v * scale.double()
        s = scale.double() if by_row else scale.double().t()
        return v * s.repeat_interleave(run, dim=1)

    mode = case["mode"]
    if mode == "mx":
        sa, sb = (torch.pow(2.0, st[k].double() - 127) for k in ("sa", "sb"))
        a, b = values(st["A"], sa, case["fmt"], 32, False), values(st["B"], sb, "e4m3", 32, False)
    elif mode == "block":
        rows = st["sb"].repeat_interleave(128, dim=0)[: case["n"]]
        a, b = values(st["A"], st["sa"], case["fmt"], 128, False), values(st["B"], rows, "e4m3", 128, True)
    else:
        a, b = values(st["A"], st["sa"], case["fmt"], None, True), values(st["B"], st["sb"], "e4m3", None, True)
    v = a.mm(b.t().contiguous())
    if case["bias"]:
        v += st["bias"].double()
    if case["act"] == "gelu":
        v = v * (1 + torch.erf(v / 2 ** 0.5)) / 2
    elif case["act"] == "swiglu":
        gate, up = v.unflatten(1, (-1, 2)).unbind(2)
        v = gate * torch.sigmoid(gate) * up
    return v + st["R"].double()
