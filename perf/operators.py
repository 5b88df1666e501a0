"""Cases of the MoE-block operators: RMS norm with the residual's addition and
an MX output (forward and backward), routing to experts with its dispatch plan
(forward and backward), and matrix-vector products with 4-bit weights (dense
NVFP4 and MXFP4, and the routed expert form).

`run` computes a case in its plain form, elementary torch operations, or, where
`own` is true, through this package.  `exact` computes it in 64 bits, written
apart from the plain form.

8-bit outputs are returned as what their bytes stand for: E4M3 codes as
float8_e4m3fn and E8M0 scale bytes as float8_e8m0fnu.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # decode: one token's residual stream, normalised into the MXFP8
        # operand of the next product
        dict(name="norm_token", op="norm", rows=1, cols=7168, dtype="bf16", mx=True, y=False),
        # prefill of 8192 tokens, hidden 5120: both the MXFP8 operand and the BF16
        # value a router reads
        dict(name="norm_prefill", op="norm", rows=8192, cols=5120, dtype="bf16", mx=True, y=True),
        # training, one step's 16384 tokens at hidden 7168: the backward pass,
        # with the residual stream's own gradient
        dict(name="norm_backward", op="norm_bwd", rows=16384, cols=7168, dtype="bf16"),
        # a ragged binary32 layer: odd row count, width not a multiple of anything
        dict(name="norm_backward_ragged", op="norm_bwd", rows=777, cols=1003, dtype="f32"),
        # decode: one token over 256 experts in 8 groups, sigmoid scores with a
        # balance bias
        dict(name="route_token", op="route", tokens=1, experts=256, top_k=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, dtype="f32"),
        # the MoE layer of 32 experts, 16384 tokens, top 4, softmax scores
        dict(name="route_32", op="route", tokens=16384, experts=32, top_k=4, score="softmax", bias=False,
             groups=1, top_groups=1, dtype="bf16"),
        # many fine-grained experts: 256 in 8 groups, top 8, sigmoid with bias
        dict(name="route_256", op="route", tokens=16384, experts=256, top_k=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, dtype="f32"),
        # training: gradients of the weights and of an auxiliary balance loss
        # on all scores back to the logits
        dict(name="route_backward", op="route_bwd", tokens=16384, experts=256, top_k=8, score="softmax",
             dtype="bf16"),
        # a few tokens against a small odd-sized layer, binary32 activations
        dict(name="gemv_small", op="gemv", m=3, n=1000, k=1040, fmt="nvfp4", two_d=False, dtype="f32"),
        # decode: one token against a 20480 x 5120 weight with 16x16 scales
        dict(name="gemv_token", op="gemv", m=1, n=20480, k=5120, fmt="nvfp4", two_d=True, dtype="bf16"),
        # a small batch of tokens against an 8192 x 8192 MXFP4 weight
        dict(name="gemv_mx", op="gemv", m=8, n=8192, k=8192, fmt="mx", two_d=False, dtype="bf16"),
        # decode of four tokens through the routed experts: up-projection with
        # SwiGLU, down-projection with the weighted sum over the token's experts
        dict(name="expert_ffn", op="expert", tokens=4, top_k=4, experts=32, hidden=7168, ffn=2048,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "route", "route_bwd", "gemv", "gemv", "expert"])
    if op in ("norm", "norm_bwd"):
        cols = _log(rng, 32, 16384)
        rows = _log(rng, 1, max(1, min(16384, (8192 * 5120) // cols)))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "norm_bwd":
            return dict(op=op, rows=rows, cols=cols, dtype=dtype)
        mx = rng.random() < 0.7
        if mx:
            cols = max(32, cols // 32 * 32)
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, mx=mx, y=(not mx) or rng.random() < 0.5)
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * rng.randint(max(2, 8 // groups), 512 // groups)
        tokens = _log(rng, 1, 16384)
        score = rng.choice(["softmax", "sigmoid"])
        dtype = rng.choice(["bf16", "f32"])
        if op == "route_bwd":
            return dict(op=op, tokens=tokens, experts=experts, top_k=rng.randint(1, 8), score=score, dtype=dtype)
        top_groups = rng.randint(1, groups)
        return dict(op=op, tokens=tokens, experts=experts, top_k=rng.randint(1, min(8, top_groups * (experts // groups))),
                    score=score, bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, dtype=dtype)
    if op == "gemv":
        fmt = rng.choice(["nvfp4", "nvfp4", "mx"])
        two_d = fmt == "nvfp4" and rng.random() < 0.5
        unit = 32 if fmt == "mx" else 16
        k = unit * _log(rng, 2, 20480 // unit)
        n = _log(rng, 16, min(20480, (20480 * 5120) // k))
        if two_d:
            n = max(16, n // 16 * 16)
        return dict(op=op, m=_log(rng, 1, 16), n=n, k=k, fmt=fmt, two_d=two_d,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    experts = rng.randint(4, 32)
    return dict(op=op, tokens=rng.randint(1, 8), top_k=rng.randint(1, min(4, experts)), experts=experts,
                hidden=16 * _log(rng, 4, 7168 // 16), ffn=16 * _log(rng, 2, 2048 // 16), dtype="bf16")


def work(c):
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        n, es = c["rows"] * c["cols"], 2 if c["dtype"] == "bf16" else 4
        if op == "norm":  # x, residual in; h, (y), (codes and scales), rstd out
            b = n * es * 3 + 4 * c["rows"] + c["cols"] * 4
            b += n * es if c["y"] else 0
            b += n * 33 // 32 if c["mx"] else 0
            return {"bytes": b, "flops": 6 * n}
        # dy, h, dh in; dx, dweight out
        return {"bytes": n * es * 4 + 4 * c["rows"] + c["cols"] * 8, "flops": 11 * n}
    if op in ("route", "route_bwd"):
        n, a, es = c["tokens"] * c["experts"], c["tokens"] * c["top_k"], 2 if c["dtype"] == "bf16" else 4
        if op == "route":  # logits, bias in; ids, weights, order, position, offsets out
            return {"bytes": n * es + 16 * a + 12 * c["experts"], "flops": 4 * n}
        return {"bytes": 2 * n * es + 4 * n + 8 * a, "flops": 8 * n}  # logits, dscores in; dlogits out
    if op == "gemv":
        nk, es = c["n"] * c["k"], 2 if c["dtype"] == "bf16" else 4
        scales = nk // 256 if c["two_d"] else nk // (32 if c["fmt"] == "mx" else 16)
        return {"bytes": nk // 2 + scales + c["m"] * (c["k"] + c["n"]) * es, "flops": 2 * c["m"] * nk}
    # the weights of the experts that the tokens chose (about this many distinct ones)
    t, k, e, h, f = c["tokens"], c["top_k"], c["experts"], c["hidden"], c["ffn"]
    distinct = e * (1.0 - (1.0 - k / e) ** t)
    return {"bytes": int(distinct * 3 * f * h * (0.5 + 1 / 256)) + t * 4 * h + t * k * 2 * f,
            "flops": 2 * t * k * 3 * f * h}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _activations(g, shape, dtype):
    """Normal values, a few channels (last dimension) far larger, as hidden states have."""
    x = torch.randn(shape, generator=g, device=DEV)
    loud = torch.rand(shape[-1], generator=g, device=DEV) < 0.005
    return (x * (1.0 + 20.0 * loud)).to(dtype)


def _e2m1_codes(y):
    """E2M1 codes (uint8) of y, nearest, by the grid's midpoints; magnitudes past 6 saturate."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=y.device)
    return torch.bucketize(y.abs(), mid).to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _nvfp4_weight(g, rows, cols, two_d):
    """A normal weight's NVFP4 codes, scale bytes and tensor scale."""
    w = 0.02 * torch.randn((rows, cols), generator=g, device=DEV)
    ts = w.abs().max() / 2688.0
    if two_d:
        amax = w.view(rows // 16, 16, cols // 16, 16).abs().amax(dim=(1, 3))
    else:
        amax = w.view(rows, cols // 16, 16).abs().amax(dim=2)
    sb = (amax / (6.0 * ts)).clamp(max=448.0).to(torch.float8_e4m3fn)
    full = (sb.float() * ts).clamp(min=1e-30)
    full = full.repeat_interleave(16, 0) if two_d else full
    q = (w.view(rows, cols // 16, 16) / full.unsqueeze(2)).view(rows, cols)
    return _pack(_e2m1_codes(q)), sb.view(torch.uint8), ts.reshape(1)


def _mx_weight(g, rows, cols):
    """A normal weight's MXFP4 codes and E8M0 scale bytes."""
    w = 0.02 * torch.randn((rows, cols), generator=g, device=DEV)
    s = torch.frexp(w.view(rows, cols // 32, 32).abs().amax(dim=2)).exponent - 1 - 2
    q = torch.ldexp(w.view(rows, cols // 32, 32), -s.unsqueeze(2)).view(rows, cols)
    return _pack(_e2m1_codes(q)), (s + 127).to(torch.uint8)


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = DTYPES[c["dtype"]]
    st = {"case": dict(c)}
    if c["op"] == "norm":
        st["x"] = 0.1 * _activations(g, (c["rows"], c["cols"]), dt)
        st["residual"] = _activations(g, (c["rows"], c["cols"]), dt)
        st["weight"] = (1.0 + 0.1 * torch.randn(c["cols"], generator=g, device=DEV)).to(dt)
    elif c["op"] == "norm_bwd":
        st["h"] = _activations(g, (c["rows"], c["cols"]), dt)
        st["weight"] = (1.0 + 0.1 * torch.randn(c["cols"], generator=g, device=DEV)).to(dt)
        st["dy"] = torch.randn((c["rows"], c["cols"]), generator=g, device=DEV).to(dt)
        st["dh"] = torch.randn((c["rows"], c["cols"]), generator=g, device=DEV).to(dt)
        # what the forward pass kept
        st["rstd"] = torch.rsqrt(st["h"].float().square().mean(dim=1) + 1e-6)
    elif c["op"] in ("route", "route_bwd"):
        t, e = c["tokens"], c["experts"]
        popular = 0.5 * torch.randn(e, generator=g, device=DEV)
        st["logits"] = (torch.randn((t, e), generator=g, device=DEV) + popular).to(dt)
        st["bias"] = 0.05 * torch.randn(e, generator=g, device=DEV) if c.get("bias") else None
        if c["op"] == "route_bwd":
            st["ids"] = torch.topk(st["logits"].float(), min(c["top_k"], e), dim=1).indices.to(torch.int32)
            st["dweights"] = torch.randn(st["ids"].shape, generator=g, device=DEV)
            st["dscores"] = 0.1 * torch.randn((t, e), generator=g, device=DEV)
    elif c["op"] == "gemv":
        st["x"] = _activations(g, (c["m"], c["k"]), dt)
        if c["fmt"] == "mx":
            st["w"] = _mx_weight(g, c["n"], c["k"])
        else:
            st["w"] = _nvfp4_weight(g, c["n"], c["k"], c["two_d"])
    else:
        t, k, e, h, f = c["tokens"], c["top_k"], c["experts"], c["hidden"], c["ffn"]
        st["x"] = _activations(g, (t, h), dt)
        score = torch.rand((t, e), generator=g, device=DEV)
        st["ids"] = torch.topk(score, k, dim=1).indices.to(torch.int32)
        w = torch.rand((t, k), generator=g, device=DEV) + 0.1
        st["weights"] = w / w.sum(dim=1, keepdim=True)
        for name, rows, cols in (("up", 2 * f, h), ("down", h, f)):
            per = [_nvfp4_weight(g, rows, cols, True) for _ in range(e)]
            st[name] = tuple(torch.cat([p[i] for p in per]) for i in range(3))
    return st


# ------------------------------------------------------------------ the plain forms
def _f8(codes, scales):
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def _mx_plain(y):
    r, c = y.shape
    b = y.view(r, c // 32, 32)
    amax = b.abs().amax(dim=2)
    s = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 8, -127).clamp(min=-127)
    q = torch.ldexp(b, -s.unsqueeze(2)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return _f8(q.view(r, c), (s + 127).to(torch.uint8))


def _norm_plain(st):
    c, dt = st["case"], st["x"].dtype
    h = (st["x"].float() + st["residual"].float()).to(dt)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(dim=1) + 1e-6)
    y = hf * rstd.unsqueeze(1) * st["weight"].float()
    out = {"h": h, "rstd": rstd}
    if c["y"]:
        out["y"] = y.to(dt)
    if c["mx"]:
        out["mx"] = _mx_plain(y)
    return out


def _norm_bwd_plain(st):
    dy, h, rstd = st["dy"].float(), st["h"].float(), st["rstd"].unsqueeze(1)
    g, xhat = dy * st["weight"].float(), h * rstd
    dx = rstd * (g - xhat * (g * xhat).mean(dim=1, keepdim=True)) + st["dh"].float()
    return {"dx": dx.to(st["dy"].dtype), "dweight": (dy * xhat).sum(dim=0)}


def _scores(logits, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _route_plain(st):
    c = st["case"]
    t, e, k, ng = c["tokens"], c["experts"], c["top_k"], c["groups"]
    # in 64 bits: two experts' scores may lie closer than 32 bits resolve
    p = _scores(st["logits"].double(), c["score"])
    s = p if st["bias"] is None else p + st["bias"].double()
    if ng > 1:
        by = s.view(t, ng, e // ng).sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
        kept = by.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros((t, ng), dtype=torch.bool, device=p.device).scatter_(1, kept, True)
        s = torch.where(keep.repeat_interleave(e // ng, 1), s, -math.inf)
    ids = s.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    w = (w / w.sum(dim=1, keepdim=True)).float()
    flat = ids.reshape(-1)
    order = flat.sort(stable=True)
    position = torch.empty_like(order.indices).scatter_(0, order.indices, torch.arange(t * k, device=p.device))
    offsets = torch.searchsorted(order.values, torch.arange(e + 1, device=p.device))
    return {"ids": ids.to(torch.int32), "weights": w, "offsets": offsets,
            "order": order.indices.to(torch.int32), "position": position.to(torch.int32)}


def _route_bwd_plain(st):
    c = st["case"]
    ids, dw = st["ids"].long(), st["dweights"]
    p = _scores(st["logits"].float(), c["score"])
    w = p.gather(1, ids)
    total = w.sum(dim=1, keepdim=True)
    w = w / total
    dsel = (dw - (dw * w).sum(dim=1, keepdim=True)) / total
    dp = st["dscores"].scatter_add(1, ids, dsel)
    if c["score"] == "sigmoid":
        dl = dp * p * (1.0 - p)
    else:
        dl = p * (dp - (p * dp).sum(dim=1, keepdim=True))
    return {"dlogits": dl.to(st["logits"].dtype)}


def _e2m1_values(codes, dtype):
    v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device,
                     dtype=dtype)
    both = torch.stack((codes & 15, codes >> 4), dim=-1).view(*codes.shape[:-1], 2 * codes.shape[-1])
    return v[both.long()]


def _nvfp4_values(w, two_d):
    """The weight without its tensor scale."""
    codes, sb, _ = w
    s = sb.view(torch.float8_e4m3fn).float()
    s = s.repeat_interleave(16, 0) if two_d else s
    return _e2m1_values(codes, torch.float32) * s.repeat_interleave(16, 1)


def _gemv_plain(st):
    c, x = st["case"], st["x"].float()
    if c["fmt"] == "mx":
        codes, sb = st["w"]
        s = torch.ldexp(torch.ones((), device=x.device), sb.int() - 127)
        w, ts = _e2m1_values(codes, torch.float32) * s.repeat_interleave(32, 1), 1.0
    else:
        w, ts = _nvfp4_values(st["w"], c["two_d"]), st["w"][2]
    return {"y": (torch.matmul(x, w.t()) * ts).to(st["x"].dtype)}


def _expert_plain(st):
    c = st["case"]
    t, k, e, h, f = c["tokens"], c["top_k"], c["experts"], c["hidden"], c["ffn"]
    ids = st["ids"].long().reshape(-1)

    def chosen(w, rows, cols):
        codes, sb, ts = w
        codes = codes.view(e, rows, cols // 2)[ids].view(-1, cols // 2)
        sb = sb.view(e, rows // 16, cols // 16)[ids].view(-1, cols // 16)
        return _nvfp4_values((codes, sb, ts), True).view(t * k, rows, cols), ts[ids].view(-1, 1)

    up, ts = chosen(st["up"], 2 * f, h)
    x = st["x"].float().repeat_interleave(k, 0)
    z = torch.bmm(up, x.unsqueeze(2)).squeeze(2) * ts
    del up
    gate, lin = z[:, :f], z[:, f:]
    a = (gate / (1.0 + torch.exp(-gate)) * lin).to(st["x"].dtype)
    down, ts = chosen(st["down"], h, f)
    y = torch.bmm(down, a.float().unsqueeze(2)).squeeze(2) * ts
    y = (y.view(t, k, h) * st["weights"].unsqueeze(2)).sum(dim=1)
    return {"a": a, "y": y.to(st["x"].dtype)}


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    import bit_block_scaled_quantize_amd as nv

    c = st["case"]
    if c["op"] == "norm":
        r = nv.nvfp4_rmsnorm(st["x"], st["weight"], residual=st["residual"], eps=1e-6, y=c["y"],
                             mx_elem=nv.NVFP4_MX_E4M3 if c["mx"] else None, rstd=True)
        out = {"h": r.h, "rstd": r.rstd}
        if c["y"]:
            out["y"] = r.y
        if c["mx"]:
            out["mx"] = _f8(r.mx.codes, r.mx.scales)
        return out
    if c["op"] == "norm_bwd":
        dx, dweight = nv.nvfp4_rmsnorm_backward(st["dy"], st["h"], st["rstd"], st["weight"], dh=st["dh"])
        return {"dx": dx, "dweight": dweight}
    if c["op"] in ("route", "route_bwd"):
        score = nv.NVFP4_ROUTE_SIGMOID if c["score"] == "sigmoid" else nv.NVFP4_ROUTE_SOFTMAX
        if c["op"] == "route_bwd":
            return {"dlogits": nv.nvfp4_route_backward(st["dweights"], st["logits"], st["ids"], score=score,
                                                       renorm=True, dscores=st["dscores"])}
        r = nv.nvfp4_route(st["logits"], c["top_k"], bias=st["bias"], score=score, groups=c["groups"],
                           top_groups=c["top_groups"], group_score=nv.NVFP4_GROUP_TOP2, renorm=True)
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "order": r.order,
                "position": r.position}
    if c["op"] == "gemv":
        if c["fmt"] == "mx":
            w = nv.MXTensor(*st["w"], c["n"], c["k"], nv.NVFP4_MX_E2M1)
            return {"y": nv.nvfp4_mx_gemv(st["x"], w)}
        w = nv.NVFP4Tensor(*st["w"], c["n"], c["k"], nv.NVFP4_SCALE_2D if c["two_d"] else nv.NVFP4_SCALE_1D)
        return {"y": nv.nvfp4_gemv(st["x"], w)}
    e, h, f = c["experts"], c["hidden"], c["ffn"]
    up = nv.NVFP4Tensor(*st["up"], e * 2 * f, h, nv.NVFP4_SCALE_2D)
    down = nv.NVFP4Tensor(*st["down"], e * h, f, nv.NVFP4_SCALE_2D)
    a = nv.nvfp4_expert_gemv(st["x"], st["ids"], up, e, epilogue=nv.NVFP4_EPI_SWIGLU)
    y = nv.nvfp4_expert_gemv(a, st["ids"], down, e, weights=st["weights"])
    return {"a": a, "y": y}


PLAIN = {"norm": _norm_plain, "norm_bwd": _norm_bwd_plain, "route": _route_plain, "route_bwd": _route_bwd_plain,
         "gemv": _gemv_plain, "expert": _expert_plain}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits
def _exact_mx(y):
    r, c = y.shape
    b = y.reshape(r, c // 32, 32)
    amax = b.abs().max(dim=2, keepdim=True).values
    s = torch.where(amax > 0, torch.floor(torch.log2(amax.clamp(min=1e-300))) - 8, -127.0).clamp(min=-127.0)
    m = (b.abs() / 2.0 ** s)
    step = 2.0 ** (torch.floor(torch.log2(m.clamp(min=2.0 ** -6))) - 3)
    q = torch.copysign((torch.round(m / step) * step).clamp(max=448.0), b)
    return {"codes": q.reshape(r, c), "scales": (2.0 ** s).squeeze(2)}


def _exact_scores(logits, score):
    l = logits.double()
    return torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, dim=1)


def _exact_weight(w, rows, cols, two_d):
    """The rows x cols weight of codes and E4M3 scale bytes, without its tensor scale."""
    grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], device=w[0].device, dtype=torch.float64) / 2
    low, high = w[0] % 16, w[0] // 16
    v = torch.empty((rows, cols), dtype=torch.float64, device=w[0].device)
    for at, code in ((0, low), (1, high)):
        v[:, at::2] = grid[(code % 8).long()] * (1 - 2 * (code // 8).double())
    sb = w[1].int()
    s = torch.where(sb >= 8, (8 + sb % 8).double() * 2.0 ** ((sb // 8).double() - 10), (sb % 8).double() * 2.0 ** -9)
    v = v.view(rows // 16, 16, cols // 16, 16) if two_d else v.view(rows, cols // 16, 16)
    v *= s[:, None, :, None] if two_d else s[:, :, None]
    return v.view(rows, cols)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "norm":
        x, r = st["x"].double(), st["residual"].double()
        h = (x + r).to(st["x"].dtype).double()  # the norm is that of the stored sum
        rstd = 1.0 / torch.sqrt((h * h).sum(dim=1) / c["cols"] + 1e-6)
        y = h * rstd[:, None] * st["weight"].double()
        out = {"h": x + r, "rstd": rstd}
        if c["y"]:
            out["y"] = y
        if c["mx"]:
            out["mx"] = _exact_mx(y)
        return out
    if c["op"] == "norm_bwd":
        h, dy, w = st["h"].double(), st["dy"].double(), st["weight"].double()
        rstd = st["rstd"].double()[:, None]  # an input, as the forward pass kept it
        dot = (dy * w * h).sum(dim=1, keepdim=True) / c["cols"]
        dx = rstd * dy * w - rstd ** 3 * h * dot + st["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("ij,ij->j", dy, h * rstd)}
    if c["op"] == "route":
        p = _exact_scores(st["logits"], c["score"])
        s = p if st["bias"] is None else p + st["bias"].double()
        if c["groups"] > 1:
            g = s.view(c["tokens"], c["groups"], -1)
            best = torch.topk(torch.topk(g, min(2, g.shape[2]), dim=2).values.sum(dim=2), c["top_groups"], dim=1)
            out = torch.ones(g.shape[:2], dtype=torch.bool, device=DEV)
            out[torch.arange(c["tokens"], device=DEV)[:, None], best.indices] = False
            s = g.masked_fill(out[:, :, None], -math.inf).view_as(s)
        # equal scores have equal weights, whichever of them is taken
        w = torch.take_along_dim(p, torch.topk(s, c["top_k"], dim=1).indices, dim=1)
        return {"ids": None, "weights": w / w.sum(dim=1, keepdim=True), "offsets": None, "order": None,
                "position": None}
    if c["op"] == "route_bwd":
        # by the chain rule through an autograd graph in 64 bits
        l = st["logits"].double().requires_grad_(True)
        p = _exact_scores(l, c["score"])
        w = torch.take_along_dim(p, st["ids"].long(), dim=1)
        w = w / w.sum(dim=1, keepdim=True)
        ((w * st["dweights"].double()).sum() + (p * st["dscores"].double()).sum()).backward()
        return {"dlogits": l.grad}
    if c["op"] == "gemv":
        x = st["x"].double()
        if c["fmt"] == "mx":
            codes, sb = st["w"]
            w = _exact_weight((codes, torch.full((c["n"], c["k"] // 16), 56, dtype=torch.uint8, device=x.device)),
                              c["n"], c["k"], False)  # byte 56 stands for 1
            w = (w.view(c["n"], -1, 32) * (2.0 ** (sb.double() - 127))[:, :, None]).view(c["n"], c["k"])
            return {"y": torch.mm(x, w.t().contiguous())}
        w = _exact_weight(st["w"], c["n"], c["k"], c["two_d"])
        return {"y": torch.mm(x, w.t().contiguous()) * st["w"][2].double()}
    t, k, h, f = c["tokens"], c["top_k"], c["hidden"], c["ffn"]
    a = torch.empty((t * k, f), dtype=torch.float64, device=DEV)
    y = torch.zeros((t, h), dtype=torch.float64, device=DEV)
    x, wts = st["x"].double(), st["weights"].double()
    for i, e in enumerate(st["ids"].reshape(-1).tolist()):
        cu, su, tu = st["up"]
        w = _exact_weight((cu[e * 2 * f:(e + 1) * 2 * f], su[e * 2 * f // 16:(e + 1) * 2 * f // 16]), 2 * f, h, True)
        z = torch.mv(w, x[i // k]) * tu[e].double()
        a[i] = z[:f] * torch.sigmoid(z[:f]) * z[f:]
        cd, sd, td = st["down"]
        w = _exact_weight((cd[e * h:(e + 1) * h], sd[e * h // 16:(e + 1) * h // 16]), h, f, True)
        # the down-projection reads the stored activation
        y[i // k] += wts[i // k, i % k] * td[e].double() * torch.mv(w, a[i].to(st["x"].dtype).double())
    return {"a": a, "y": y}
