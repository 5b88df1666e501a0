"""Cases of the paged key/value cache in 4 bits: appending keys and values with
the rotation of their positions, reading them back (gather), and attention over
the cache (decode of single tokens, a few tokens a sequence, prefill).

`run` computes a case in its plain form, elementary torch operations, or, where
`own` is true, through this package.  `exact` computes it in 64 bits, written
apart from the plain form.

A cache holds, for every page, kv head and slot, `dim` E2M1 codes (two to a byte)
and a scale byte for 16 of them (NVFP4: E4M3, times a float of the head) or 32
(MXFP4: E8M0).  Row t of sequence s, the i-th of its n, has the position
lengths[s] - n + i.  What an append writes is returned as the values that it
stands for, read back by a gather of the same rows.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
THETA = 10000.0  # of the rotation's angles


# ------------------------------------------------------------------ cases
def listed():
    return [
        # decode: one new token of a model of hidden size 5120 (40 heads of 128,
        # 8 kv heads)
        dict(name="append_token", op="append", seqs=1, new=1, ctx=4095, ragged=False, q_heads=40, kv_heads=8, dim=128,
             page=64, fmt="nvfp4", dtype="bf16", rot=128, interleaved=False),
        # prefill of prompts of different lengths, hidden size 7168 (56 heads)
        dict(name="append_prefill", op="append", seqs=6, new=4096, ctx=4096, ragged=True, q_heads=56, kv_heads=8,
             dim=128, page=64, fmt="nvfp4", dtype="bf16", rot=128, interleaved=False),
        # a small odd-sized binary32 model, half of each head rotated in pairs
        dict(name="append_ragged", op="append", seqs=5, new=333, ctx=100, ragged=True, q_heads=9, kv_heads=3, dim=64,
             page=16, fmt="mx", dtype="f32", rot=32, interleaved=True),
        # cached prompts read back whole, to move them to another cache
        dict(name="gather_long", op="gather", seqs=8, new=16384, ctx=0, ragged=True, q_heads=8, kv_heads=8, dim=128,
             page=64, fmt="nvfp4", dtype="bf16"),
        # the last tokens of a few sequences, to check them
        dict(name="gather_few", op="gather", seqs=3, new=50, ctx=1000, ragged=True, q_heads=4, kv_heads=4, dim=64,
             page=16, fmt="mx", dtype="f32"),
        # decode of one sequence of 8192 tokens: latency
        dict(name="attend_token", op="attend", seqs=1, new=1, ctx=8191, ragged=False, q_heads=40, kv_heads=8, dim=128,
             page=64, fmt="nvfp4", dtype="bf16", window=0),
        # decode of a large batch of short conversations
        dict(name="attend_short", op="attend", seqs=256, new=1, ctx=500, ragged=True, q_heads=40, kv_heads=8, dim=128,
             page=16, fmt="nvfp4", dtype="bf16", window=0),
        # decode of a batch of long ones of any length, one slot of the batch unused
        dict(name="attend_batch", op="attend", seqs=64, new=1, ctx=20479, ragged=True, q_heads=56, kv_heads=8, dim=128,
             page=64, fmt="nvfp4", dtype="bf16", window=0),
        # MXFP4, wide heads, one kv head for 16, a sliding window
        dict(name="attend_window", op="attend", seqs=33, new=1, ctx=9999, ragged=True, q_heads=16, kv_heads=1, dim=256,
             page=256, fmt="mx", dtype="bf16", window=4096),
        # a draft of up to 5 tokens to verify for each sequence, binary32
        dict(name="attend_draft", op="attend", seqs=9, new=5, ctx=3001, ragged=True, q_heads=12, kv_heads=4, dim=64,
             page=32, fmt="nvfp4", dtype="f32", window=0),
        # prefill of one prompt of 8192 tokens
        dict(name="attend_prefill", op="attend", seqs=1, new=8192, ctx=0, ragged=False, q_heads=40, kv_heads=8, dim=128,
             page=64, fmt="nvfp4", dtype="bf16", window=0),
        # chunks of prompts behind long cached beginnings
        dict(name="attend_chunk", op="attend", seqs=3, new=1000, ctx=16384, ragged=True, q_heads=32, kv_heads=4, dim=128,
             page=64, fmt="nvfp4", dtype="bf16", window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "gather", "attend", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, ragged=True, kv_heads=kv, q_heads=kv * rng.choice([1, 2, 4, 5, 7, 8, 16]), dim=dim,
             page=rng.choice([16, 32, 64, 128, 256]), fmt=rng.choice(["nvfp4", "nvfp4", "mx"]),
             dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op in ("append", "gather"):
        c["seqs"] = _log(rng, 1, 64)
        most = 15000 * 72 * 128 // (c["seqs"] * (c["q_heads"] + 2 * kv) * dim * (1 if c["dtype"] == "bf16" else 2))
        c["new"] = _log(rng, 1, max(2, min(8192, most)))
        c["ctx"] = _log(rng, 1, 8192)
        if op == "append":
            c["rot"] = rng.choice([r for r in (0, 32, 64, 128, 256) if r <= dim])
            c["interleaved"] = rng.random() < 0.5
        return c
    c["window"] = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    kind = rng.choice(["decode", "decode", "few", "prefill"])
    if kind == "prefill":
        c["seqs"] = rng.randint(1, 4)
        c["new"] = _log(rng, 16, min(2048 if c["dtype"] == "bf16" else 512, 2048 * 64 // c["q_heads"]))
        c["ctx"] = _log(rng, 1, 8192)
    else:
        c["seqs"] = _log(rng, 1, 256)
        c["new"] = 1 if kind == "decode" else rng.randint(2, 8)
        c["ctx"] = _log(rng, 1, max(2, min(32768, (64 * 20480 * 8 * 128) // (c["seqs"] * max(kv, c["q_heads"] // 4) * dim))))
    return c


def _sizes(c):
    """(new rows, length after them) of each sequence, in an order that a seed changes."""
    out = []
    for i in range(c["seqs"]):
        if c["ragged"]:
            new = 1 + round((c["new"] - 1) * math.modf(0.91 + i * math.sqrt(2.0))[0])
            out.append((new, new + round(c["ctx"] * math.modf(0.96 + i * 0.6180339887)[0])))
        else:
            out.append((c["new"], c["new"] + c["ctx"]))
    if c["op"] == "attend" and c["new"] == 1 and c["ragged"] and c["seqs"] >= 8:
        out[-1] = (1, 0)  # a slot of the batch that no sequence uses
    return out


def work(c):
    es, d, hk, hq = 2 if c["dtype"] == "bf16" else 4, c["dim"], c["kv_heads"], c["q_heads"]
    held = d // 2 + d // (32 if c["fmt"] == "mx" else 16)  # bytes of a slot of one head
    sizes = _sizes(c)
    rows = sum(n for n, _ in sizes)
    pages = sum(-(-l // c["page"]) for _, l in sizes)
    plan = 4 * pages + 8 * c["seqs"]
    if c["op"] == "gather":  # slots in; k, v out
        return {"bytes": rows * hk * 2 * (held + d * es) + plan, "flops": 4 * rows * hk * d}
    if c["op"] == "append":  # q, k, v and the angles in; q and slots out, which the gather reads; k, v out
        return {"bytes": rows * (2 * hq * d * es + 2 * hk * d * es + 4 * c["rot"]) + rows * hk * 2 * (2 * held + d * es) + plan,
                "flops": rows * d * (3 * hq + 20 * hk)}
    pairs = keys = 0
    for n, l in sizes:
        w = c["window"] or l + 1
        first = max(0, l - n)  # the position of the first row that has one
        keys += l - max(0, first - w + 1)
        pairs += sum(min(p + 1, w) for p in range(first, l)) if n < 64 or c["window"] else (l - first) * (first + 1 + l) // 2
    return {"bytes": keys * hk * 2 * held + rows * hq * (2 * d * es + 4) + plan, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _heads(g, shape, dtype):
    """Normal values, a few channels (last dimension) larger, as keys and queries have."""
    x = torch.randn(shape, generator=g, device=DEV)
    loud = torch.rand(shape[-1], generator=g, device=DEV) < 0.02
    return (x * (1.0 + 3.0 * loud)).to(dtype)


def _random_slots(g, pages, hk, page, d, fmt, loud):
    """Codes and scale bytes of a normal cache: uniform bytes would stand for no
    distribution that is met, so the codes are those of normal values over
    their block's largest."""
    per = 32 if fmt == "mx" else 16
    codes = torch.empty((pages, hk, page, d // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((pages, hk, page, d // per), dtype=torch.uint8, device=DEV)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    most = max(1, (1 << 27) // (hk * page * d))
    for a in range(0, pages, most):
        n = min(most, pages - a)
        x = torch.randn((n * hk * page, d // per, per), generator=g, device=DEV)
        if loud is not None:
            x *= loud.view(1, d // per, per)
        top = x.abs().amax(dim=2, keepdim=True)
        if fmt == "mx":
            e = torch.frexp(top).exponent - 3
            s, b = torch.ldexp(torch.ones_like(top), e), (e + 127).to(torch.uint8)
        else:
            q = (top / 6.0 * 8.0).to(torch.float8_e4m3fn)  # the head's float is 1 / 8 or near it
            s, b = q.float() / 8.0, q.view(torch.uint8)
        y = x / s
        m = (torch.bucketize(y.abs(), mid, out_int32=True) + 8 * torch.signbit(y)).to(torch.uint8).view(n, hk, page, d // 2, 2)
        codes[a:a + n] = m[..., 0] | (m[..., 1] << 4)
        scales[a:a + n] = b.view(n, hk, page, d // per)
    return codes, scales


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt, hk, hq, d, page = DTYPES[c["dtype"]], c["kv_heads"], c["q_heads"], c["dim"], c["page"]
    sizes = _sizes(c)
    sizes = [sizes[i] for i in torch.randperm(len(sizes), generator=g, device=DEV).tolist()]
    rows, width = sum(n for n, _ in sizes), max(1, max(-(-l // page) for _, l in sizes))
    used = [-(-l // page) for _, l in sizes]
    pages = sum(used) + 3
    st = {"case": dict(c), "rows": rows, "width": width, "pages": pages}
    st["lengths"] = torch.tensor([l for _, l in sizes], dtype=torch.int32).to(DEV)
    new = torch.tensor([n for n, _ in sizes], dtype=torch.int32)
    st["offsets"] = None if c["new"] == 1 else torch.cat([new.new_zeros(1), new.cumsum(0).to(torch.int32)]).to(DEV)
    # pages in any order; places behind a sequence's last page hold -1
    order = torch.randperm(pages, generator=g, device=DEV)[:sum(used)].to(torch.int32)
    count = torch.tensor(used).to(DEV)
    table = torch.full((len(sizes), width), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV)[None, :] < count[:, None]] = order
    st["table"] = table
    loud = 1.0 + 3.0 * (torch.rand(d, generator=g, device=DEV) < 0.02)
    st["k_codes"], st["k_scales"] = _random_slots(g, pages, hk, page, d, c["fmt"], loud)
    st["v_codes"], st["v_scales"] = _random_slots(g, pages, hk, page, d, c["fmt"], None)
    # slots behind a sequence's end hold no number: memory that nothing has written
    slot = torch.arange(width * page, device=DEV)[None, :]
    live = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
    at = table.clamp(min=0).long()[:, slot[0] // page] * page + slot % page
    live.view(-1)[at[slot < st["lengths"][:, None]]] = True
    for name in ("k_scales", "v_scales"):
        st[name].masked_fill_(~live[:, None, :, None], 255)
    if c["fmt"] == "mx":
        st["k_scale"] = st["v_scale"] = None
    else:
        st["k_scale"] = (1.0 + 0.1 * torch.rand(hk, generator=g, device=DEV)) / 8.0
        st["v_scale"] = (1.0 + 0.1 * torch.rand(hk, generator=g, device=DEV)) / 8.0
    if c["op"] == "append":
        # as a product of queries, keys and values together gives them: one matrix, three parts of its columns
        qkv = _heads(g, (rows, hq + 2 * hk, d), dt)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        st["rope"] = None
        if c["rot"]:
            f = THETA ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
            a = torch.arange(width * page, device=DEV, dtype=torch.float64)[:, None] * f
            st["rope"] = torch.cat([a.cos(), a.sin()], dim=1).float()
    elif c["op"] == "attend":
        st["q"] = _heads(g, (rows, hq, d), dt)
    return st


# ------------------------------------------------------------------ the plain forms
def _pairs_table(dtype):
    v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device=DEV, dtype=dtype)
    b = torch.arange(256, device=DEV)
    return torch.stack((v[b & 15], v[b >> 4]), dim=1)


def _values(codes, scales, head_scale, fmt):
    """Values [..., heads, slots, dim] of codes [..., heads, slots, dim / 2]."""
    v = _pairs_table(torch.float32)[codes.int()].flatten(-2)
    if fmt == "mx":
        s = torch.ldexp(torch.ones((), device=DEV), scales.int() - 127)
    else:
        s = scales.view(torch.float8_e4m3fn).float()
    v = v.view(*scales.shape, -1)
    v = (v * s.unsqueeze(-1)).view(*codes.shape[:-1], -1)
    return v if head_scale is None else v * head_scale.view(-1, 1, 1)


def _places(st):
    """Sequence, position, page and slot of each row."""
    c, t = st["case"], torch.arange(st["rows"], device=DEV)
    if st["offsets"] is None:
        s, p = t, st["lengths"].long() - 1
    else:
        o = st["offsets"].long()
        s = torch.searchsorted(o[1:], t, right=True)
        p = st["lengths"].long()[s] - o[s + 1] + t
    return s, p, st["table"][s, (p // c["page"]).clamp(min=0)].long(), p % c["page"]


def _rotated(x, rope, p, rot, interleaved):
    x = x.float()
    if rope is None:
        return x
    cos, sin = rope[p].unsqueeze(1).split(rot // 2, dim=2)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _quantized(x, head_scale, fmt):
    """Codes and scale bytes of x [rows, heads, dim], nearest, ties to the even code."""
    per = 32 if fmt == "mx" else 16
    b = x.unflatten(2, (-1, per))
    top = b.abs().amax(dim=3)
    if fmt == "mx":
        e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(min=-127)
        y, sb = torch.ldexp(b, -e.unsqueeze(3)), (e + 127).to(torch.uint8)
    else:
        hs = head_scale.view(-1, 1)
        q = (top / (6.0 * hs)).clamp(max=448.0).to(torch.float8_e4m3fn)
        s, sb = q.float() * hs, q.view(torch.uint8)
        y = b * torch.where(s > 0, 1.0 / s, 0.0).unsqueeze(3)
    a = y.abs().clamp(max=6.0)
    # on the grid's three steps; round() takes ties to the even multiple, which is the even code
    r = torch.where(a < 2.0, torch.round(a * 2.0) * 0.5, torch.where(a < 4.0, torch.round(a), torch.round(a * 0.5) * 2.0))
    m = torch.bucketize(r, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV), out_int32=True)
    m = (m + 8 * torch.signbit(y)).to(torch.uint8).flatten(2)
    return m[..., 0::2] | (m[..., 1::2] << 4), sb


def _gather_plain(st):
    c = st["case"]
    _, _, page, slot = _places(st)
    out = {}
    for n in ("k", "v"):
        v = _values(st[n + "_codes"][page, :, slot].unsqueeze(2), st[n + "_scales"][page, :, slot].unsqueeze(2),
                    st[n + "_scale"], c["fmt"])
        out[n] = v.squeeze(2).to(DTYPES[c["dtype"]])
    return out


def _append_plain(st):
    c = st["case"]
    _, p, page, slot = _places(st)
    q = _rotated(st["q"], st["rope"], p, c["rot"], c["interleaved"]).to(st["q"].dtype)
    for n, x in (("k", _rotated(st["k"], st["rope"], p, c["rot"], c["interleaved"])), ("v", st["v"].float())):
        codes, scales = _quantized(x, st[n + "_scale"], c["fmt"])
        st[n + "_codes"][page, :, slot] = codes
        st[n + "_scales"][page, :, slot] = scales
    return {"q": q, **_gather_plain(st)}


def _attend_plain(st):
    c = st["case"]
    B, hk, d, n = c["seqs"], c["kv_heads"], c["dim"], c["new"]
    G, L = c["q_heads"] // hk, st["width"] * c["page"]
    s, p, _, _ = _places(st)
    i = torch.arange(st["rows"], device=DEV) - (0 if st["offsets"] is None else st["offsets"].long()[s])
    if st["offsets"] is None:
        i = torch.zeros_like(s)
    key = torch.arange(L, device=DEV)
    there = key < st["lengths"][:, None]

    def values(name):  # every sequence's slots in order: B, heads, L, dim; those behind its end are zero
        at = st["table"].clamp(min=0).long()
        v = _values(st[name + "_codes"][at], st[name + "_scales"][at], st[name + "_scale"], c["fmt"])
        return v.transpose(1, 2).reshape(B, hk, L, d).masked_fill(~there[:, None, :, None], 0.0)

    q = torch.zeros((B, n, hk, G, d), device=DEV)
    q[s, i] = st["q"].float().view(-1, hk, G, d)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, hk, n * G, d)
    score = torch.matmul(q, values("k").transpose(2, 3)) * d ** -0.5
    at = torch.full((B, n), -1, dtype=torch.long, device=DEV)
    at[s, i] = p
    seen = (key <= at[:, :, None]) & there[:, None, :]
    if c["window"]:
        seen &= key > at[:, :, None] - c["window"]
    score = score.view(B, hk, n, G, L).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(dim=4, keepdim=True)
    e = score.sub_(top.clamp(min=-1e30)).exp_()
    total = e.sum(dim=4, keepdim=True)
    o = torch.matmul(e.view(B, hk, n * G, L), values("v")).view(B, hk, n, G, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total)).squeeze(4)
    return {"o": o[s, :, i].reshape(-1, hk * G, d).to(st["q"].dtype), "lse": lse[s, :, i].reshape(-1, hk * G)}


# ------------------------------------------------------------------ the framework's calls
def _own(st):
    import bit_block_scaled_quantize_amd as nv

    c = st["case"]
    cache = nv.NVFP4KVCache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], st["k_scale"], st["v_scale"],
                            format=nv.NVFP4_KV_MXFP4 if c["fmt"] == "mx" else nv.NVFP4_KV_NVFP4)
    plan = (cache, st["table"], st["lengths"])
    if c["op"] == "attend":
        o, lse = nv.nvfp4_kv_attention(st["q"], *plan, offsets=st["offsets"], window=c["window"], lse=True)
        return {"o": o, "lse": lse}
    out = {}
    if c["op"] == "append":
        out["q"] = nv.nvfp4_kv_append(st["k"], st["v"], *plan, offsets=st["offsets"], q=st["q"], rope=st["rope"],
                                      interleaved=c["interleaved"])
    out["k"], out["v"] = nv.nvfp4_kv_gather(*plan, offsets=st["offsets"], rows=st["rows"], dtype=DTYPES[c["dtype"]])
    return out


PLAIN = {"append": _append_plain, "gather": _gather_plain, "attend": _attend_plain}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits
def _exact_slots(st, name, s):
    """Keys or values of sequence s: heads, length, dim."""
    c, l = st["case"], int(st["lengths"][s])
    at = st["table"][s, :-(-l // c["page"])].long()
    codes = torch.cat(list(st[name + "_codes"][at]), dim=1)[:, :l]
    sb = torch.cat(list(st[name + "_scales"][at]), dim=1)[:, :l].int()
    grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], device=DEV, dtype=torch.float64) / 2
    v = torch.empty((*codes.shape[:2], c["dim"]), dtype=torch.float64, device=DEV)
    for at, code in ((0, codes % 16), (1, codes // 16)):
        v[..., at::2] = grid[(code % 8).long()] * (1 - 2 * (code // 8).double())
    if c["fmt"] == "mx":
        return (v.unflatten(2, (-1, 32)) * (2.0 ** (sb.double() - 127))[..., None]).flatten(2)
    m = torch.where(sb >= 8, (8 + sb % 8).double() * 2.0 ** ((sb // 8).double() - 10), (sb % 8).double() * 2.0 ** -9)
    return (v.unflatten(2, (-1, 16)) * m[..., None]).flatten(2) * st[name + "_scale"].double()[:, None, None]


def _exact_rows(st):
    """(sequence, its first row, its rows, its first position) of each sequence."""
    first = 0
    for s in range(st["case"]["seqs"]):
        n = 1 if st["offsets"] is None else int(st["offsets"][s + 1] - st["offsets"][s])
        yield s, first, n, int(st["lengths"][s]) - n
        first += n


def _exact_grid(x, head_scale, fmt):
    """The values that x [rows, heads, dim] is held as."""
    per = 32 if fmt == "mx" else 16
    b = x.unflatten(2, (-1, per))
    top = b.abs().max(dim=3, keepdim=True).values
    if fmt == "mx":
        s = 2.0 ** torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - 2, -127.0).clamp(min=-127.0)
    else:
        u = (top / (6 * head_scale[:, None, None])).clamp(max=448.0)
        step = 2.0 ** (torch.floor(torch.log2(u.clamp(min=2.0 ** -6))) - 3)
        s = torch.round(u / step) * step * head_scale[:, None, None]
    y = torch.where(s > 0, b / s.clamp(min=1e-300), 0.0)
    step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=1.0))) - 1)
    return ((torch.round(y / step) * step).clamp(-6.0, 6.0) * s).flatten(2)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    hk, hq, d, rows = c["kv_heads"], c["q_heads"], c["dim"], st["rows"]
    if c["op"] == "gather":
        out = {}
        for name in ("k", "v"):
            out[name] = torch.cat([_exact_slots(st, name, s)[:, p:p + n].transpose(0, 1) for s, _, n, p in _exact_rows(st)])
        return out
    if c["op"] == "append":
        pos = torch.cat([torch.arange(p, p + n, device=DEV) for _, _, n, p in _exact_rows(st)])

        def rotate(x):
            x = x.double().clone()
            if c["rot"]:
                # the angles are an input, as the program keeps them; pairs as complex numbers
                r, h = st["rope"][pos].double(), c["rot"] // 2
                turn = torch.complex(r[:, :h], r[:, h:])[:, None, :]
                at = torch.arange(c["rot"], device=DEV).view(h, 2) if c["interleaved"] else torch.arange(c["rot"], device=DEV).view(2, h).t()
                z = torch.complex(x[..., at[:, 0]], x[..., at[:, 1]]) * turn
                x[..., at[:, 0]], x[..., at[:, 1]] = z.real, z.imag
            return x

        ks, vs = (None if st[n] is None else st[n].double() for n in ("k_scale", "v_scale"))
        return {"q": rotate(st["q"]), "k": _exact_grid(rotate(st["k"]), ks, c["fmt"]),
                "v": _exact_grid(st["v"].double(), vs, c["fmt"])}
    o = torch.zeros((rows, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=DEV)
    for s, first, n, p0 in _exact_rows(st):
        l = int(st["lengths"][s])
        if not l:
            continue
        k, v = _exact_slots(st, "k", s), _exact_slots(st, "v", s)
        for a in range(0, n, 512):
            m = min(512, n - a)
            pos = torch.arange(p0 + a, p0 + a + m, device=DEV)[:, None]
            key = torch.arange(l, device=DEV)[None, :]
            hidden = (key > pos) | (key <= pos - c["window"]) if c["window"] else key > pos
            for h in range(hq):
                kv = h // (hq // hk)
                x = torch.mm(st["q"][first + a:first + a + m, h].double(), k[kv].t().contiguous()) / math.sqrt(d)
                x.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(x, dim=1)
                lse[first + a:first + a + m, h] = z
                w = torch.exp(x - torch.where(z.isfinite(), z, 0.0)[:, None])
                o[first + a:first + a + m, h] = torch.mm(w, v[kv])
    return {"o": o, "lse": lse}
