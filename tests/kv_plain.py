"""Plain forms of the paged 4-bit key/value cache: its values, what an append
stores (binary32, one rounding at a time) and attention in 64 bits, by
sequence, with the bounds of its rounding errors."""
import math

import torch

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def unpack(codes):
    return torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)


def values(codes, scales, head_scale):
    """binary64 values of [..., heads, slots, dim / 2] codes (head_scale None: MX)."""
    v = E2M1.to(codes.device)[unpack(codes).long()]
    if head_scale is None:
        s = torch.ldexp(torch.ones((), dtype=torch.float64, device=codes.device), scales.int() - 127)
    else:
        s = scales.view(torch.float8_e4m3fn).double() * head_scale.double().view(-1, 1, 1)
    return (v.unflatten(-1, (scales.shape[-1], -1)) * s.unsqueeze(-1)).flatten(-2)


def rotate(x, pos, rope, interleaved):
    """binary32: [rows, heads, dim] turned by the angles of pos."""
    x = x.float().clone()
    if rope is None:
        return x
    r = rope.shape[1]
    cos, sin = rope[pos, None, :r // 2], rope[pos, None, r // 2:]
    ia = torch.arange(0, r, 2) if interleaved else torch.arange(r // 2)
    ib = ia + 1 if interleaved else ia + r // 2
    a, b = x[..., ia], x[..., ib]
    x[..., ia], x[..., ib] = a * cos - b * sin, b * cos + a * sin
    return x


def quantize(x, head_scale):
    """(codes, scale bytes) of binary32 x [rows, heads, dim] by the library's rules."""
    per = 32 if head_scale is None else 16
    b = x.unflatten(-1, (-1, per))
    top = b.abs().amax(dim=-1)
    if head_scale is None:
        e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(min=-127)
        byte, y = (e + 127).to(torch.uint8), torch.ldexp(b, -e.unsqueeze(-1))
    else:
        hs = head_scale.view(-1, 1)
        q = (top / (6.0 * hs)).clamp(max=448.0).to(torch.float8_e4m3fn)
        S = q.float() * hs
        byte, y = q.view(torch.uint8), b * torch.where(S > 0, 1.0 / S, 0.0).unsqueeze(-1)
    y = y.flatten(-2)
    a = y.abs().double()
    grid = E2M1[:8].to(x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    code = torch.searchsorted(mid, a)  # a tie goes down, and up where the lower code is odd
    tie = (a == mid[code.clamp(max=6)]) & (code < 7) & (code % 2 == 1)
    code = code + tie
    code = (code + 8 * torch.signbit(y)).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte


def rows_of(lengths, offsets, rows):
    """(sequence, first row, rows, first position) of each sequence."""
    for s, l in enumerate(lengths):
        first, n = (s, 1) if offsets is None else (offsets[s], offsets[s + 1] - offsets[s])
        yield s, first, n, l - n


def attention(q, cache, table, lengths, offsets, scale, window, pages, page_size):
    """(out, lse, sum w |v| / sum w, relative error of a weight, what FP16 weights lose), binary64.  The bounds are
    of what binary32 sums and roundings of scores and weights do, without the
    weights' and the output's own rounding; per row and head:
      score    1e-5 sum |q k| scale (accumulation) + 2^-21 |score| (its products)
      weight   that, twice (itself and the sum), + 2^-20 (exponential)
      sum      1e-5 sum w |v| / sum w."""
    dev = q.device
    rows, hq, d = q.shape
    hk = cache.k_codes.shape[1]
    group = hq // hk
    out = torch.zeros((rows, hq, d), dtype=torch.float64, device=dev)
    lse = torch.full((rows, hq), -math.inf, dtype=torch.float64, device=dev)
    mean_abs, lost = torch.zeros_like(out), torch.zeros((rows, hq, 1), dtype=torch.float64, device=dev)
    eps = torch.zeros((rows, hq, 1), dtype=torch.float64, device=dev)
    for s, first, n, p0 in rows_of(lengths, offsets, rows):
        l = lengths[s]
        if n == 0 or l == 0:
            continue
        at = table[s, :-(-l // page_size)].long()
        there = ((at >= 0) & (at < pages)).repeat_interleave(page_size)[:l]
        at = torch.where((at >= 0) & (at < pages), at, 0)

        def held(codes, scales, hs):
            v = values(codes[at], scales[at], hs).transpose(0, 1).reshape(hk, -1, d)[:, :l]
            return torch.where(there[None, :, None], v, 0.0)

        k = held(cache.k_codes, cache.k_scales, cache.k_scale)
        v = held(cache.v_codes, cache.v_scales, cache.v_scale)
        pos = torch.arange(p0, p0 + n, device=dev)[:, None]
        key = torch.arange(l, device=dev)[None, :]
        seen = (key <= pos) & there[None, :]
        if window:
            seen &= key > pos - window
        for h in range(hq):
            x = q[first:first + n, h].double()
            score = (x @ k[h // group].t().contiguous()) * scale
            size = (x.abs() @ k[h // group].abs().t().contiguous()) * abs(scale)
            e = torch.where(seen, 1e-5 * size + 2.0 ** -21 * score.abs(), 0.0).amax(dim=1)
            score = torch.where(seen, score, -math.inf)
            z = torch.logsumexp(score, dim=1)
            w = torch.exp(score - torch.where(z.isfinite(), z, 0.0)[:, None])
            out[first:first + n, h] = w @ v[h // group]
            mean_abs[first:first + n, h] = w @ v[h // group].abs()
            lse[first:first + n, h] = z
            eps[first:first + n, h, 0] = e
            lost[first:first + n, h, 0] = 2.0 ** -36 * seen.sum(dim=1) * v[h // group].abs().max()
    weight = 2.0 * eps + 2.0 ** -19
    return out, lse, mean_abs, weight, lost


#: relative error of a weight as it goes into the second product (half a step of each part)
WEIGHT = {("bf16", False): 2.0 ** -12, ("bf16", True): 2.0 ** -17, ("f32", False): 2.0 ** -22, ("f32", True): 2.0 ** -24}


def check_attention(got, got_lse, want, dtype, mx, rows=None):
    out, lse, mean_abs, weight, lost = want
    half = torch.finfo(DT[dtype]).eps / 2
    # FP16 weights are taken times 2^11 over a maximum that is at most the row's own: below 2^-14 a rounding is off by up to
    # 2^-25, which is 2^-36 of the largest weight or less, so of the result by up to 2^-36 max |v| for each key: `lost`.  It
    # counts where the keys of the large weights hold zeros, as E2M1 values often are.
    tol = (weight + WEIGHT[dtype, mx] + 1e-5) * mean_abs + half * out.abs() + (0.0 if mx else 1.0) * lost + 1e-37
    tol = tol * (1.0 + 2.0 ** -7)
    keep = slice(None) if rows is None else rows
    off = (got.double() - out).abs()[keep]
    assert bool((off <= tol[keep]).all()), (off / tol[keep]).max().item()
    if got_lse is not None:
        empty = torch.isinf(lse)
        assert torch.equal(torch.isinf(got_lse)[keep], empty[keep])
        lim = weight.squeeze(2) + 2.0 ** -21 * torch.where(empty, 0.0, lse).abs()
        d = torch.where(empty, 0.0, got_lse.double() - lse).abs()
        assert bool((d <= lim)[keep].all()), (d / lim)[keep].max().item()


#: As WEIGHT, with the whole half step of FP16: of 11 significant bits, a weight in [2^k, 2^(k + 1)) is rounded by up to
#: 2^(k - 11), which is 2^-11 of it at the lower end.  (Two parts: the first leaves up to 2^(k - 11), the second's half step
#: is then 2^(k - 23); BF16's 8 bits leave 2^(k - 8), then 2^(k - 17).)
HALF_STEP = {**WEIGHT, ("bf16", False): 2.0 ** -11}


def check(got, got_lse, want, dtype, mx, rows=None):
    """check_attention with weights off by HALF_STEP in the results (the sums are of unrounded ones)."""
    out, lse, mean_abs, weight, lost = want
    more = HALF_STEP[dtype, mx] - WEIGHT[dtype, mx]
    check_attention(got, None, (out, lse, mean_abs, weight + more, lost), dtype, mx, rows)
    if got_lse is not None:
        check_attention(out, got_lse, want, dtype, mx, rows)
