"""Attention over the paged 4-bit cache at the ends of its number formats: values,
scores and head scales far from 1, elements that were not finite when they were
appended.  Against the 64-bit form of kv_plain.py, which derives the bounds, or
against what must hold whatever the sums' order."""
import math

import numpy as np
import pytest
import torch

import kv_plain as P
from test_kv_cache import make

pytestmark = pytest.mark.gpu
DT = P.DT
#: (dim, type of q, new rows of each sequence or None: one): the kernel of few columns, and (BF16, over 64 columns) of many
FORMS = [(64, "f32", None), (128, "bf16", None), (256, "bf16", None), (128, "f32", [3, 1, 70]),
         (64, "bf16", [40, 1, 100]), (128, "bf16", [33, 1, 70]), (256, "bf16", [40, 1, 70])]
LENGTHS = [40, 1, 2500]


@pytest.fixture(scope="module")
def nv():
    import bit_block_scaled_quantize_amd.nvfp4 as nv
    return nv


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def held(nv, lengths, k, v, page, mx, k_scale=0.01, v_scale=0.01):
    """A cache with k and v (binary32, the sequences' rows one after the other) in it."""
    rows, heads, dim = k.shape
    cache, table = make(nv, lengths, heads, dim, page, mx)
    if not mx:
        cache.k_scale.fill_(k_scale)
        cache.v_scale.fill_(v_scale)
    nv.nvfp4_kv_append(k, v, cache, table, ints(lengths), ints([0, *np.cumsum(lengths).tolist()]))
    return cache, table


def normal(seed, *sizes):
    return torch.randn(sizes, generator=torch.Generator().manual_seed(seed)).cuda()


def attend_and_check(nv, lengths, new, q, cache, table, page, mx, dtype, scale, window=0):
    offsets = None if new is None else [0, *np.cumsum(new).tolist()]
    o, lse = nv.nvfp4_kv_attention(q, cache, table, ints(lengths), None if new is None else ints(offsets), scale=scale,
                                   window=window, lse=True)
    torch.cuda.synchronize()
    want = P.attention(q, cache, table, lengths, offsets, scale, window, cache.k_codes.shape[0], page)
    P.check(o, lse, want, dtype, mx)
    return o, lse


def rows_of(new):
    return len(LENGTHS) if new is None else sum(new)


# ---------------------------------------------------------------- values of MXFP4
@pytest.mark.parametrize("e", [-90, 0, 100, 118, 125])
@pytest.mark.parametrize("dim,dtype,new", FORMS)
def test_values_of_any_size_over_mxfp4(nv, dim, dtype, new, e):
    """Values from 2^e to 6 x 2^e, of either sign and all of one: a mean is no larger than
    its largest value, so nothing overflows."""
    n = sum(LENGTHS)
    k = normal(1, n, 2, dim)
    v = (1.0 + 4.9 * torch.rand((n, 2, dim), generator=torch.Generator().manual_seed(2))).cuda()
    v[:, 0] *= torch.sign(normal(3, n, dim))
    v = torch.ldexp(v, torch.tensor(e))
    cache, table = held(nv, LENGTHS, k, v, 32, True)
    q = normal(4, rows_of(new), 6, dim).to(DT[dtype])
    for window in (0, 300):
        attend_and_check(nv, LENGTHS, new, q, cache, table, 32, True, dtype, dim ** -0.5, window)


@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("f32", 1), ("bf16", 70)])
def test_many_equal_values_at_mxfp4s_largest(nv, dtype, rows):
    """40000 keys of weight 1 whose values are 6 x 2^125: so is their mean."""
    n, dim = 40000, 64
    v = torch.full((n, 1, dim), 1.5 * 2.0 ** 127, device="cuda")
    cache, table = held(nv, [n], torch.zeros_like(v), v, 256, True)
    q = torch.ones((rows, 1, dim), device="cuda").to(DT[dtype])
    o, lse = nv.nvfp4_kv_attention(q, cache, table, ints([n]), ints([0, rows]), lse=True)
    off = (o.double() / (1.5 * 2.0 ** 127) - 1.0).abs().max().item()
    # (weights of one, sums 1e-5, rounding)
    assert off <= 1e-5 + torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -17, off
    want = torch.log(torch.arange(n - rows + 1, n + 1, dtype=torch.float64)).view(-1, 1).cuda()
    assert (lse.double() - want).abs().max().item() <= 2e-5 * math.log(n)


# ---------------------------------------------------------------- scores
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("e", [20, 22, 24, 25, 26, 27, 28, 30, 40, 100])
@pytest.mark.parametrize("dim,dtype,new", FORMS)
def test_scores_of_any_size(nv, dim, dtype, new, e, mx):
    n = sum(LENGTHS)
    cache, table = held(nv, LENGTHS, normal(5, n, 2, dim), normal(6, n, 2, dim), 32, mx)
    q = normal(7, rows_of(new), 6, dim).to(DT[dtype])
    attend_and_check(nv, LENGTHS, new, q, cache, table, 32, mx, dtype, dim ** -0.5 * 2.0 ** e)


def steps(nv, n, dim, mx, v, t):
    """Keys whose products with q = (2^14, 2^-6, 0 ...) are 6 x 2^14 + 2^-6 t: neighbouring
    binary32 numbers for neighbouring t."""
    k = torch.zeros((n, 1, dim), device="cuda")
    k[:, 0, 0] = 6.0
    k[:, 0, 1] = t
    cache, table = held(nv, [n], k, v, 64, mx, k_scale=1.0, v_scale=0.01)
    got = nv.nvfp4_kv_gather(cache, table, ints([n]), ints([0, n]), rows=n, dtype=torch.float32)
    assert torch.equal(got[0], k)
    return cache, table, got[1].double()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("most", [2.0 ** 21, 1.2 * 2.0 ** 25, 1.5 * 2.0 ** 26, 1.5 * 2.0 ** 27, 1.9 * 2.0 ** 29, 2.0 ** 60])
@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("f32", 1), ("bf16", 70)])
def test_a_maximum_that_grows_by_a_unit_in_the_last_place(nv, dtype, rows, most, mx):
    """Scores (in powers of two) of `most` that rise along the sequence by steps of the last
    bit.  Values of one: whatever the weights, their mean is one; its weights add up to at
    least that of the last key and at most that of all keys at the last score."""
    n, dim = 500, 64
    t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")[torch.arange(n, device="cuda") // 64]
    cache, table, v = steps(nv, n, dim, mx, torch.ones((n, 1, dim), device="cuda"), t)
    q = torch.zeros((rows, 1, dim), device="cuda")
    q[..., 0] = 2.0 ** 14
    q[..., 1] = 2.0 ** -6
    scale = most / (6 * 2.0 ** 14) * math.log(2.0)
    o, lse = nv.nvfp4_kv_attention(q.to(DT[dtype]), cache, table, ints([n]), ints([0, rows]), scale=scale, lse=True)
    off = (o.double() / v[0, 0] - 1.0).abs().max().item()
    assert off <= P.HALF_STEP[dtype, mx] + 1e-5 + torch.finfo(DT[dtype]).eps / 2, off
    # 2^-24 each: the scale in binary32, log2(e), their product, the sum of products, the score's product, the sum with
    # the weights' logarithm, log(2), its product
    top = scale * (6 * 2.0 ** 14 + 2.0 ** -6 * 6)
    tol = 8 * 2.0 ** -24 * top + 1e-4
    assert bool((lse.double() >= top - tol).all()) and bool((lse.double() <= top + math.log(n) + tol).all())


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("most", [2.0 ** 21, 1.2 * 2.0 ** 25, 1.5 * 2.0 ** 27, 2.0 ** 60])
@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("f32", 1), ("bf16", 70)])
def test_equal_scores_of_any_size_give_the_mean(nv, dtype, rows, most, mx):
    n, dim = 500, 64
    cache, table, v = steps(nv, n, dim, mx, normal(8, n, 1, dim), 3.0)
    q = torch.zeros((rows, 1, dim), device="cuda")
    q[..., 0] = 2.0 ** 14
    scale = -most / (6 * 2.0 ** 14) if rows == 1 else most / (6 * 2.0 ** 14)
    o = nv.nvfp4_kv_attention(q.to(DT[dtype]), cache, table, ints([n]), ints([0, rows]), scale=scale)
    for r in range(rows):
        seen = v[:n - rows + 1 + r, 0]
        want, size = seen.mean(dim=0), seen.abs().mean(dim=0)
        tol = (P.HALF_STEP[dtype, mx] + 1e-5) * size + torch.finfo(DT[dtype]).eps / 2 * want.abs()
        assert bool(((o[r, 0].double() - want).abs() <= 1.01 * tol).all()), r


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("most", [2.0 ** 18, 1.2 * 2.0 ** 25, 1.5 * 2.0 ** 27, 1.9 * 2.0 ** 28, 2.0 ** 60])
@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("f32", 1), ("bf16", 70)])
def test_scores_far_below_others_leave_nothing(nv, dtype, rows, most, mx):
    """300 keys at -most, 130 at 0, 70 at -most: the mean of the 130."""
    n, dim = 500, 64
    k = torch.zeros((n, 1, dim), device="cuda")
    k[:, 0, 0] = -6.0
    k[300:430] = 0.0
    cache, table = held(nv, [n], k, normal(22, n, 1, dim), 64, mx, k_scale=1.0)
    v = nv.nvfp4_kv_gather(cache, table, ints([n]), ints([0, n]), rows=n, dtype=torch.float32)[1].double()
    q = torch.zeros((rows, 1, dim), device="cuda")
    q[..., 0] = 2.0 ** 14
    o = nv.nvfp4_kv_attention(q.to(DT[dtype]), cache, table, ints([n]), ints([0, rows]), scale=most / (6 * 2.0 ** 14))
    want, size = v[300:430, 0].mean(dim=0), v[300:430, 0].abs().mean(dim=0)
    tol = (P.HALF_STEP[dtype, mx] + 1e-5) * size + torch.finfo(DT[dtype]).eps / 2 * want.abs()
    assert bool(((o[:, 0].double() - want).abs() <= 1.01 * tol).all())


# ---------------------------------------------------------------- head scales of values
@pytest.mark.parametrize("e", [-124, -110, -60, 60, 114])
@pytest.mark.parametrize("dim,dtype,new", FORMS)
def test_value_scales_of_any_size(nv, dim, dtype, new, e):
    n = sum(LENGTHS)
    v = torch.ldexp(normal(9, n, 2, dim).clamp(-5, 5) * 400.0, torch.tensor(e))
    cache, table = held(nv, LENGTHS, normal(10, n, 2, dim), v, 32, False, v_scale=2.0 ** e)
    q = normal(11, rows_of(new), 6, dim).to(DT[dtype])
    attend_and_check(nv, LENGTHS, new, q, cache, table, 32, False, dtype, dim ** -0.5)


@pytest.mark.parametrize("dtype,rows", [("bf16", 1), ("f32", 1), ("bf16", 70)])
def test_the_mean_of_many_small_values(nv, dtype, rows):
    """65536 equal keys: their weights' sum is far above the value scale's reciprocal."""
    n, dim = 65536, 64
    v = torch.full((n, 1, dim), 2688 * 2.0 ** -124, device="cuda")
    cache, table = held(nv, [n], torch.zeros_like(v), v, 256, False, v_scale=2.0 ** -124)
    q = torch.ones((rows, 1, dim), device="cuda").to(DT[dtype])
    o = nv.nvfp4_kv_attention(q, cache, table, ints([n]), ints([0, rows]))
    off = (o.double() / (2688 * 2.0 ** -124) - 1.0).abs().max().item()
    assert off <= 1e-5 + torch.finfo(DT[dtype]).eps / 2, off


# ---------------------------------------------------------------- head scales of keys
@pytest.mark.parametrize("large", [False, True])
@pytest.mark.parametrize("dim,dtype,new", FORMS)
def test_key_scales_of_any_size(nv, dim, dtype, new, large):
    """Scores of ordinary size where the scale times the key scale alone leaves binary32's
    normal numbers (small keys, large rows of q) or its range (the other way round)."""
    n, rows = sum(LENGTHS), rows_of(new)
    g = torch.Generator().manual_seed(12)
    if large:
        e, scale = 118, 2.0 ** 11
        k = torch.ldexp(normal(13, n, 2, dim), torch.tensor(118))
        q = torch.ldexp(normal(14, rows, 6, dim), torch.tensor(-127))
    else:
        e, scale = -124, 8.0 / (dim * 0.5625 * 2600 * 8)
        k, q = (0.5 + 0.5 * torch.rand(size, generator=g).cuda() for size in ((n, 2, dim), (rows, 6, dim)))
        k, q = k * 2600 * 2.0 ** -124, torch.ldexp(q, torch.tensor(127))
    cache, table = held(nv, LENGTHS, k, normal(15, n, 2, dim), 32, False, k_scale=2.0 ** e)
    attend_and_check(nv, LENGTHS, new, q.to(DT[dtype]), cache, table, 32, False, dtype, scale)


# ---------------------------------------------------------------- what was not finite
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dim,dtype,rows", [(128, "bf16", 120), (64, "f32", 120), (256, "bf16", 120), (128, "bf16", 12)])
def test_appended_values_that_are_not_finite(nv, dim, dtype, rows, mx):
    """They are unspecified; rows that do not see them have their results, bit for bit."""
    n, bad = 120, 113
    k, v, q = normal(16, n, 2, dim), normal(17, n, 2, dim), normal(18, rows, 8, dim).to(DT[dtype])
    L, O = ints([n]), ints([0, rows])
    got = []
    for x in (1.0, math.inf, -math.inf, math.nan):
        v[bad, :, 3] = x
        v[bad, 1, :] = x
        cache, table = held(nv, [n], k, v, 32, mx)
        rest = torch.ones(n, dtype=torch.bool)
        rest[bad] = False
        read = nv.nvfp4_kv_gather(cache, table, L, ints([0, n]), rows=n, dtype=torch.float32)[1]
        assert bool(read.isfinite().all())
        got.append((read[rest], nv.nvfp4_kv_attention(q, cache, table, L, O)[:bad - n],
                    nv.nvfp4_kv_attention(q, cache, table, L, O, window=3)[-3:]))
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))
    assert all(bool(x.isfinite().all()) for x in got[0])


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dim,dtype,rows", [(128, "bf16", 120), (64, "f32", 120), (256, "bf16", 120), (128, "bf16", 12)])
def test_appended_keys_that_are_not_finite(nv, dim, dtype, rows, mx):
    """Rows that do not see them have their results to the bounds."""
    n, bad = 120, 113
    k, v, q = normal(19, n, 2, dim), normal(20, n, 2, dim), normal(21, rows, 8, dim).to(DT[dtype])
    clean, table = held(nv, [n], k, v, 32, mx)
    want = P.attention(q, clean, table, [n], [0, rows], dim ** -0.5, 0, clean.k_codes.shape[0], 32)
    for x in (math.inf, -math.inf, math.nan):
        k[bad, :, 3] = x
        k[bad, 1, :] = x
        cache, table = held(nv, [n], k, v, 32, mx)
        o, lse = nv.nvfp4_kv_attention(q, cache, table, ints([n]), ints([0, rows]), lse=True)
        P.check(o, lse, want, dtype, mx, rows=slice(0, rows + bad - n))
