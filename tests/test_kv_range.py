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
    P.check_attention(o, lse, want, dtype, mx)
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
