"""Attention over the paged 4-bit cache against its 64-bit form (kv_plain.py,
which derives the bounds)."""
import math

import pytest
import torch

import kv_plain as P
from test_kv_cache import make

pytestmark = pytest.mark.gpu
DT = P.DT


@pytest.fixture(scope="module")
def nv():
    import bit_block_scaled_quantize_amd.nvfp4 as nv
    return nv


def fill(nv, cache, table, lengths, seed):
    """Appends normal keys and values to every position."""
    heads, dim = cache.k_codes.shape[1], 2 * cache.k_codes.shape[3]
    rows = sum(lengths)
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn((rows, heads, dim), generator=g, device="cuda") for _ in range(2))
    k[..., 5] *= 6.0
    if cache.k_scale is not None:
        cache.k_scale.mul_(0.01)
        cache.v_scale.mul_(0.01)
    offsets = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32).cuda()
    nv.nvfp4_kv_append(k, v, cache, table, torch.tensor(lengths, dtype=torch.int32).cuda(), offsets)


def case(nv, lengths, new, heads, group, dim, page, mx, dtype, seed=0, scale=None):
    cache, table = make(nv, lengths, heads, dim, page, mx, seed=seed)
    fill(nv, cache, table, lengths, seed)
    offsets = None if new is None else [0, *torch.tensor(new).cumsum(0).tolist()]
    rows = len(lengths) if new is None else offsets[-1]
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn((rows, heads * group, dim), generator=g, device="cuda")
    q *= torch.exp2(torch.randint(-4, 2, (rows, heads * group, 1), generator=g, device="cuda").float())
    L = torch.tensor(lengths, dtype=torch.int32).cuda()
    O = None if new is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    return cache, table, L, O, offsets, q.to(DT[dtype])


def run_and_check(nv, lengths, new, heads, group, dim, page, mx, dtype, window=0, seed=0, scale=None):
    print(f"attention {lengths[:6]} new {new and new[:6]} {heads}x{group} dim {dim} page {page} mx {mx} {dtype} window {window}",
          flush=True)
    cache, table, L, O, offsets, q = case(nv, lengths, new, heads, group, dim, page, mx, dtype, seed)
    o, lse = nv.nvfp4_kv_attention(q, cache, table, L, O, scale=scale, window=window, lse=True)
    torch.cuda.synchronize()
    want = P.attention(q, cache, table, lengths, offsets, dim ** -0.5 if scale is None else scale, window,
                       cache.k_codes.shape[0], page)
    P.check_attention(o, lse, want, dtype, mx)
    return cache, table, L, O, q, o, lse


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_single_tokens(nv, dim, dtype, mx):
    run_and_check(nv, [1], None, 1, 1, dim, 16, mx, dtype)
    run_and_check(nv, [0, 1, 15, 16, 17, 63, 64, 65, 300], None, 2, 5, dim, 16, mx, dtype, seed=1)
    run_and_check(nv, [2049, 5], None, 1, 16, dim, 128, mx, dtype, seed=2)
    run_and_check(nv, [777, 0, 1500], None, 3, 7, dim, 32, mx, dtype, window=100, seed=3)
    run_and_check(nv, [100, 200], None, 2, 20, dim, 64, mx, dtype, seed=4)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_of_a_sequence(nv, dim, dtype, mx):
    run_and_check(nv, [5, 70, 33], [5, 3, 0], 2, 3, dim, 16, mx, dtype)
    run_and_check(nv, [300, 129, 64], [129, 129, 64], 1, 4, dim, 64, mx, dtype, seed=1)
    run_and_check(nv, [500, 40], [77, 40], 2, 5, dim, 32, mx, dtype, window=33, seed=2)
    run_and_check(nv, [3, 10], [8, 2], 1, 2, dim, 16, mx, dtype, seed=3)  # five rows before the first position
    run_and_check(nv, [900], [400], 1, 8, dim, 128, mx, dtype, window=1, seed=4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(nv, dtype):
    """Chunks of prompts: several blocks of rows, ragged, behind cached beginnings."""
    run_and_check(nv, [1500, 700, 64, 1], [600, 700, 1, 1], 2, 4, 128, 64, False, dtype, seed=5)
    run_and_check(nv, [1100], [1030], 1, 5, 64, 16, True, dtype, window=500, seed=6)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_blocks_of_many_columns(nv, dim, mx):
    """Sequences of over 64 columns beside ones of few, whole and split by keys."""
    run_and_check(nv, [65, 10, 700, 33], [65, 1, 300, 0], 2, 3, dim, 16, mx, "bf16", seed=20)
    run_and_check(nv, [40, 1000], [50, 17], 1, 8, dim, 32, mx, "bf16", seed=21)  # ten rows before the first position
    run_and_check(nv, [2100, 900], [257, 128], 1, 4, dim, 64, mx, "bf16", window=200, seed=22)
    run_and_check(nv, [300], [100], 1, 5, dim, 64, mx, "bf16", scale=-0.7, seed=23)
    run_and_check(nv, [300], [100], 1, 5, dim, 64, mx, "bf16", scale=0.0, seed=24)
    run_and_check(nv, [500, 20], None, 1, 70, dim, 64, mx, "bf16", seed=25)  # one row of 70 heads to a kv head
    new = [1 + (13 * i) % 30 for i in range(40)]
    run_and_check(nv, [n + (97 * i) % 250 for i, n in enumerate(new)], new, 8, 6, dim, 16, mx, "bf16", seed=26)


def test_holes_under_many_rows(nv):
    cache, table, L, O, offsets, q = case(nv, [400, 200], [150, 100], 2, 4, 128, 16, False, "bf16", seed=27)
    table[0, 3] = -1
    table[0, 20] = cache.k_codes.shape[0]
    table[1, :] = -5
    for window in (0, 40):
        o, lse = nv.nvfp4_kv_attention(q, cache, table, L, O, lse=True, window=window)
        want = P.attention(q, cache, table, [400, 200], offsets, 128 ** -0.5, window, cache.k_codes.shape[0], 16)
        P.check_attention(o, lse, want, "bf16", False)
        assert bool((o[150:] == 0).all()) and bool(torch.isinf(lse[150:]).all())


@pytest.mark.parametrize("seqs", [65, 200, 301, 700, 1030])
def test_many_sequences(nv, seqs):
    lengths = [(37 * i * i + 11 * i) % 90 for i in range(seqs)]
    run_and_check(nv, lengths, None, 2, 2, 64, 16, False, "bf16", seed=7)
    run_and_check(nv, lengths, None, 2, 5, 128, 16, seqs % 2 == 0, "f32", seed=7)
    if seqs < 1000:
        new = [min(l, (5 * i) % 4) for i, l in enumerate(lengths)]
        run_and_check(nv, lengths, new, 1, 3, 64, 16, True, "f32", seed=8)
    # with one longer sequence among them
    lengths[seqs // 2] = 2500
    run_and_check(nv, lengths, None, 2, 2, 64, 16, False, "bf16", seed=9, window=seqs % 2 * 1000)


def test_scales_and_large_scores(nv):
    run_and_check(nv, [400, 90], None, 2, 4, 128, 32, False, "bf16", scale=1.5, seed=1)
    run_and_check(nv, [400, 90], None, 2, 4, 128, 32, True, "f32", scale=-0.3, seed=2)
    run_and_check(nv, [400, 90], None, 2, 4, 128, 32, False, "f32", scale=0.0, seed=3)
    # rows of q from 2^-100 to 2^100 (the scale brings the scores back)
    for e in (-100, 100):
        cache, table, L, O, offsets, q = case(nv, [200, 31], None, 2, 4, 128, 32, False, "f32", seed=4)
        q = q * 2.0 ** e
        scale = 128 ** -0.5 * 2.0 ** -e
        o, lse = nv.nvfp4_kv_attention(q, cache, table, L, scale=scale, lse=True)
        P.check_attention(o, lse, P.attention(q, cache, table, [200, 31], None, scale, 0, cache.k_codes.shape[0], 32), "f32", False)


def test_equal_keys_give_the_mean(nv):
    """A long sequence of equal scores: every weight counts alike, also where one
    key outweighs each of them."""
    n, dim = 40000, 64
    cache, table = make(nv, [n], 1, dim, 256, False)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    k = torch.zeros((n, 1, dim), device="cuda")
    k[17] = 1.0
    v = torch.ones((n, 1, dim), device="cuda")
    v[17] = -1.0
    L = torch.tensor([n], dtype=torch.int32).cuda()
    nv.nvfp4_kv_append(k, v, cache, table, L, torch.tensor([0, n], dtype=torch.int32).cuda())
    for c in (0.0, 8.0, 15.0):
        q = torch.full((1, 1, dim), c / dim, device="cuda")
        o, lse = nv.nvfp4_kv_attention(q.bfloat16(), cache, table, L, scale=1.0, lse=True)
        held = 6 * 0.171875  # of a block of ones: the E4M3 value nearest 1 / 6, and the code of 6
        s = float(q.bfloat16().double().sum()) * held
        total = n - 1 + math.exp(s)
        want = (n - 1 - math.exp(s)) / total * held
        # weights as FP16 (each by 2^-12 of itself, all equal ones alike), sums 1e-5, bf16 output
        assert (o.double() - want).abs().max().item() <= (2.0 ** -12 + 2e-5) + 2.0 ** -8 * abs(want), (c, o[0, 0, 0].item(), want)
        assert abs(lse.item() - math.log(total)) <= 1e-5 * (1 + math.log(total))


def test_pages_that_are_none_are_not_seen(nv):
    cache, table, L, O, offsets, q = case(nv, [200, 100, 60], None, 2, 4, 128, 16, False, "bf16", seed=9)
    table[0, 3] = -1
    table[0, 12] = cache.k_codes.shape[0] + 7
    table[1, :] = -5
    o, lse = nv.nvfp4_kv_attention(q, cache, table, L, lse=True)
    want = P.attention(q, cache, table, [200, 100, 60], None, 128 ** -0.5, 0, cache.k_codes.shape[0], 16)
    P.check_attention(o, lse, want, "bf16", False)
    assert bool((o[1] == 0).all()) and bool(torch.isinf(lse[1]).all())


def test_other_rows_are_left_alone(nv):
    lengths, rows = [50, 80, 30], 12
    cache, table, L, _, _, _ = case(nv, lengths, None, 2, 4, 64, 16, False, "bf16", seed=10)
    offsets = [2, 5, 5, 9]
    O = torch.tensor(offsets, dtype=torch.int32).cuda()
    q = torch.randn((rows, 8, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q[:2] = float("nan")
    q[9:] = float("nan")
    out, lse = torch.full_like(q, 3.0), torch.full((rows, 8), 3.0).cuda()
    nv.nvfp4_kv_attention(q, cache, table, L, O, lse=True, out=out, out_lse=lse)
    for x in (out, lse):
        assert bool((x[:2] == 3).all()) and bool((x[9:] == 3).all())
    want = P.attention(q.nan_to_num(), cache, table, lengths, offsets, 64 ** -0.5, 0, cache.k_codes.shape[0], 16)
    P.check_attention(out, lse, want, "bf16", False, rows=slice(2, 9))


def test_strides_and_results_in_place(nv):
    lengths, new = [90, 33], [20, 4]
    cache, table, L, O, offsets, q = case(nv, lengths, new, 2, 4, 128, 16, False, "bf16", seed=11)
    ref, lse = nv.nvfp4_kv_attention(q, cache, table, L, O, lse=True)
    first = q.transpose(0, 1).contiguous().transpose(0, 1)  # heads first
    assert torch.equal(nv.nvfp4_kv_attention(first, cache, table, L, O), ref)
    wide = torch.full((24, 8 * 128 + 9), 2.0, device="cuda").bfloat16()
    inner = wide[:, 3:3 + 8 * 128].unflatten(1, (8, 128))
    inner.copy_(q)
    got = nv.nvfp4_kv_attention(inner, cache, table, L, O, out=inner)
    assert got.data_ptr() == inner.data_ptr() and torch.equal(inner, ref)
    assert bool((wide[:, :3] == 2).all()) and bool((wide[:, -6:] == 2).all())
    heads_first = torch.empty((8, 24, 128), device="cuda").bfloat16()
    nv.nvfp4_kv_attention(q, cache, table, L, O, out=heads_first.transpose(0, 1))
    assert torch.equal(heads_first.transpose(0, 1), ref)
    again, lse2 = nv.nvfp4_kv_attention(q, cache, table, L, O, lse=True)
    assert torch.equal(again, ref) and torch.equal(lse, lse2)
    # a table with more places than pages, and rows of it apart
    longer = torch.full((2, 40), -1, dtype=torch.int32).cuda()
    longer[:, 5:5 + table.shape[1]] = table
    assert torch.equal(nv.nvfp4_kv_attention(q, cache, longer[:, 5:], L, O), ref)


def test_heads_of_the_tensor_scale(nv):
    """Per-head scales far apart."""
    cache, table, L, O, offsets, q = case(nv, [120, 55], None, 3, 2, 64, 16, False, "f32", seed=12)
    for t, f in ((cache.k_scale, [1.0, 8.0, 0.001]), (cache.v_scale, [1e20, 1e-20, 3.0])):
        t.copy_(torch.tensor(f))
    o, lse = nv.nvfp4_kv_attention(q, cache, table, L, scale=0.001, lse=True)
    want = P.attention(q, cache, table, [120, 55], None, 0.001, 0, cache.k_codes.shape[0], 16)
    P.check_attention(o, lse, want, "f32", False)


def test_another_stream_and_a_given_workspace(nv):
    cache, table, L, O, offsets, q = case(nv, [3000, 70], None, 2, 4, 128, 64, False, "bf16", seed=13)
    ref = nv.nvfp4_kv_attention(q, cache, table, L)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = torch.empty(nv.nvfp4_kv_attention_workspace_size(2, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    ws.fill_(255)
    torch.cuda.synchronize()
    got = [nv.nvfp4_kv_attention(q, cache, table, L, stream=side, workspace=ws) for _ in range(3)]
    own = nv.nvfp4_kv_attention(q, cache, table, L, stream=side)
    side.synchronize()
    assert all(torch.equal(x, ref) for x in got) and torch.equal(own, ref)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_kv_attention(q, cache, table, L, workspace=ws[:1024])


def test_a_captured_step_follows_its_inputs(nv):
    """Append and attention of one token a sequence in a graph, replayed while
    lengths grow, against the same calls made eagerly."""
    page, dim, heads, group, steps = 16, 128, 2, 4, 40
    start = [30, 1, 100]
    most = [l + steps for l in start]
    caches = []
    for _ in range(2):
        cache, table = make(nv, most, heads, dim, page, False, seed=14)
        fill(nv, cache, table, start, 14)
        caches.append((cache, table))
    g = torch.Generator(device="cuda").manual_seed(15)
    f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    a = torch.arange(max(most), dtype=torch.float64)[:, None] * f
    rope = torch.cat([a.cos(), a.sin()], dim=1).float().cuda()
    q, k, v = (torch.zeros((3, h, dim), device="cuda").bfloat16() for h in (heads * group, heads, heads))
    L = torch.tensor(start, dtype=torch.int32).cuda() + 1
    ws = torch.empty(nv.nvfp4_kv_attention_workspace_size(3, 3, heads * group, heads, dim), dtype=torch.uint8, device="cuda")

    def step(cache, table, workspace=None):
        r = nv.nvfp4_kv_append(k, v, cache, table, L, q=q, rope=rope)
        return nv.nvfp4_kv_attention(r, cache, table, L, lse=True, workspace=workspace)

    step(*caches[0], ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*caches[0], ws)
    for i in range(steps):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        L.copy_(torch.tensor([l + i + 1 for l in start], dtype=torch.int32))
        graph.replay()
        ref = step(*caches[1])
        torch.cuda.synchronize()
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1]), i
    for n in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert torch.equal(getattr(caches[0][0], n), getattr(caches[1][0], n))
    lengths = [l + steps for l in start]
    r = nv.nvfp4_kv_append(k, v, *caches[1], L, q=q, rope=rope)
    want = P.attention(r, *caches[1], lengths, None, dim ** -0.5, 0, caches[1][0].k_codes.shape[0], page)
    P.check_attention(ref[0], ref[1], want, "bf16", False)


def test_one_token_at_a_time_equals_a_prefill(nv):
    """Tokens appended and attended one by one, and all at once: the cache bit for
    bit, the results to the bounds of each."""
    page, dim, heads, group, n = 16, 64, 2, 3, 50
    cache, table = make(nv, [n], heads, dim, page, True, seed=16)
    other = nv.NVFP4KVCache(*[t.clone() for t in cache.args()[:4]], format=nv.NVFP4_KV_MXFP4)
    g = torch.Generator(device="cuda").manual_seed(17)
    q, k, v = (torch.randn((n, h, dim), generator=g, device="cuda") for h in (heads * group, heads, heads))
    one = []
    for t in range(n):
        L = torch.tensor([t + 1], dtype=torch.int32).cuda()
        nv.nvfp4_kv_append(k[t:t + 1], v[t:t + 1], cache, table, L)
        one.append(nv.nvfp4_kv_attention(q[t:t + 1], cache, table, L))
    L, O = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([n], [0, n]))
    nv.nvfp4_kv_append(k, v, other, table, L, O)
    for a, b in zip(cache.args()[:4], other.args()[:4]):
        assert torch.equal(a, b)
    want = P.attention(q, cache, table, [n], [0, n], dim ** -0.5, 0, cache.k_codes.shape[0], page)
    P.check_attention(torch.cat(one), None, want, "f32", True)
    P.check_attention(nv.nvfp4_kv_attention(q, other, table, L, O), None, want, "f32", True)


def test_a_cache_past_32_bits(nv):
    """Pages whose codes lie past 2^32 bytes."""
    heads, dim, page = 8, 128, 64
    pages = (1 << 32) // (heads * page * dim // 2) + 40
    cache = nv.NVFP4KVCache.empty(pages, heads, dim, page, k_scale=0.01, v_scale=0.01)
    small, stable = make(nv, [300, 129], heads, dim, page, False, seed=18)
    fill(nv, small, stable, [300, 129], 18)
    cache.k_scale.copy_(small.k_scale)
    cache.v_scale.copy_(small.v_scale)
    table = torch.where(stable >= 0, pages - 1 - stable, -1).to(torch.int32)
    L, O = torch.tensor([300, 129], dtype=torch.int32).cuda(), torch.tensor([0, 300, 429], dtype=torch.int32).cuda()
    k, v = nv.nvfp4_kv_gather(small, stable, L, O, rows=429, dtype=torch.float32)
    nv.nvfp4_kv_append(k, v, cache, table, L, O)
    k2, v2 = nv.nvfp4_kv_gather(cache, table, L, O, rows=429, dtype=torch.float32)
    assert bool((k2 - k).abs().max() <= 0.26 * k.abs().max()) and bool(k2.any())
    q = torch.randn((2, heads * 4, dim), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    o, lse = nv.nvfp4_kv_attention(q, cache, table, L, lse=True)
    low = nv.NVFP4KVCache(*[t[pages - small.k_codes.shape[0]:].clone() for t in cache.args()[:4]], cache.k_scale, cache.v_scale)
    base = torch.where(table >= 0, table - (pages - small.k_codes.shape[0]), -1).to(torch.int32)
    o2, lse2 = nv.nvfp4_kv_attention(q, low, base, L, lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_lengths_past_the_table(nv):
    """A length past what the table's row holds counts as that, a negative one as 0."""
    cache, table, _, _, _, q = case(nv, [160, 96, 50], None, 2, 4, 128, 16, False, "bf16", seed=28)
    table[1, 6:] = -1
    L = torch.tensor([100000, 96, -7], dtype=torch.int32).cuda()
    o, lse = nv.nvfp4_kv_attention(q, cache, table, L, lse=True)
    want = P.attention(q, cache, table, [160, 96, 0], None, 128 ** -0.5, 0, cache.k_codes.shape[0], 16)
    P.check_attention(o, lse, want, "bf16", False)
    offsets = [0, 90, 100, 103]
    O = torch.tensor(offsets, dtype=torch.int32).cuda()
    many = torch.randn((103, 8, 128), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    o, lse = nv.nvfp4_kv_attention(many, cache, table, L, O, lse=True)
    want = P.attention(many, cache, table, [160, 96, 0], offsets, 128 ** -0.5, 0, cache.k_codes.shape[0], 16)
    P.check_attention(o, lse, want, "bf16", False)


@pytest.mark.parametrize("dim,mx", [(64, True), (128, False), (256, False), (256, True)])
def test_captured_chunks(nv, dim, mx):
    """Chunks of prompts of changing lengths in a graph, replayed with eager work between."""
    page, heads, group, rows = 32, 2, 4, 150
    cache, table = make(nv, [400, 300], heads, dim, page, mx, seed=29)
    fill(nv, cache, table, [400, 300], 29)
    g = torch.Generator(device="cuda").manual_seed(30)
    q = torch.zeros((rows, heads * group, dim), device="cuda").bfloat16()
    L = torch.tensor([400, 300], dtype=torch.int32).cuda()
    O = torch.tensor([0, 100, 150], dtype=torch.int32).cuda()
    ws = torch.empty(nv.nvfp4_kv_attention_workspace_size(rows, 2, heads * group, heads, dim), dtype=torch.uint8, device="cuda")
    nv.nvfp4_kv_attention(q, cache, table, L, O, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.nvfp4_kv_attention(q, cache, table, L, O, workspace=ws)
    for lengths, offsets in (([400, 300], [0, 100, 150]), ([150, 10], [0, 140, 150]), ([399, 1], [0, 149, 150]),
                             ([64, 300], [0, 3, 150])):
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        L.copy_(torch.tensor(lengths, dtype=torch.int32))
        O.copy_(torch.tensor(offsets, dtype=torch.int32))
        graph.replay()
        ref = nv.nvfp4_kv_attention(q, cache, table, L, O)
        torch.cuda.synchronize()
        assert torch.equal(out, ref), (lengths, offsets)


def test_two_calls_at_once(nv):
    """Two streams, each with its own workspace, on one cache."""
    cache, table, L, O, offsets, q = case(nv, [5000, 700], [1, 1], 2, 4, 128, 64, False, "bf16", seed=31)
    many = torch.randn((200, 8, 128), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    OM = torch.tensor([0, 120, 200], dtype=torch.int32).cuda()
    ref = nv.nvfp4_kv_attention(q, cache, table, L, O), nv.nvfp4_kv_attention(many, cache, table, L, OM)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append((nv.nvfp4_kv_attention(q, cache, table, L, O, stream=a), nv.nvfp4_kv_attention(many, cache, table, L, OM, stream=b)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, ref[0]) and torch.equal(y, ref[1])


def test_a_row_that_is_not_finite(nv):
    """It is unspecified; the others are theirs."""
    for lengths, offsets in (([300, 64], [0, 4, 9]), ([300, 200], [0, 100, 150])):
        cache, table = make(nv, lengths, 2, 128, 16, False, seed=32)
        fill(nv, cache, table, lengths, 32)
        L, O = torch.tensor(lengths, dtype=torch.int32).cuda(), torch.tensor(offsets, dtype=torch.int32).cuda()
        q = torch.randn((offsets[-1], 8, 128), generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
        ref = nv.nvfp4_kv_attention(q, cache, table, L, O)
        bad = q.clone()
        bad[1, 2, 5] = float("inf")
        bad[3, 4] = float("nan")
        got = nv.nvfp4_kv_attention(bad, cache, table, L, O)
        keep = torch.ones(q.shape[:2], dtype=torch.bool)
        keep[1, 2] = keep[3, 4] = False
        # (a block's rescaling may come earlier for its other columns: the last bits)
        off = (got.double() - ref.double()).abs()[keep]
        assert bool((off <= 2.0 ** -7 * ref.double().abs()[keep] + 1e-4).all())


@pytest.mark.parametrize("page", [16, 1024, 4096])
def test_page_sizes(nv, page):
    run_and_check(nv, [1500, 17, 4096], None, 2, 4, 128, page, False, "bf16", seed=33)
    run_and_check(nv, [1500, 60], [130, 60], 2, 4, 128, page, True, "bf16", seed=34)


@pytest.mark.parametrize("dim,mx", [(64, False), (128, True), (256, False)])
def test_parts_of_chunks(nv, dim, mx):
    """Blocks whose keys are split beside ones that are not, and one row more or less
    than a part's least."""
    run_and_check(nv, [2100, 300, 1023, 1024, 1025, 2047, 2048, 2049], [70, 300, 40, 40, 40, 33, 33, 33], 1, 4, dim, 64, mx,
                  "bf16", seed=35)
    run_and_check(nv, [4000, 65], [65, 65], 2, 2, dim, 32, mx, "bf16", window=1500, seed=36)
