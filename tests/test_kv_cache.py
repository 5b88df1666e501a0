"""The paged 4-bit key/value cache: refusals (no GPU), and what append stores
and gather reads, bit for bit against plain binary32 forms of the library's
rules (kv_plain.py), each operation rounded once."""
import ctypes

import pytest
import torch

import kv_plain as P

E = dict(OK=0, NULL=1, ENUM=2, SHAPE=3, ALIGN=4, UNSUP=5, WS=6)
DT = P.DT


@pytest.fixture(scope="module")
def nv():
    import bit_block_scaled_quantize_amd.nvfp4 as nv
    return nv


# ---------------------------------------------------------------- refusals (no GPU)
def _cache(nv, kc=65536, ks=65537, vc=65536, vs=65537, kf=65536, vf=65536, pages=8, size=32, heads=2, dim=128, fmt=0):
    return nv.CKVCache(kc, ks, vc, vs, kf, vf, pages, size, heads, dim, fmt)


def _plan(nv, table=65536, ld=4, width=4, lengths=65536, offsets=65536, seqs=3, rows=5):
    return nv.CKVPlan(table, ld, width, lengths, offsets, seqs, rows)


CACHE_FAULTS = [("NULL", dict(kc=None)), ("NULL", dict(ks=None)), ("NULL", dict(vc=None)), ("NULL", dict(vs=None)),
                ("NULL", dict(kf=None)), ("NULL", dict(vf=None)), ("ENUM", dict(fmt=2)), ("ENUM", dict(fmt=-1)),
                ("SHAPE", dict(pages=-1)), ("SHAPE", dict(size=0)), ("SHAPE", dict(heads=0)), ("SHAPE", dict(dim=0)),
                ("ALIGN", dict(kc=65544)), ("ALIGN", dict(vc=65537)), ("ALIGN", dict(kf=65538)),
                ("UNSUP", dict(dim=96)), ("UNSUP", dict(dim=512)), ("UNSUP", dict(size=8)), ("UNSUP", dict(size=48)),
                ("UNSUP", dict(pages=1 << 31)), ("UNSUP", dict(size=1 << 31))]
PLAN_FAULTS = [("NULL", dict(table=None)), ("NULL", dict(lengths=None)), ("SHAPE", dict(ld=3)), ("SHAPE", dict(rows=-1)),
               ("SHAPE", dict(seqs=-1)), ("SHAPE", dict(width=-1)), ("SHAPE", dict(offsets=None)),
               ("ALIGN", dict(table=65538)), ("ALIGN", dict(lengths=65537)), ("ALIGN", dict(offsets=65538)),
               ("UNSUP", dict(width=(1 << 25) + 1, ld=1 << 26)), ("UNSUP", dict(seqs=65537)),
               ("UNSUP", dict(rows=(1 << 30) + 1))]


def _rows(nv, data=65536, row=256, head=128):
    return nv.CKVRows(data, row, head)


def _calls(nv):
    """Each entry point on a cache and a plan, other arguments in order."""
    ref = ctypes.byref

    def append(c, p, k=None, v=None, dt=1, rope=None, q=None, hq=0, qo=None):
        k, v = k or _rows(nv), v or _rows(nv)
        return nv.lib.nvfp4_kv_append(ref(k), ref(v), dt, ref(c), ref(p), None if rope is None else ref(rope),
                                      None if q is None else ref(q), hq, None if qo is None else ref(qo), None)

    def gather(c, p, k=None, v=None, dt=1):
        k, v = k or _rows(nv), v or _rows(nv)
        return nv.lib.nvfp4_kv_gather(ref(c), ref(p), ref(k), ref(v), dt, None)

    def attention(c, p, q=None, out=None, dt=1, hq=4, window=0, lse=None, ws=65536, ws_bytes=1 << 40):
        q, out = q or _rows(nv, row=1024), out or _rows(nv, row=1024)
        return nv.lib.nvfp4_kv_attention(ref(q), dt, hq, ref(c), ref(p), 0.1, window, ref(out), lse, ws, ws_bytes, None)

    return append, gather, attention


@pytest.mark.parametrize("which", [0, 1, 2])
def test_cache_and_plan_are_checked(nv, which):
    call = _calls(nv)[which]
    for want, kw in CACHE_FAULTS:
        assert call(_cache(nv, **kw), _plan(nv)) == E[want], kw
    for want, kw in PLAN_FAULTS:
        assert call(_cache(nv), _plan(nv, **kw)) == E[want], kw
    assert call(_cache(nv), _plan(nv), dt=2) == E["ENUM"]
    # nothing to do
    empty = _plan(nv, seqs=0, rows=0, lengths=None, table=None)
    none = nv.CKVRows(None, 256, 128)
    assert call(_cache(nv), empty, none, none) == E["OK"]


def test_append_rejects_bad_arguments(nv):
    append = _calls(nv)[0]
    c, p = _cache(nv), _plan(nv)

    def rope(table=65536, positions=100, ld=128, dim=128):
        return nv.CKVRope(table, positions, ld, dim, 0)

    for want, kw in [("NULL", dict(k=_rows(nv, data=None))), ("NULL", dict(v=_rows(nv, data=None))),
                     ("SHAPE", dict(k=_rows(nv, row=-1))), ("SHAPE", dict(v=_rows(nv, head=-128))),
                     ("ALIGN", dict(k=_rows(nv, data=65537))), ("ALIGN", dict(dt=0, v=_rows(nv, data=65538))),
                     ("SHAPE", dict(q=_rows(nv), qo=_rows(nv), hq=0)), ("SHAPE", dict(hq=2)),
                     ("NULL", dict(q=_rows(nv), hq=2)), ("NULL", dict(q=_rows(nv, data=None), qo=_rows(nv), hq=2)),
                     ("SHAPE", dict(q=_rows(nv), qo=_rows(nv, head=64), hq=2)),
                     ("SHAPE", dict(q=_rows(nv), qo=_rows(nv, row=255), hq=2)),
                     ("NULL", dict(rope=rope(table=None))), ("SHAPE", dict(rope=rope(ld=127))),
                     ("SHAPE", dict(rope=rope(positions=-1))), ("SHAPE", dict(rope=rope(dim=0))),
                     ("ALIGN", dict(rope=rope(table=65538))), ("UNSUP", dict(rope=rope(dim=16))),
                     ("UNSUP", dict(rope=rope(dim=96))), ("UNSUP", dict(rope=rope(dim=256, ld=256)))]:
        assert append(c, p, **kw) == E[want], (want, kw)


def test_gather_and_attention_reject_bad_arguments(nv):
    _, gather, attention = _calls(nv)
    c, p = _cache(nv), _plan(nv)
    for want, kw in [("NULL", dict(k=_rows(nv, data=None))), ("SHAPE", dict(v=_rows(nv, row=128))),
                     ("SHAPE", dict(k=_rows(nv, row=0))), ("SHAPE", dict(k=_rows(nv, head=0))),
                     ("ALIGN", dict(v=_rows(nv, data=65537)))]:
        assert gather(c, p, **kw) == E[want], (want, kw)
    for want, kw in [("NULL", dict(q=_rows(nv, data=None))), ("NULL", dict(out=_rows(nv, data=None))),
                     ("SHAPE", dict(hq=3)), ("SHAPE", dict(hq=0)), ("SHAPE", dict(window=-1)),
                     ("SHAPE", dict(out=_rows(nv, row=511))), ("ALIGN", dict(out=_rows(nv, data=65537, row=1024))),
                     ("ALIGN", dict(lse=65538)), ("WS", dict(ws=None)), ("WS", dict(ws_bytes=1000)),
                     ("ALIGN", dict(ws=65544))]:
        assert attention(c, p, **kw) == E[want], (want, kw)
    assert attention(c, _plan(nv, rows=(1 << 26) + 1), hq=4, q=_rows(nv, row=0), out=_rows(nv, row=512)) == E["UNSUP"]
    size = nv.nvfp4_kv_attention_workspace_size
    assert size(5, 3, 4, 2, 128) > 0 and size(0, 3, 4, 2, 128) == 0
    assert size(5, 3, 3, 2, 128) == 0 and size(5, 3, 4, 2, 96) == 0 and size(-1, 3, 4, 2, 128) == 0
    assert size(5, -1, 4, 2, 128) == 0 and size(1 << 27, 3, 4, 2, 128) == 0


def test_the_binding_checks_shapes_and_types(nv):
    cache = nv.NVFP4KVCache.empty(4, 2, 64, page_size=16, device="cpu")
    table, lengths = torch.zeros((3, 2), dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    q, k = torch.zeros((3, 4, 64)), torch.zeros((3, 2, 64))
    with pytest.raises(ValueError, match="GPU"):
        nv.nvfp4_kv_attention(q, cache, table, lengths)
    for bad, what in [((q[:, :, :32], cache, table, lengths), "q is"), ((q[:2], cache, table, lengths), "one row a sequence"),
                      ((q, cache, table, lengths[:2]), "lengths"), ((q.transpose(1, 2), cache, table, lengths), "unit stride")]:
        with pytest.raises(ValueError, match=what):
            nv.nvfp4_kv_attention(*bad)
    for bad in [(q.half(), cache, table, lengths), (q, cache, table.long(), lengths), (q, cache, table, lengths.long())]:
        with pytest.raises(TypeError, match="dtype"):
            nv.nvfp4_kv_attention(*bad)
    with pytest.raises(TypeError, match="dtype"):
        nv.nvfp4_kv_append(k, k.bfloat16(), cache, table, lengths)
    with pytest.raises(ValueError, match="v is"):
        nv.nvfp4_kv_append(k, k[:, :1], cache, table, lengths)
    with pytest.raises(ValueError, match="offsets"):
        nv.nvfp4_kv_gather(cache, table, lengths, offsets=torch.zeros(3, dtype=torch.int32), rows=4)
    with pytest.raises(TypeError):
        nv.nvfp4_kv_gather(cache, table, lengths, dtype=torch.float16)
    wrong = nv.NVFP4KVCache(cache.k_codes, cache.k_scales[..., :2], cache.v_codes, cache.v_scales, cache.k_scale, cache.v_scale)
    with pytest.raises(ValueError, match="k_scales"):
        nv.nvfp4_kv_gather(wrong, table, lengths)


# ---------------------------------------------------------------- on the GPU
def make(nv, seqs, heads, dim, page, mx, seed=0, spare=3, width=None):
    """A cache whose slots all hold no number, and a table of pages in any order
    for sequences of up to the given lengths."""
    g = torch.Generator().manual_seed(seed)
    used = [-(-l // page) for l in seqs]
    pages = sum(used) + spare
    fmt = nv.NVFP4_KV_MXFP4 if mx else nv.NVFP4_KV_NVFP4
    cache = nv.NVFP4KVCache.empty(pages, heads, dim, page, fmt)
    for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales):
        t.fill_(255)
    if not mx:
        cache.k_scale.copy_(0.01 + torch.rand(heads, generator=g))
        cache.v_scale.copy_(0.01 + torch.rand(heads, generator=g))
    width = max(1, max(used)) if width is None else width
    table = torch.full((len(seqs), width), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
    return cache, table.cuda()


def heads_tensor(g, rows, heads, dim, dtype):
    x = torch.randn((rows, heads, dim), generator=g) * torch.exp2(torch.randint(-3, 4, (rows, heads, 1), generator=g))
    x[..., : dim // 2] *= (torch.rand((rows, heads, dim // 2), generator=g) > 0.2)  # zeros, whole blocks of them too
    if rows:
        x[0, 0, :32] = 0.0
    return x.to(dtype).cuda()


def rope_table(positions, dim):
    f = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    a = torch.arange(positions, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float().cuda()


def expected(cache, k, v, q, table, lengths, offsets, rope, inter, page):
    """The cache's arrays and q after the append (on clones, on the CPU)."""
    arrays = {n: getattr(cache, n).cpu().clone() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    qo = None if q is None else torch.zeros_like(q.cpu())
    hs = {n: None if getattr(cache, n) is None else getattr(cache, n).cpu() for n in ("k_scale", "v_scale")}
    table, rope = table.cpu(), None if rope is None else rope.cpu()
    for s, first, n, p0 in P.rows_of(lengths, offsets, k.shape[0]):
        for i in range(n):
            p, t = p0 + i, first + i
            if p < 0 or (rope is not None and p >= rope.shape[0]):
                continue
            at = torch.tensor([p])
            if q is not None:
                qo[t] = P.rotate(q[t:t + 1].cpu(), at, rope, inter)[0].to(q.dtype)
            pg = int(table[s, p // page])
            if not 0 <= pg < cache.k_codes.shape[0]:
                continue
            for name, x in (("k", P.rotate(k[t:t + 1].cpu(), at, rope, inter)), ("v", v[t:t + 1].cpu().float())):
                codes, byte = P.quantize(x, hs[name + "_scale"])
                arrays[name + "_codes"][pg, :, p % page] = codes[0]
                arrays[name + "_scales"][pg, :, p % page] = byte[0]
    return arrays, qo


def same(cache, arrays):
    for n, want in arrays.items():
        got = getattr(cache, n).cpu()
        assert torch.equal(got, want), (n, (got != want).nonzero()[:4].tolist())


# (lengths after the append, new rows or None: one each)
PLANS = [([1], None), ([5, 64, 0, 17, 33], None), ([40, 0, 7, 129], [13, 0, 7, 64]), ([70] * 70, [1] * 69 + [3])]
CASES = [(64, 0, False), (64, 32, False), (64, 64, True), (128, 128, False), (128, 32, True), (128, 64, False),
         (256, 256, False), (256, 128, True), (256, 32, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,rot,inter", CASES)
def test_append_stores_and_gather_reads(nv, dim, rot, inter, dtype, mx):
    for i, (lengths, new) in enumerate(PLANS):
        page, heads, hq = (16, 3, 5) if i % 2 else (32, 1, 4)
        print(f"append dim {dim} rot {rot} plan {i}", flush=True)
        offsets = None if new is None else [0, *torch.tensor(new).cumsum(0).tolist()]
        rows = len(lengths) if new is None else offsets[-1]
        cache, table = make(nv, lengths, heads, dim, page, mx, seed=i)
        g = torch.Generator().manual_seed(100 + i)
        k, v = (heads_tensor(g, rows, heads, dim, DT[dtype]) for _ in range(2))
        q = heads_tensor(g, rows, hq, dim, DT[dtype])
        rope = rope_table(max(lengths), rot) if rot else None
        want, qwant = expected(cache, k, v, q, table, lengths, offsets, rope, inter, page)
        L = torch.tensor(lengths, dtype=torch.int32).cuda()
        O = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
        got = nv.nvfp4_kv_append(k, v, cache, table, L, O, q=q, rope=rope, interleaved=inter)
        torch.cuda.synchronize()
        same(cache, want)
        assert torch.equal(got.cpu().view(torch.uint8), qwant.view(torch.uint8))
        for out_dtype in (torch.float32, torch.bfloat16):
            gk, gv = nv.nvfp4_kv_gather(cache, table, L, O, rows=rows, dtype=out_dtype)
            for name, x in (("k", gk), ("v", gv)):
                hs = getattr(cache, name + "_scale")
                wide = P.values(want[name + "_codes"], want[name + "_scales"], None if hs is None else hs.cpu())
                for s, first, n, p0 in P.rows_of(lengths, offsets, rows):
                    for j in range(n):
                        p = p0 + j
                        exp = wide[int(table[s, p // page]), :, p % page] if p >= 0 else torch.zeros((heads, dim))
                        # (one rounding to binary32, then one to bfloat16)
                        assert torch.equal(x[first + j].cpu(), exp.float().to(out_dtype)), (name, s, j)


@pytest.mark.gpu
def test_append_of_strided_rows_in_place(nv):
    """One matrix of q, k and v together, heads first, odd offsets; q rotated in place."""
    lengths, new, page, dim = [9, 30, 2], [5, 3, 2], 16, 128
    offsets, rows = [0, 5, 8, 10], 10
    g = torch.Generator().manual_seed(3)
    L, O = torch.tensor(lengths, dtype=torch.int32).cuda(), torch.tensor(offsets, dtype=torch.int32).cuda()
    rope = rope_table(64, 64)
    wide = torch.randn(64, 70, generator=g).cuda()
    wide[:, 3:67] = rope
    x = torch.randn((rows, 9 * dim + 7), generator=g).bfloat16().cuda()
    tall = torch.randn((9, rows, dim), generator=g).cuda()
    for name, (q, k, v) in {"columns": (x[:, 1:1 + 5 * dim].unflatten(1, (5, dim)),
                                        x[:, 1 + 5 * dim:1 + 7 * dim].unflatten(1, (2, dim)),
                                        x[:, 1 + 7 * dim:1 + 9 * dim].unflatten(1, (2, dim))),
                            "heads first": (tall[:5].transpose(0, 1), tall[5:7].transpose(0, 1), tall[7:].transpose(0, 1)),
                            "one head for all": (tall[:5].transpose(0, 1), tall[5:6].transpose(0, 1).expand(-1, 2, -1),
                                                 tall[7:].transpose(0, 1))}.items():
        print(name, flush=True)
        cache, table = make(nv, lengths, 2, dim, page, False)
        before = k.clone(), v.clone()
        want, qwant = expected(cache, k, v, q, table, lengths, offsets, rope, False, page)
        out = nv.nvfp4_kv_append(k, v, cache, table, L, O, q=q, rope=wide[:, 3:67], out=q)
        torch.cuda.synchronize()
        assert out.data_ptr() == q.data_ptr()
        same(cache, want)
        assert torch.equal(q.cpu(), qwant) and torch.equal(k, before[0]) and torch.equal(v, before[1])
        # read back into the other half of a wider tensor
        both = torch.full((rows, 4, dim), 7.0).cuda()
        gk, gv = nv.nvfp4_kv_gather(cache, table, L, O, rows=rows, out=(both[:, 0::2], both[:, 1::2]))
        k2, v2 = nv.nvfp4_kv_gather(cache, table, L, O, rows=rows, dtype=torch.float32)
        assert torch.equal(both[:, 0::2], k2) and torch.equal(both[:, 1::2], v2)


@pytest.mark.gpu
@pytest.mark.parametrize("mx", [False, True])
def test_rows_without_a_place(nv, mx):
    """Pages that are none, positions before the first and past the angles,
    lengths past the table, rows before the first and behind the last sequence."""
    page, dim, rows = 16, 64, 20
    lengths = [40, 3, 64, 25]  # of 3 pages: 48 at most
    offsets = [2, 7, 12, 16, 18]
    cache, table = make(nv, [48, 48, 48, 48], 2, dim, page, mx)
    table[0, 2] = -1
    table[3, 1] = cache.k_codes.shape[0]
    g = torch.Generator().manual_seed(5)
    k, v = (heads_tensor(g, rows, 2, dim, torch.bfloat16) for _ in range(2))
    q = heads_tensor(g, rows, 3, dim, torch.bfloat16)
    rope = rope_table(47, 32)
    L, O = torch.tensor(lengths, dtype=torch.int32).cuda(), torch.tensor(offsets, dtype=torch.int32).cuda()
    want, qwant = expected(cache, k, v, q, table, [40, 3, 48, 25], offsets, rope, False, page)
    out = torch.full_like(q, 5.0)
    nv.nvfp4_kv_append(k, v, cache, table, L, O, q=q, rope=rope, out=out)
    torch.cuda.synchronize()
    same(cache, want)
    qwant[:2] = 5.0
    qwant[18:] = 5.0
    assert torch.equal(out.cpu(), qwant)
    assert bool((out[7:9] == 0).all()) and bool((out[15] == 0).all())  # before the first; past the angles
    pair = (torch.full((rows, 2, dim), 5.0).cuda(), torch.full((rows, 2, dim), 5.0).cuda())
    nv.nvfp4_kv_gather(cache, table, L, O, rows=rows, out=pair)
    for x in pair:
        assert bool((x[:2] == 5.0).all()) and bool((x[18:] == 5.0).all())
        assert bool((x[7:9] == 0).all()) and bool((x[2 + 0:7] == 0).all())  # sequence 0's rows: positions 35 to 39, no page
        assert bool((x[16:18] == 0).all())


@pytest.mark.gpu
def test_offsets_out_of_order_stay_in_bounds(nv):
    cache, table = make(nv, [30, 30, 30], 2, 64, 16, False)
    k = torch.ones((6, 2, 64)).cuda()
    L = torch.tensor([30, -4, 1 << 30], dtype=torch.int32).cuda()
    for offsets in ([0, 9, 2, 6], [-5, 3, 100, 2], [4, 2, 1, 0]):
        O = torch.tensor(offsets, dtype=torch.int32).cuda()
        nv.nvfp4_kv_append(k, k, cache, table, L, O)
        nv.nvfp4_kv_gather(cache, table, L, O, rows=6)
        nv.nvfp4_kv_attention(k, cache, table, L, O)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_blocks_at_the_ends_of_the_scales(nv):
    """Block maxima past the largest E4M3 scale saturate, tiny ones become zero
    (NVFP4) or the smallest scale (MXFP4), as the quantize operators have it."""
    for mx in (False, True):
        cache, table = make(nv, [16], 1, 128, 16, mx)
        if not mx:
            cache.k_scale.fill_(1.0)
            cache.v_scale.fill_(2.0 ** -140)  # (a subnormal tensor scale)
        x = torch.randn((6, 1, 128), generator=torch.Generator().manual_seed(1))
        x = x * torch.tensor([1e30, 1e4, 1.0, 1e-3, 1e-30, 1e-42]).view(6, 1, 1)
        x = x.cuda()
        L, O = torch.tensor([6], dtype=torch.int32).cuda(), torch.tensor([0, 6], dtype=torch.int32).cuda()
        want, _ = expected(cache, x, x if mx else x * 0.0, None, table, [6], [0, 6], None, False, 16)
        nv.nvfp4_kv_append(x, x if mx else x * 0.0, cache, table, L, O)
        torch.cuda.synchronize()
        same(cache, want)


@pytest.mark.gpu
def test_no_sequences_and_no_pages(nv):
    """Rows of no sequence are left alone; without a page nothing is stored or seen."""
    k = torch.ones((5, 2, 64)).cuda()
    q = torch.ones((5, 4, 64)).cuda().bfloat16()
    cache, _ = make(nv, [16], 2, 64, 16, False)
    none = torch.zeros((0, 3), dtype=torch.int32).cuda(), torch.zeros(0, dtype=torch.int32).cuda()
    O = torch.zeros(1, dtype=torch.int32).cuda()
    out = torch.full_like(k, 3.0)
    nv.nvfp4_kv_append(k, k, cache, *none, O, q=k[:, :1], out=out[:, :1])
    nv.nvfp4_kv_gather(cache, *none, O, rows=5, out=(out, out))
    o = nv.nvfp4_kv_attention(k, cache, *none, O, out=out)
    assert bool((o == 3.0).all())
    empty = nv.NVFP4KVCache.empty(0, 2, 64, 16)
    table = torch.zeros((2, 3), dtype=torch.int32).cuda()
    for rows, offsets in ((5, [0, 2, 5]), (100, [0, 70, 100])):
        L, O = torch.tensor([40, 48], dtype=torch.int32).cuda(), torch.tensor(offsets, dtype=torch.int32).cuda()
        kk, qq = torch.ones((rows, 2, 64)).cuda(), torch.ones((rows, 4, 64)).cuda().bfloat16()
        nv.nvfp4_kv_append(kk, kk, empty, table, L, O)
        assert not bool(nv.nvfp4_kv_gather(empty, table, L, O, rows=rows)[0].any())
        o, lse = nv.nvfp4_kv_attention(qq, empty, table, L, O, lse=True)
        assert not bool(o.any()) and bool(torch.isinf(lse).all())


@pytest.mark.parametrize("which", [0, 1, 2])
def test_rows_of_no_sequence_launch_nothing(nv, which):
    assert _calls(nv)[which](_cache(nv), _plan(nv, seqs=0, rows=5, lengths=None, table=None)) == E["OK"]


@pytest.mark.gpu
def test_rows_of_no_sequence_are_not_read(nv):
    """A call whose rows are all but padding takes no time for them: reading their 1.3 GB
    alone takes 43% of what appending them does."""
    rows, dim, page = 65536, 128, 64
    cache, table = make(nv, [rows], 8, dim, page, False)
    k, v = (torch.randn((rows, 8, dim), device="cuda") for _ in range(2))
    q = torch.randn((rows, 24, dim), device="cuda")
    out = torch.empty_like(q)

    def least(lengths, offsets):
        L, O = torch.tensor(lengths, dtype=torch.int32).cuda(), torch.tensor(offsets, dtype=torch.int32).cuda()
        times = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            nv.nvfp4_kv_append(k, v, cache, table, L, O, q=q, out=out)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    whole = least([rows], [0, rows])
    for offsets in ([0, 16], [rows - 16, rows], [rows // 2, rows // 2]):
        part = least([rows], offsets)
        assert part < 0.3 * whole, (offsets, part, whole)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_beside_rows_of_a_wave(nv, dtype):
    """Many rows, a few to a wave, of which some belong to no sequence: what they hold
    reaches nothing."""
    rows, dim, page, lengths = 20000, 64, 64, [9000, 9500]
    offsets = [700, 9003, 18001]
    cache, table = make(nv, lengths, 8, dim, page, False)
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v, q = (torch.randn((rows, h, dim), generator=g, device="cuda").to(DT[dtype]) for h in (8, 8, 16))
    L, O = torch.tensor(lengths, dtype=torch.int32).cuda(), torch.tensor(offsets, dtype=torch.int32).cuda()
    rope = rope_table(9500, 64)
    own = slice(offsets[0], offsets[-1])
    nv.nvfp4_kv_append(k[own], v[own], cache, table, L, O - offsets[0], q=q[own], rope=rope, out=(want := q[own].clone()))
    arrays = {n: getattr(cache, n).cpu() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    for n in arrays:
        getattr(cache, n).fill_(255)
    for x in (k, v, q):
        x[:offsets[0]] = float("nan")
        x[offsets[-1]:] = float("inf")
    out = torch.full_like(q, 5.0)
    nv.nvfp4_kv_append(k, v, cache, table, L, O, q=q, rope=rope, out=out)
    same(cache, arrays)
    assert torch.equal(out[own], want) and bool((out[:offsets[0]] == 5).all()) and bool((out[offsets[-1]:] == 5).all())
    pair = tuple(torch.full((rows, 8, dim), 5.0, device="cuda") for _ in range(2))
    nv.nvfp4_kv_gather(cache, table, L, O, rows=rows, out=pair)
    ref = nv.nvfp4_kv_gather(cache, table, L, O - offsets[0], rows=offsets[-1] - offsets[0], dtype=torch.float32)
    for x, y in zip(pair, ref):
        assert torch.equal(x[own], y) and bool((x[:offsets[0]] == 5).all()) and bool((x[offsets[-1]:] == 5).all())


def test_gather_by_offsets_needs_its_rows(nv):
    """Their number lies on the device: taken as one a sequence, other rows would come back."""
    cache = nv.NVFP4KVCache.empty(4, 2, 64, page_size=16, device="cpu")
    table, lengths = torch.zeros((3, 2), dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    offsets = torch.tensor([0, 4, 5, 9], dtype=torch.int32)
    with pytest.raises(ValueError, match="rows"):
        nv.nvfp4_kv_gather(cache, table, lengths, offsets)
    pair = torch.zeros((9, 2, 64)), torch.zeros((9, 2, 64))
    for args in (dict(rows=9), dict(out=pair), dict(rows=9, out=pair)):  # (as far as the tensors' device)
        with pytest.raises(ValueError, match="GPU"):
            nv.nvfp4_kv_gather(cache, table, lengths, offsets, **args)


@pytest.mark.gpu
def test_gather_by_offsets_into_given_rows(nv):
    lengths, offsets = [30, 7], [0, 20, 27]
    cache, table = make(nv, lengths, 2, 64, 16, False)
    k, v = torch.randn((27, 2, 64)).cuda(), torch.randn((27, 2, 64)).cuda()
    L, O = torch.tensor(lengths, dtype=torch.int32).cuda(), torch.tensor(offsets, dtype=torch.int32).cuda()
    nv.nvfp4_kv_append(k, v, cache, table, L, O)
    pair = torch.empty_like(k), torch.empty_like(v)
    nv.nvfp4_kv_gather(cache, table, L, O, out=pair)
    assert all(torch.equal(x, y) for x, y in zip(pair, nv.nvfp4_kv_gather(cache, table, L, O, rows=27, dtype=torch.float32)))


# (row stride, head stride) of 5 rows of 2 heads of 128 (attention: 4 heads), apart or not
APART = [(256, 128), (384, 256), (128, 640), (256, 1152), (1 << 62, 128), (128, 1 << 62)]
TOGETHER = [(255, 128), (383, 256), (256, 127), (128, 639), (256, 1151), (127, 1 << 62), (1 << 62, 127), (0, 128), (128, 0)]


def test_heads_written_to_are_refused_only_where_they_overlap(nv):
    """(A misaligned address comes after the strides: nothing is launched.)"""
    append, gather, attention = _calls(nv)
    c, p = _cache(nv), _plan(nv)
    for strides, want in [(x, "ALIGN") for x in APART] + [(x, "SHAPE") for x in TOGETHER]:
        out = _rows(nv, 65537, *strides)
        assert gather(c, p, k=out) == E[want] and gather(c, p, v=out) == E[want], strides
        assert append(c, p, q=_rows(nv), hq=2, qo=out) == E[want], strides
        assert attention(c, p, q=_rows(nv), hq=2, out=out) == E[want], strides
    one = _plan(nv, seqs=1, rows=1, offsets=None)
    for strides, want in (((0, 128), "ALIGN"), ((0, 1 << 62), "ALIGN"), ((0, 127), "SHAPE")):
        assert gather(c, one, k=_rows(nv, 65537, *strides)) == E[want], strides
    single = _cache(nv, heads=1)
    for strides, want in (((128, 0), "ALIGN"), ((127, 0), "SHAPE"), ((127, 1 << 62), "SHAPE")):
        assert gather(single, p, k=_rows(nv, 65537, *strides)) == E[want], strides


@pytest.mark.gpu
def test_results_into_every_second_head(nv):
    """Heads 0 and 2 of a tensor of three: the last row ends where the tensor does."""
    lengths, offsets, rows, dim = [30, 7], [0, 20, 27], 27, 64
    cache, table = make(nv, lengths, 2, dim, 16, False)
    g = torch.Generator().manual_seed(7)
    k, v, q = (torch.randn((rows, 2, dim), generator=g).cuda() for _ in range(3))
    L, O = torch.tensor(lengths, dtype=torch.int32).cuda(), torch.tensor(offsets, dtype=torch.int32).cuda()
    rope = rope_table(30, dim)
    wide = [torch.full((rows, 3, dim), 7.0, device="cuda") for _ in range(4)]
    turned = nv.nvfp4_kv_append(k, v, cache, table, L, O, q=q, rope=rope)
    nv.nvfp4_kv_append(k, v, cache, table, L, O, q=q, rope=rope, out=wide[0][:, ::2])
    nv.nvfp4_kv_attention(q, cache, table, L, O, out=wide[1][:, ::2])
    nv.nvfp4_kv_gather(cache, table, L, O, out=(wide[2][:, ::2], wide[3][:, ::2]))
    want = [turned, nv.nvfp4_kv_attention(q, cache, table, L, O),
            *nv.nvfp4_kv_gather(cache, table, L, O, rows=rows, dtype=torch.float32)]
    for x, y in zip(wide, want):
        # (bits: the first sequence's first ten slots hold no numbers)
        assert torch.equal(x[:, ::2].contiguous().view(torch.int32), y.view(torch.int32)) and bool((x[:, 1] == 7.0).all())
