"""Expert routing, its dispatch plan and its backward pass against the plain
64-bit forms of moe_plain.py.

The chosen experts and the plan are compared for equality.  Weights: an
exponential within 2 steps of binary32 (4 U, U = 2^-24 half a step), sums of
up to 16 chosen scores (5 roundings over the lanes) on both sides of a
division: 16 U; the softmax over all experts sums up to 32 scores a lane and
6 times over lanes: 48 U more."""
import numpy as np
import pytest
import torch

import moe_plain as P

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def test_plain_backward_against_differences():
    g = np.random.default_rng(0)
    l, ds, v = g.standard_normal((4, 11)), g.standard_normal((4, 11)), g.standard_normal((4, 11))
    t = 1e-5
    for sigmoid in (False, True):
        for renorm in (False, True):
            ids, _ = P.route(l, 3, sigmoid=sigmoid)
            dw = g.standard_normal(ids.shape)

            def loss(a):
                p = P.scores(a, sigmoid)
                w = np.take_along_axis(p, ids, axis=1)
                w = w / w.sum(axis=1, keepdims=True) if renorm else w
                return (w * dw).sum() + (p * ds).sum()

            got = (P.route_backward(dw, l, ids, sigmoid, renorm, ds) * v).sum()
            assert abs((loss(l + t * v) - loss(l - t * v)) / (2 * t) - got) < 1e-7


# ---------------------------------------------------------------- refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    import bit_block_scaled_quantize_amd.nvfp4 as nv
    return nv


E = dict(OK=0, NULL=1, ENUM=2, SHAPE=3, ALIGN=4, UNSUP=5, WS=6)


def test_route_rejects_bad_arguments(lib):
    import ctypes

    def call(l=65536, dt=0, T=100, n=64, ld=64, k=4, score=0, groups=1, top_groups=1, gs=1, bias=None, opts=True,
             ids=65536, w=65536, off=65536, order=65536, pos=65536, ws=65536, ws_bytes=1 << 20):
        o = lib.CRouteOpts(k, score, groups, top_groups, gs, 1, bias)
        return lib.lib.nvfp4_route(l, dt, T, n, ld, ctypes.byref(o) if opts else None, ids, w, off, order, pos, ws,
                                   ws_bytes, None)

    for kw in (dict(l=None), dict(opts=False), dict(ids=None), dict(w=None), dict(off=None), dict(order=None),
               dict(pos=None)):
        assert call(**kw) == E["NULL"], kw
    for kw in (dict(dt=2), dict(score=2), dict(score=-1), dict(gs=2)):
        assert call(**kw) == E["ENUM"], kw
    for kw in (dict(T=-1), dict(n=0, ld=0), dict(ld=63), dict(k=0), dict(k=65), dict(groups=0), dict(groups=5),
               dict(groups=4, top_groups=0), dict(groups=4, top_groups=5), dict(groups=16, top_groups=1, k=5)):
        assert call(**kw) == E["SHAPE"], kw
    for kw in (dict(l=65538), dict(ids=65538), dict(w=65537), dict(off=65540), dict(order=65538), dict(pos=65538),
               dict(bias=65538), dict(ws=65544)):
        assert call(**kw) == E["ALIGN"], kw
    for kw in (dict(n=2049, ld=2049), dict(k=17), dict(groups=64, top_groups=64, n=64 * 33, ld=64 * 33),
               dict(n=130, ld=130, groups=65, top_groups=65), dict(T=1 << 30)):
        assert call(**kw) == E["UNSUP"], kw
    assert call(ws=None) == E["WS"]
    assert call(ws_bytes=lib.nvfp4_route_workspace_size(100, 64) - 1) == E["WS"]
    assert lib.nvfp4_route_workspace_size(1, 64) == 0
    assert lib.nvfp4_route_workspace_size(-1, 64) == 0 and lib.nvfp4_route_workspace_size(100, 4096) == 0


def test_route_backward_rejects_bad_arguments(lib):
    def call(dw=65536, l=65536, dt=0, T=8, n=64, ld=64, ids=65536, k=4, score=0, ds=65536, ldds=64, out=65536, ldo=64):
        return lib.lib.nvfp4_route_backward(dw, l, dt, T, n, ld, ids, k, score, 1, ds, ldds, out, ldo, None)

    for kw in (dict(dw=None), dict(l=None), dict(ids=None), dict(out=None)):
        assert call(**kw) == E["NULL"], kw
    assert call(dt=3) == E["ENUM"] and call(score=3) == E["ENUM"]
    for kw in (dict(T=-1), dict(ld=63), dict(ldds=63), dict(ldo=63), dict(k=0), dict(k=65)):
        assert call(**kw) == E["SHAPE"], kw
    for kw in (dict(dw=65538), dict(l=65538), dict(ids=65538), dict(ds=65538), dict(out=65538)):
        assert call(**kw) == E["ALIGN"], kw
    assert call(n=4096, ld=4096, ldds=4096, ldo=4096) == E["UNSUP"] and call(k=17) == E["UNSUP"]
    assert call(T=0, l=None, out=None, ids=None, dw=None, ds=None) == E["OK"]


def test_python_refusals(lib):
    l = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        lib.nvfp4_route(l, 2)                                     # not on a GPU
    with pytest.raises(ValueError):
        lib.nvfp4_route(l, 2, bias=torch.zeros(7))
    with pytest.raises(TypeError):
        lib.nvfp4_route(l, 2, bias=torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        lib.nvfp4_route(l.double(), 2)
    with pytest.raises(TypeError):
        lib.nvfp4_route_backward(torch.zeros(4, 2), l, torch.zeros(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError):
        lib.nvfp4_route_backward(torch.zeros(4, 3), l, torch.zeros(4, 2, dtype=torch.int32))


# ---------------------------------------------------------------- on the GPU
@pytest.fixture(scope="module")
def nv():
    from parity_utils import require_gpu
    return require_gpu()


def check(nv, logits, k, bias=None, sigmoid=False, groups=1, top_groups=1, top2=True, renorm=True):
    r = nv.nvfp4_route(logits, k, bias=bias, score=nv.NVFP4_ROUTE_SIGMOID if sigmoid else nv.NVFP4_ROUTE_SOFTMAX,
                       groups=groups, top_groups=top_groups,
                       group_score=nv.NVFP4_GROUP_TOP2 if top2 else nv.NVFP4_GROUP_MAX, renorm=renorm)
    l = P.host(logits)
    ids, w = P.route(l, k, None if bias is None else P.host(bias), sigmoid, groups, top_groups, top2, renorm)
    got = r.ids.cpu().numpy()
    assert np.array_equal(got, ids), f"first differing token {np.argwhere((got != ids).any(axis=1))[0]}"
    tol = (16 + (0 if renorm or sigmoid else 48)) * P.U
    assert (np.abs(P.host(r.weights) - w) <= tol * w + 2.0 ** -149).all()
    off, order, pos = P.plan(ids, logits.shape[1])
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.position.cpu().numpy(), pos)
    r2 = nv.nvfp4_route(logits, k, bias=bias, score=nv.NVFP4_ROUTE_SIGMOID if sigmoid else nv.NVFP4_ROUTE_SOFTMAX,
                        groups=groups, top_groups=top_groups,
                        group_score=nv.NVFP4_GROUP_TOP2 if top2 else nv.NVFP4_GROUP_MAX, renorm=renorm, plan=False)
    assert torch.equal(r.ids, r2.ids) and torch.equal(r.weights, r2.weights) and r2.order is None
    return r


def make(seed, T, n, dt, spread=1.0):
    g = np.random.default_rng(seed)
    return torch.from_numpy(spread * g.standard_normal((T, n)) + 0.5 * g.standard_normal(n)).to(dt).cuda()


SHAPES = [  # tokens, experts, top_k, groups, top_groups
    (1, 256, 8, 8, 4), (1, 1, 1, 1, 1), (32, 32, 4, 1, 1), (33, 8, 2, 1, 1), (100, 13, 3, 1, 1), (257, 256, 8, 8, 4),
    (65, 160, 6, 8, 3), (50, 30, 5, 3, 2), (40, 512, 16, 4, 1), (20, 500, 8, 5, 3), (20, 2048, 16, 64, 7),
    (35, 1000, 8, 1, 1), (64, 96, 2, 32, 5), (300, 64, 1, 2, 2), (3000, 40, 3, 4, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,n,k,groups,top_groups", SHAPES)
def test_route(nv, T, n, k, groups, top_groups, sigmoid, dtype):
    l = make(T + n, T, n, DT[dtype])
    bias = 0.05 * torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda()
    for b in (None, bias):
        check(nv, l, k, b, sigmoid, groups, top_groups)
    check(nv, l, k, bias, sigmoid, groups, top_groups, top2=False, renorm=False)
    check(nv, l, k, None, sigmoid, groups, top_groups, top2=False)


@pytest.mark.gpu
@pytest.mark.parametrize("sigmoid", [False, True])
def test_scores_nearer_than_binary32(nv, sigmoid):
    """Scores that binary32 cannot tell apart, ordered by the bias in
    binary64: logits 0 and biases that differ by 2^-30 in a shuffled order,
    beside exact ties."""
    n = 64
    g = np.random.default_rng(3)
    step = g.permutation(n) // 2  # every value twice
    bias = torch.from_numpy((0.25 + step * 2.0 ** -24).astype(np.float32)).cuda()
    l = torch.zeros(40, n, device="cuda")
    l[1::2] = torch.from_numpy(g.integers(0, 2, (20, n)).astype(np.float32)).cuda() * 1.3e-7
    check(nv, l, 16, bias, sigmoid)
    # (groups: only the rows whose sums are exact, so that equal ones tie)
    check(nv, l[::2], 8, bias, sigmoid, 8, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("size", [64.0, 1e3, 1e4, 1e6])
def test_groups_whose_best_two_cancel(nv, size, sigmoid):
    """A favoured and a barred expert in each group: the sum of their scores is
    near 1, but each is rounded by its own size.  Ordinary logits, and logits so
    near that the groups' sums differ by about those roundings."""
    g = np.random.default_rng(12)
    for n in (16, 64):
        bias = np.full((8, n // 8), -2 * size)
        bias[:, 0], bias[:, 1] = size, -size
        bias = torch.from_numpy(bias.reshape(-1)).float().cuda()
        for spread in (1.0, size * 2.0 ** -23):
            l = torch.from_numpy(spread * g.standard_normal((1000, n))).float().cuda()
            check(nv, l, 4, bias, sigmoid, 8, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_binary64_rounds_alike(nv, dtype):
    """Sigmoids of 17 to 60, many of which are 1 in binary64, and softmax scores
    that underflow: by the logits without a bias, ties with a bias of zeros."""
    g = np.random.default_rng(16)
    l = torch.from_numpy(g.uniform(17, 60, (60, 64))).to(DT[dtype]).cuda()
    low = torch.from_numpy(g.uniform(-1500, -700, (60, 64))).to(DT[dtype]).cuda()
    low[:, 5] = 0.0
    zeros = torch.zeros(64, device="cuda")
    for logits, sigmoid in ((l, True), (low, False)):
        for b in (None, zeros):
            check(nv, logits, 8, b, sigmoid)
            check(nv, logits, 8, b, sigmoid, 8, 3)
            check(nv, logits, 8, b, sigmoid, 8, 3, top2=False)
    row = l[:1].sort(dim=1).values
    r, z = (nv.nvfp4_route(row, 4, bias=b, score=nv.NVFP4_ROUTE_SIGMOID) for b in (None, zeros))
    assert torch.equal(r.ids[0].long(), row[0].sort(descending=True, stable=True).indices[:4]) and z.ids[0, 0] < 60


@pytest.mark.gpu
@pytest.mark.parametrize("top_k", [3, 8])
def test_many_near_experts_in_groups_without_a_bias(nv, top_k):
    """More near experts than the quick path settles: the groups of the largest
    logits stay, though all sigmoids are 1 in binary64."""
    l = torch.full((4, 128), 40.0, device="cuda")
    l[0, 64:], l[1, 64:], l[2, :64] = 50.0, 40.000004, 50.0
    r = check(nv, l, top_k, None, True, 2, 1, top2=False)
    assert r.ids[:, 0].tolist() == [64, 64, 0, 0]
    check(nv, l, top_k, None, True, 2, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("sigmoid", [False, True])
def test_group_sums_past_binary32(nv, sigmoid):
    """Biases whose sums no binary32 holds, of either sign, beside ordinary and
    masked groups."""
    inf = float("inf")
    l = make(15, 50, 16, torch.float32)
    for bias in ([-3e38, -2e38, -3e38, -1e38, -3e38, -3e38, -3e38, -0.5e38, -1e38, -3.2e38, -inf, -inf, -2e38, -2e38, -3e38, -inf],
                 [3e38, 2e38, 3e38, 1e38, 3e38, 3e38, 3e38, 0.5e38, 1e38, 3.2e38, inf, inf, 2e38, 2e38, 3e38, inf],
                 [0, 0, -3e38, -1e38, -3e38, -3e38, 0, 0, 3e38, 1e38, 3e38, 3e38, -inf, -inf, 3e38, -3e38]):
        bias = torch.tensor(bias, device="cuda")
        for top_groups in range(1, 8):
            check(nv, l, 2, bias, sigmoid, 8, top_groups)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups_with_masked_experts(nv, sigmoid, dtype):
    """Experts masked by a bias of -inf, of NaN or of the lowest value: groups
    without a live one, with one (a sum that the masked one rounds away: ties to
    the lower index) and with more; and experts that a bias of inf makes certain."""
    inf, low = float("inf"), torch.finfo(torch.float32).min
    l = make(13, 200, 64, DT[dtype])
    for mask in (-inf, low, float("nan")):
        bias = 0.05 * torch.randn(64, generator=torch.Generator().manual_seed(14))
        bias[:8] = mask           # group 0: none left
        bias[9:16] = mask         # 1 and 3: one
        bias[24:31] = mask
        bias[34:40] = mask        # 4: two
        bias[56:] = mask          # 7: none
        for top_groups in (2, 5, 7):
            check(nv, l, 6, bias.cuda(), sigmoid, 8, top_groups)
            check(nv, l, 6, bias.cuda(), sigmoid, 8, top_groups, top2=False)
        bias[50], bias[20], bias[21] = inf, inf, inf
        check(nv, l, 6, bias.cuda(), sigmoid, 8, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ties_go_to_the_lower_index(nv, dtype):
    g = np.random.default_rng(4)
    l = torch.from_numpy(g.integers(0, 3, (70, 96)).astype(np.float32)).to(DT[dtype]).cuda()
    for sigmoid in (False, True):
        check(nv, l, 8, None, sigmoid, 4, 2)
        check(nv, l, 8, torch.zeros(96, device="cuda"), sigmoid, 4, 2)
        check(nv, torch.zeros(5, 96, dtype=DT[dtype], device="cuda"), 5, None, sigmoid, 4, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_logits(nv, dtype):
    inf = float("inf")
    low = torch.finfo(DT[dtype]).min
    l = make(5, 12, 32, torch.float32)
    l[0, 4:] = -inf                   # fewer than top_k left
    l[1, :] = -inf                    # nothing left
    l[2, :] = low
    l[3, :16] = low
    l[4, 3] = inf
    l[5, 2], l[5, 9] = inf, inf
    l[6, 7] = float("nan")
    l[7, :] = float("nan")
    l[8, :] = inf
    l[9, :] = -200.0                  # sigmoids below binary32's range
    l[9, 5] = -199.0
    l[10, :] = 90.0
    l[11, ::2] = -inf
    l = l.to(DT[dtype])
    for sigmoid in (False, True):
        r = check(nv, l, 8, None, sigmoid)
        assert torch.isfinite(r.weights).all()
        # (with groups: the group scores of the hidden rows are ties of underflown sums)
        check(nv, l[:9], 8, None, sigmoid, 4, 2, top2=False)
    r = check(nv, l, 8, None, False)
    assert r.ids[1].tolist() == list(range(8)) and (r.weights[1] == 0.125).all()
    bias = torch.zeros(32, device="cuda")
    bias[:30] = -inf
    bias[3] = float("nan")
    l = make(6, 10, 32, DT[dtype])
    r = nv.nvfp4_route(l, 3, bias=bias, score=nv.NVFP4_ROUTE_SIGMOID)
    assert (r.ids[:, :2].sort(dim=1).values.cpu() == torch.tensor([30, 31])).all() and (r.ids[:, 2] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_logits(nv, dtype):
    buf = make(7, 90, 131, DT[dtype])
    check(nv, buf[:, 1:129], 8, None, False, 8, 4)
    check(nv, buf[:, 3:70], 4, None, True)


@pytest.mark.gpu
def test_given_outputs(nv):
    """Some tensors given: the result has them and new ones for the rest; without
    a plan it holds none, whatever the given object still has of an earlier call."""
    l = make(17, 30, 32, torch.float32)
    want = nv.nvfp4_route(l, 4)
    some = nv.RouteOutput(torch.empty_like(want.ids), torch.empty_like(want.weights))
    got = nv.nvfp4_route(l, 4, out=some)
    assert got.ids is some.ids and got.weights is some.weights
    for a, b in zip((want.ids, want.weights, want.offsets, want.order, want.position),
                    (got.ids, got.weights, got.offsets, got.order, got.position)):
        assert torch.equal(a, b)
    plan = [t.clone() for t in (got.offsets, got.order, got.position)]
    again = nv.nvfp4_route(-l, 4, plan=False, out=got)
    assert again.ids is got.ids and again.offsets is None and again.order is None and again.position is None
    assert all(torch.equal(a, b) for a, b in zip(plan, (got.offsets, got.order, got.position)))
    assert torch.equal(again.ids, nv.nvfp4_route(-l, 4).ids)


@pytest.mark.gpu
def test_no_tokens(nv):
    r = nv.nvfp4_route(torch.zeros(0, 16, device="cuda"), 4)
    assert r.ids.shape == (0, 4) and (r.offsets == 0).all()
    assert nv.nvfp4_route_backward(torch.zeros(0, 4, device="cuda"), torch.zeros(0, 16, device="cuda"),
                                   r.ids).shape == (0, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,k", [(16384, 256, 8), (20001, 32, 4), (16385, 9, 2)])
def test_plan_of_many_tokens(nv, T, n, k):
    """More than one assignment chunk a span and spans of unequal length: the
    plan against a stable sort, the ids against a sort of the logits."""
    l = make(8, T, n, torch.bfloat16)
    r = nv.nvfp4_route(l, k)
    ids = l.float().sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)
    assert torch.equal(r.ids, ids)
    off, order, pos = P.plan(ids.cpu().numpy(), n)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.order.cpu().numpy(), order) and np.array_equal(r.position.cpu().numpy(), pos)


def backward_tol(dw, l, ids, sigmoid, renorm, ds, dl, dt, n):
    """Roundings counted on each term: scores within (n / 16 + 24) U (their sum
    over n experts included), a few more around them."""
    p = P.scores(l, sigmoid)
    w = np.take_along_axis(p, ids, axis=1)
    if renorm:
        w = w / w.sum(axis=1, keepdims=True)
    D = np.zeros_like(p)
    np.put_along_axis(D, ids, w * (np.abs(dw) + ((np.abs(dw) * w).sum(axis=1, keepdims=True) if renorm else 0)), 1)
    a = 0 if ds is None else np.abs(ds)
    terms = p * a + D
    if not sigmoid:
        terms = terms + p * ((p * a).sum(axis=1, keepdims=True) + (0 if renorm else (np.abs(dw) * w).sum(axis=1, keepdims=True)))
    tol = 2 * (n / 16 + 24) * P.U * terms
    return tol + (2.0 ** -8 if dt == torch.bfloat16 else 0.0) * (np.abs(dl) + tol)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,n,k", [(1, 256, 8), (5, 1, 1), (33, 8, 2), (70, 13, 3), (257, 128, 4), (40, 129, 8),
                                   (50, 300, 6), (19, 512, 16), (21, 700, 8), (9, 2048, 16)])
def test_backward(nv, T, n, k, sigmoid, dtype):
    dt = DT[dtype]
    score = nv.NVFP4_ROUTE_SIGMOID if sigmoid else nv.NVFP4_ROUTE_SOFTMAX
    g = np.random.default_rng(T)
    l = make(T, T, n, dt)
    ids = np.stack([g.permutation(n)[:k] for _ in range(T)])  # (any experts, not only the largest)
    dw, ds = g.standard_normal((T, k)).astype(np.float32), (0.1 * g.standard_normal((T, n))).astype(np.float32)
    for renorm in (True, False):
        for d in (ds, None):
            got = nv.nvfp4_route_backward(torch.from_numpy(dw).cuda(), l, torch.from_numpy(ids).int().cuda(), score=score,
                                          renorm=renorm, dscores=None if d is None else torch.from_numpy(d).cuda())
            a = (dw.astype(np.float64), P.host(l), ids, sigmoid, renorm, None if d is None else d.astype(np.float64))
            want = P.route_backward(*a)
            assert (np.abs(P.host(got) - want) <= backward_tol(*a, want, dt, n)).all(), (renorm, d is None)


@pytest.mark.gpu
def test_sigmoids_below_the_normal_numbers(nv):
    """Logits of -80 to -104 beside ordinary ones: weights and gradients down to
    binary32's smallest numbers.  An exponential within 2 steps of 2^-149 and one
    rounding after it; a gradient's term multiplies the steps by its factors and
    is rounded four times."""
    step = 2.0 ** -149
    l = torch.from_numpy(np.random.default_rng(18).uniform(-104, -80, (40, 12))).float().cuda()
    l[:, 5] = torch.linspace(-3, 3, 40)
    g = np.random.default_rng(19)
    dw, ds = g.standard_normal((40, 8)).astype(np.float32), g.standard_normal((40, 12)).astype(np.float32)
    for renorm in (True, False):
        r = nv.nvfp4_route(l, 8, score=nv.NVFP4_ROUTE_SIGMOID, renorm=renorm)
        ids, w = P.route(P.host(l), 8, None, True, renorm=renorm)
        assert np.array_equal(r.ids.cpu().numpy(), ids)
        scale = 1.0 / P.scores(P.host(l), True).max(axis=1, keepdims=True) if renorm else 1.0
        assert (np.abs(P.host(r.weights) - w) <= 16 * P.U * w + 2 * step * scale + step).all()
        got = nv.nvfp4_route_backward(torch.from_numpy(dw).cuda(), l, r.ids, score=nv.NVFP4_ROUTE_SIGMOID, renorm=renorm,
                                      dscores=torch.from_numpy(ds).cuda())
        a = (dw.astype(np.float64), P.host(l), ids, True, renorm, ds.astype(np.float64))
        want = P.route_backward(*a)
        factors = np.abs(ds) + 2 * np.abs(dw).max(axis=1, keepdims=True) * scale
        assert (np.abs(P.host(got) - want) <= backward_tol(*a, want, torch.float32, 12) + (2 * factors + 4) * step).all()


@pytest.mark.gpu
@pytest.mark.parametrize("top", [-60.0, -40.0, -3.0, 0.5])
def test_small_sigmoids_divided_by_small_sums(nv, top):
    """Chosen logits from `top` down: weights that are normal numbers though the
    sigmoids are not, and those of them that are not.  (Steps as above: what is
    left of a sigmoid's own where the largest is not small.)"""
    step = 2.0 ** -149
    g = np.random.default_rng(21)
    l = torch.from_numpy(top - g.uniform(0, 100, (60, 12))).float().cuda()
    l[:, 3] = top
    dw = g.standard_normal((60, 12)).astype(np.float32)
    r = nv.nvfp4_route(l, 12, score=nv.NVFP4_ROUTE_SIGMOID)
    ids, w = P.route(P.host(l), 12, None, True)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert (np.abs(P.host(r.weights) - w) <= 16 * P.U * w + 5 * step).all()
    got = nv.nvfp4_route_backward(torch.from_numpy(dw).cuda(), l, r.ids, score=nv.NVFP4_ROUTE_SIGMOID)
    a = (dw.astype(np.float64), P.host(l), ids, True, True, None)
    want = P.route_backward(*a)
    factors = 2 * np.abs(dw).max(axis=1, keepdims=True)
    assert (np.abs(P.host(got) - want) <= backward_tol(*a, want, torch.float32, 12) + (5 * factors + 4) * step).all()


@pytest.mark.gpu
@pytest.mark.parametrize("sigmoid", [False, True])
def test_backward_against_differences(nv, sigmoid):
    l = make(9, 6, 48, torch.float32)
    score = nv.NVFP4_ROUTE_SIGMOID if sigmoid else nv.NVFP4_ROUTE_SOFTMAX
    r = nv.nvfp4_route(l, 5, score=score)
    g = np.random.default_rng(10)
    dw, ds = g.standard_normal((6, 5)).astype(np.float32), g.standard_normal((6, 48)).astype(np.float32)
    got = P.host(nv.nvfp4_route_backward(torch.from_numpy(dw).cuda(), l, r.ids, score=score,
                                         dscores=torch.from_numpy(ds).cuda()))
    ids, L = r.ids.cpu().numpy(), P.host(l)

    def loss(a):
        p = P.scores(a, sigmoid)
        w = np.take_along_axis(p, ids, axis=1)
        return (w / w.sum(axis=1, keepdims=True) * dw).sum() + (p * ds).sum()

    t = 1e-5
    for _ in range(4):
        v = g.standard_normal(L.shape)
        assert abs((loss(L + t * v) - loss(L - t * v)) / (2 * t) - (got * v).sum()) <= 1e-5 * np.abs(got * v).sum()


@pytest.mark.gpu
def test_backward_masks_and_foreign_ids(nv):
    """Masked logits get no gradient and give no NaN; an id out of range counts
    as none; in place on the logits."""
    l = make(11, 4, 40, torch.float32)
    l[0, 20:] = float("-inf")
    l[1, :] = float("-inf")
    ids = torch.tensor([[0, 1], [2, 3], [5, -1], [40, 7]], dtype=torch.int32, device="cuda")
    dw = torch.ones(4, 2, device="cuda")
    dw[:, 1] = -2.0
    for sigmoid in (False, True):
        score = nv.NVFP4_ROUTE_SIGMOID if sigmoid else nv.NVFP4_ROUTE_SOFTMAX
        for renorm in (True, False):
            dl = nv.nvfp4_route_backward(dw, l, ids, score=score, renorm=renorm)
            assert torch.isfinite(dl).all() and (dl[0, 20:] == 0).all()
            one = nv.nvfp4_route_backward(dw[2:3, :1].contiguous(), l[2:3], ids[2:3, :1].contiguous(), score=score,
                                          renorm=renorm)
            assert torch.equal(dl[2:3], one)
            buf = l.clone()
            assert nv.nvfp4_route_backward(dw, buf, ids, score=score, renorm=renorm, out=buf) is buf
            assert torch.equal(buf, dl)


@pytest.mark.gpu
def test_offsets_past_32_bits(nv):
    ld = 2 ** 31 + 32
    buf = torch.empty(ld + 64, dtype=torch.bfloat16, device="cuda").as_strided((2, 64), (ld, 1))
    buf.copy_(make(20, 2, 64, torch.bfloat16))
    r = check(nv, buf, 8, torch.zeros(64, device="cuda"), True, 4, 2)
    dw = torch.ones(2, 8, device="cuda")
    want = nv.nvfp4_route_backward(dw, buf.contiguous(), r.ids)
    assert torch.equal(nv.nvfp4_route_backward(dw, buf, r.ids, out=buf), want)


@pytest.mark.gpu
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("n,groups,k", [(256, 8, 8), (304, 8, 8), (340, 2, 15), (48, 16, 16)])
def test_equal_rows(nv, n, groups, k, sigmoid):
    """Rows whose logits are all alike (padding tokens), among others, at token
    counts of every layout: the lowest experts, in order; with a bias of few
    values the lowest of the largest."""
    for T in (3, 300):
        l = make(T, T, n, torch.float32)
        l[::3] = 0.0
        l[1::7] = -3.5
        few = torch.from_numpy((0.25 * np.random.default_rng(n).integers(0, 2, n)).astype(np.float32)).cuda()
        for b in (None, torch.zeros(n, device="cuda"), few):
            check(nv, l, k, b, sigmoid, groups, max(groups // 2, 1))
            check(nv, l.bfloat16(), k, b, sigmoid, groups, max(groups // 2, 1))
            check(nv, l, k, b, sigmoid)


@pytest.mark.gpu
@pytest.mark.parametrize("T,n,groups,top_groups,k", [(700, 304, 8, 3, 8), (300, 512, 1, 1, 8), (300, 330, 2, 1, 16),
                                                      (290, 272, 17, 5, 4), (1030, 1024, 4, 2, 15)])
def test_shapes_of_many_tokens(nv, T, n, groups, top_groups, k):
    l = make(T + n, T, n, torch.float32)
    bias = 0.05 * torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda()
    for dt in (torch.float32, torch.bfloat16):
        check(nv, l.to(dt), k, bias, True, groups, top_groups)
        check(nv, l.to(dt), k, None, False, groups, top_groups)
        check(nv, l.to(dt), k, bias, False, groups, top_groups, top2=False)
