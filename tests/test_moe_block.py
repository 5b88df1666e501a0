"""The operators together, as examples/moe_block.py runs them: the decode path
against a 64-bit evaluation, the prefill path against the decode path, the
router's and the norm's gradients against differences of the 64-bit form, and
the decode path in a graph and on another stream."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import moe_plain as P

pytestmark = pytest.mark.gpu

HIDDEN, FFN, EXPERTS, TOP_K = 256, 64, 8, 3


@pytest.fixture(scope="module")
def example():
    from parity_utils import require_gpu
    require_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def block(example):
    return example.MoEBlock(HIDDEN, FFN, EXPERTS, TOP_K, groups=4, top_groups=2)


def inputs(tokens, seed=3):
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn(tokens, HIDDEN, generator=g).bfloat16().cuda() for _ in range(2))


def route64(block, y):
    l = P.host(y) @ P.host(block.router).T
    return P.route(l, TOP_K, P.host(block.bias), True, 4, 2)


def test_decode(block):
    x, res = inputs(5)
    h, out = block.decode(x, res)
    h64 = P.host(h)
    # (a binary32 sum, one BF16 rounding)
    assert (np.abs(h64 - P.host(x) - P.host(res)) <= (2.0 ** -8 + P.U) * np.abs(P.host(x) + P.host(res))).all()
    # from the stored y on: its own test bounds its rounding
    n = block_norm(block, x, res)
    ids, w = route64(block, n.y)
    Y, up, down = P.host(n.y), P.nvfp4_weight(block.up, EXPERTS), P.nvfp4_weight(block.down, EXPERTS)
    up, down = up.reshape(EXPERTS, 2 * FFN, HIDDEN), down.reshape(EXPERTS, HIDDEN, FFN)
    want, tol = np.zeros((5, HIDDEN)), np.zeros((5, HIDDEN))
    for t in range(5):
        for e, wt in zip(ids[t], w[t]):
            z, za = up[e] @ Y[t], 1e-5 * (np.abs(up[e]) @ np.abs(Y[t]))
            a, ta = P.swiglu(z[None], za[None])
            a, ta = a[0], ta[0] + 8 * P.U * np.abs(a[0])
            ta = ta + 2.0 ** -8 * (np.abs(a) + ta)  # the stored activation
            want[t] += wt * (down[e] @ a)
            # 1e-5 of the products and the weight's and the sum's roundings
            tol[t] += wt * (np.abs(down[e]) @ ta + (1e-5 + 32 * P.U) * (np.abs(down[e]) @ (np.abs(a) + ta)))
    assert (np.abs(P.host(out) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol)).all()


def block_norm(block, x, res):
    import bit_block_scaled_quantize_amd as nv
    return nv.nvfp4_rmsnorm(x, block.norm, residual=res, eps=block.eps)


def test_prefill_follows_decode(block):
    """The same experts, weights and residual stream; the activations' 4-bit
    rounding (a step of 1/4 to 1/2 of a value at most) leaves the outputs
    within a relative 1/4 in the norm."""
    x, res = inputs(200)
    h, moe, dense = block.prefill(x, res)
    assert dense.shape == (200, HIDDEN) and torch.isfinite(dense.float()).all()
    for at in range(0, 200, 8):
        dh, out = block.decode(x[at:at + 8], res[at:at + 8])
        assert torch.equal(dh, h[at:at + 8])
        a, b = P.host(out), P.host(moe[at:at + 8])
        assert np.linalg.norm(a - b) <= 0.25 * np.linalg.norm(a)


def test_gradients(block):
    """Along random directions of the residual stream, the norm's and the
    router's weight.  The stored y, dy and dx are BF16 (2^-8 each, on both
    factors of a product): 3 * 2^-8 of the terms' absolute sum."""
    g = np.random.default_rng(5)
    x, res = inputs(12)
    dw, ds = g.standard_normal((12, TOP_K)).astype(np.float32), 0.1 * g.standard_normal((12, EXPERTS)).astype(np.float32)
    dh = torch.from_numpy(g.standard_normal((12, HIDDEN))).bfloat16().cuda()
    dx, dnorm, drouter = block.gradients(x, res, torch.from_numpy(dw).cuda(), torch.from_numpy(ds).cuda(), dh)
    n = block_norm(block, x, res)
    ids, _ = route64(block, n.y)
    H, N, R, DH = P.host(n.h), P.host(block.norm), P.host(block.router), P.host(dh)

    def loss(h, norm, router):
        p = P.scores(P.rmsnorm(h, norm, block.eps)[1] @ router.T, True)
        w = np.take_along_axis(p, ids, axis=1)
        return (w / w.sum(axis=1, keepdims=True) * dw).sum() + (p * ds).sum() + (h * DH).sum()

    t = 1e-5
    for got, at in ((P.host(dx), 0), (P.host(dnorm), 1), (P.host(drouter), 2)):
        for _ in range(3):
            v = g.standard_normal(got.shape)
            args = [H, N, R]
            plus, minus = list(args), list(args)
            plus[at], minus[at] = args[at] + t * v, args[at] - t * v
            want = (loss(*plus) - loss(*minus)) / (2 * t)
            assert abs((got * v).sum() - want) <= 3 * 2.0 ** -8 * np.abs(got * v).sum()


def test_decode_in_a_graph_and_on_a_stream(block):
    x, res = inputs(4)
    want = block.decode(x, res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = block.decode(x, res)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block.decode(x, res)
    for seed in range(3):
        for dst, src in zip((x, res), inputs(4, 20 + seed)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(block.decode(x, res), out))
        torch.cuda.synchronize()


def test_norm_and_routing_on_a_stream_and_with_given_outputs(block):
    """`stream=` and preallocated outputs give what a plain call gives, and a
    captured training step's operators replay to the same gradients."""
    import bit_block_scaled_quantize_amd as nv
    x, res = inputs(300)
    y = block_norm(block, x, res).y
    logits = y.float() @ block.router.float().t()
    ids = nv.nvfp4_route(logits, TOP_K, bias=block.bias).ids
    rstd = torch.rsqrt(x.float().square().mean(dim=1) + 1e-6)
    dw = torch.randn(300, TOP_K, device="cuda")

    def run(stream=None, out=None, workspace=None):
        r = nv.nvfp4_route(logits, TOP_K, bias=block.bias, out=out, workspace=workspace, stream=stream)
        return (r.ids, r.weights, r.offsets, r.order, r.position,
                nv.nvfp4_route_backward(dw, logits, ids, stream=stream),
                *nv.nvfp4_rmsnorm_backward(y, x, rstd, block.norm, dh=res, stream=stream),
                nv.nvfp4_rmsnorm(x, block.norm, residual=res, mx_elem=nv.NVFP4_MX_E4M3, stream=stream).mx.codes)

    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    given = nv.RouteOutput(*(torch.full_like(t, 7) for t in want[:5]))
    ws = torch.empty(nv.nvfp4_route_workspace_size(300, EXPERTS), dtype=torch.uint8, device="cuda")
    got = run(out=given, workspace=ws)
    assert got[0] is given.ids and all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for seed in range(3):
        logits.copy_(torch.randn(300, EXPERTS, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(run(), out))
        torch.cuda.synchronize()
