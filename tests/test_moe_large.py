"""The MoE-block operators at sizes that one launch's grid cannot hold (2^32
threads): every output is compared with those of a small call whose rows, or
columns, the large one repeats.  The sizes are those at which the 32-bit number
of threads has just been passed."""
import pytest
import torch

pytestmark = pytest.mark.gpu

GB = 1 << 30


@pytest.fixture
def nv():
    from parity_utils import require_gpu
    yield require_gpu()
    torch.cuda.empty_cache()


def needs(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * GB:
        pytest.skip(f"needs {gib} GiB of free device memory")


def repeated(block, times):
    """The block's rows, `times` times under each other."""
    out = torch.empty((times,) + tuple(block.shape), dtype=block.dtype, device="cuda")
    out.copy_(block)
    return out.view((-1,) + tuple(block.shape[1:]))


def repeats(got, block):
    """Whether got's rows are the block's, again and again."""
    got = got.view((-1,) + tuple(block.shape))
    step = max(1, GB // (block.numel() * block.element_size()))
    return all(bool((got[i:i + step] == block).all()) for i in range(0, got.shape[0], step))


def test_norm_of_many_wide_rows(nv):
    """4194368 rows of 8224 columns, a workgroup of 1024 threads each."""
    needs(100)
    rows, cols, times = 64, 8224, 65537
    block = torch.randn(rows, cols, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    w = torch.linspace(0.5, 1.5, cols, device="cuda")
    want = nv.nvfp4_rmsnorm(block, w, y=False, mx_elem=nv.NVFP4_MX_E2M1, rstd=True)
    got = nv.nvfp4_rmsnorm(repeated(block, times), w, y=False, mx_elem=nv.NVFP4_MX_E2M1, rstd=True)
    assert repeats(got.mx.codes, want.mx.codes) and repeats(got.mx.scales, want.mx.scales)
    assert repeats(got.rstd, want.rstd)


def test_routing_backward_of_many_tokens(nv):
    """2^28 + 4096 tokens, four to a wave of 64 threads."""
    needs(8)
    g = torch.Generator().manual_seed(2)
    times = (2 ** 28 + 4096) // 4096
    l = torch.randn(4096, 1, generator=g).bfloat16().cuda()
    dw, ds = torch.randn(4096, 1, generator=g).cuda(), torch.randn(4096, 1, generator=g).cuda()
    ids = torch.zeros(4096, 1, dtype=torch.int32, device="cuda")
    kw = dict(score=nv.NVFP4_ROUTE_SIGMOID, renorm=False)
    want = nv.nvfp4_route_backward(dw, l, ids, dscores=ds, **kw)
    got = nv.nvfp4_route_backward(repeated(dw, times), repeated(l, times), repeated(ids, times),
                                  dscores=repeated(ds, times), **kw)
    assert repeats(got, want)


def test_routing_of_many_tokens(nv):
    """805478400 tokens, 192 to a workgroup of 1024 threads, and their plan."""
    needs(40)
    period, times = 4096, 196650
    block = torch.randn(period, 2, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    want = nv.nvfp4_route(block, 1, score=nv.NVFP4_ROUTE_SIGMOID, renorm=False)
    got = nv.nvfp4_route(repeated(block, times), 1, score=nv.NVFP4_ROUTE_SIGMOID, renorm=False)
    assert repeats(got.ids, want.ids) and repeats(got.weights, want.weights)
    # an expert's assignments lie in order, each period's after the last one's
    assert torch.equal(got.offsets, want.offsets * times)
    counts = want.offsets.diff()
    place = want.position - want.offsets[want.ids[:, 0].long()]  # within the expert and the period
    at = got.position.view(times, period)
    order = got.order
    for i in range(0, times, 16384):
        p = torch.arange(i, min(i + 16384, times), device="cuda").view(-1, 1)
        e = want.ids[:, 0].long()
        expect = got.offsets[e] + p * counts[e] + place
        assert torch.equal(at[i:i + 16384], expect.int())
        t = p * period + torch.arange(period, device="cuda")
        assert torch.equal(order[expect], t.int())


def repeated_weight(nv, rows, times):
    """A weight of 16 columns whose rows repeat, and its first `rows`."""
    g = torch.Generator().manual_seed(4)
    codes = torch.randint(0, 256, (rows, 8), generator=g, dtype=torch.uint8).cuda()
    scales = torch.randint(40, 80, (rows, 1), generator=g, dtype=torch.uint8).cuda()
    ts = torch.full((1,), 0.5, device="cuda")
    return (nv.NVFP4Tensor(codes, scales, ts, rows, 16),
            nv.NVFP4Tensor(repeated(codes, times), repeated(scales, times), ts, rows * times, 16))


@pytest.mark.parametrize("m", [1, 5])
def test_product_with_many_rows(nv, m):
    """The most rows of a weight that are taken, less 4096."""
    needs(20)
    small, large = repeated_weight(nv, 4096, 2 ** 17 - 1)
    x = torch.randn(m, 16, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    want, got = nv.nvfp4_gemv(x, small), nv.nvfp4_gemv(x, large)
    for i in range(m):
        assert repeats(got[i], want[i])
