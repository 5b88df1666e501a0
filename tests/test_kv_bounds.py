"""Plans at their bounds: nothing is written outside of what a call is given, whatever
its plan says (the arrays lie inside larger ones whose margins hold a pattern), and more
segments than there are waves."""
import pytest
import torch

import kv_plain as P
from test_kv_attention import case
from test_kv_cache import make

pytestmark = pytest.mark.gpu
DT = P.DT
MARGIN = 1 << 16  # bytes


@pytest.fixture(scope="module")
def nv():
    import bit_block_scaled_quantize_amd.nvfp4 as nv
    return nv


class Guarded:
    """Tensors with margins of a pattern before and behind them."""

    def __init__(self):
        self.held = []

    def like(self, t):
        n = t.numel() * t.element_size()
        whole = torch.empty(2 * MARGIN + n, dtype=torch.uint8, device="cuda").fill_(0xA5)
        self.held.append((whole, n))
        inner = whole[MARGIN:MARGIN + n].view(t.dtype).view(t.shape)
        inner.copy_(t)
        return inner

    def check(self):
        torch.cuda.synchronize()
        for whole, n in self.held:
            assert bool((whole[:MARGIN] == 0xA5).all()) and bool((whole[MARGIN + n:] == 0xA5).all())


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


ROWS = 300
#: (lengths, offsets) that say what no caller means
PLANS = [([300, 300, 300], [0, 300, 0, 300]), ([300, 300, 300], [300, 0, 300, 0]), ([500, -4, 1 << 30], [-7, 120, 90, 1000]),
         ([-2147483648, 2147483647, 37], [2147483647, -2147483648, 5, 250]), ([300, 250, 200], [0, 290, 10, 300]),
         ([300] * 40, [0, 300] * 20 + [0]), ([480] * 40, [(77 * i) % 301 for i in range(41)])]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("dim,dtype,group", [(64, "bf16", 5), (128, "bf16", 1), (256, "bf16", 4), (128, "f32", 3)])
def test_plans_out_of_order_write_nothing_outside(nv, dim, dtype, group, mx):
    g = Guarded()
    heads, page, rows = 2, 16, ROWS
    for lengths, offsets in PLANS:
        print(lengths[:4], offsets[:5], flush=True)
        seqs = len(lengths)
        cache, _ = make(nv, [480] * min(seqs, 3), heads, dim, page, mx)
        for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
            setattr(cache, n, g.like(getattr(cache, n).fill_(0x38)))
        pages = cache.k_codes.shape[0]
        table = torch.randint(-2, pages + 3, (seqs, 30), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        L, O = ints(lengths), ints(offsets)
        k, v, q = (torch.randn((rows, h, dim), device="cuda").to(DT[dtype]) for h in (heads, heads, heads * group))
        out, lse = g.like(torch.zeros_like(q)), g.like(torch.zeros((rows, heads * group), device="cuda"))
        pair = g.like(torch.zeros_like(k)), g.like(torch.zeros_like(v))
        need = nv.nvfp4_kv_attention_workspace_size(rows, seqs, heads * group, heads, dim, DT[dtype])
        ws = g.like(torch.zeros(need, dtype=torch.uint8, device="cuda"))
        rope = torch.randn((200, 64), device="cuda")
        nv.nvfp4_kv_append(k, v, cache, table, L, O, q=q, rope=rope, out=out)
        nv.nvfp4_kv_gather(cache, table, L, O, rows=rows, out=pair)
        for window in (0, 50):
            nv.nvfp4_kv_attention(q, cache, table, L, O, window=window, lse=True, out=out, out_lse=lse, workspace=ws)
        g.check()
        g.held.clear()


@pytest.mark.parametrize("dim,dtype,group,lengths,offsets",
                         [(64, "bf16", 5, [2100, 40], [3, 250, 290]), (128, "bf16", 1, [900, 17], [0, 283, 300]),
                          (256, "bf16", 4, [5000], [0, 17]), (128, "f32", 3, [4000, 300], [10, 20, 300]),
                          (64, "f32", 1, [20000, 9], [0, 1, 2])])
def test_plans_in_order_write_nothing_outside(nv, dim, dtype, group, lengths, offsets):
    """The workspace's last part and the rows' ends, at sizes whose keys are split."""
    g = Guarded()
    heads, page, rows, seqs = 2, 64, offsets[-1], len(lengths)
    cache, table = make(nv, lengths, heads, dim, page, False, spare=0)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        setattr(cache, n, g.like(getattr(cache, n).fill_(0x38)))
    L, O = ints(lengths), ints(offsets)
    k, v, q = (torch.randn((rows, h, dim), device="cuda").to(DT[dtype]) for h in (heads, heads, heads * group))
    out, lse = g.like(torch.zeros_like(q)), g.like(torch.zeros((rows, heads * group), device="cuda"))
    pair = g.like(torch.zeros_like(k)), g.like(torch.zeros_like(v))
    ws = g.like(torch.zeros(nv.nvfp4_kv_attention_workspace_size(rows, seqs, heads * group, heads, dim, DT[dtype]),
                            dtype=torch.uint8, device="cuda"))
    nv.nvfp4_kv_append(k, v, cache, table, L, O, q=q, out=out)
    nv.nvfp4_kv_gather(cache, table, L, O, rows=rows, out=pair)
    nv.nvfp4_kv_attention(q, cache, table, L, O, lse=True, out=out, out_lse=lse, workspace=ws)
    g.check()
    ref = nv.nvfp4_kv_attention(q, cache, table, L, O)
    assert torch.equal(out[offsets[0]:], ref[offsets[0]:]) and not bool(out[:offsets[0]].any())


def attend(nv, lengths, new, heads, dim, mx, dtype, seed):
    cache, table, L, O, offsets, q = case(nv, lengths, new, heads, 1, dim, 16, mx, dtype, seed)
    o, lse = nv.nvfp4_kv_attention(q, cache, table, L, O, lse=True)
    want = P.attention(q, cache, table, lengths, offsets, dim ** -0.5, 0, cache.k_codes.shape[0], 16)
    P.check(o, lse, want, dtype, mx)


@pytest.mark.parametrize("seqs,heads,dim,dtype", [(600, 8, 64, "bf16"), (450, 8, 128, "f32"), (1100, 8, 64, "f32"), (300, 8, 256, "bf16")])
def test_more_short_sequences_than_waves(nv, seqs, heads, dim, dtype):
    """Segments of one step and none past what all waves take at once, so that they go round
    again: sequences without a row or a position among them."""
    lengths = [0 if i % 11 == 3 else 1 + (29 * i) % 70 for i in range(seqs)]
    attend(nv, lengths, None, heads, dim, False, dtype, 37)
    new = [min(l, (3 * i) % 4) for i, l in enumerate(lengths)]
    attend(nv, lengths, new, heads, dim, True, dtype, 38)


@pytest.mark.parametrize("dim,dtype,teams", [(64, "bf16", 1024), (128, "f32", 768), (256, "bf16", 512)])
def test_as_many_short_sequences_as_teams(nv, dim, dtype, teams):
    """One segment more and less than workgroups, pairs of waves and waves there are."""
    for count in (teams, 2 * teams, 4 * teams):
        for seqs in (count // 8, count // 8 + 1):
            attend(nv, [1 + (31 * i) % 45 for i in range(seqs)], None, 8, dim, False, dtype, 39)


@pytest.mark.parametrize("longest", [1023, 1024, 1025])
def test_the_longest_segment_of_a_team(nv, longest):
    """Divided by team up to 32 steps, in shares past them."""
    lengths = [1 + (353 * i) % 1000 for i in range(80)]
    lengths[41] = longest
    attend(nv, lengths, None, 8, 64, False, "bf16", 40)
    attend(nv, lengths, None, 8, 128, True, "f32", 41)
