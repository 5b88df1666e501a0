"""RMS norm with the residual's addition and an MX output, and its backward
pass, against the plain 64-bit forms of moe_plain.py.

Tolerances count roundings.  A binary32 operation is off by at most U = 2^-24
of its result, a BF16 store by 2^-8.  A row's sum of n squares goes through at
most 32 additions in a thread (4 chunks of 8), 6 over a wave's lanes and 16
over its waves, each of nonnegative terms: relative error below 55 U with the
squares' own; half of that in the square root, and 4 U for the mean, eps, root
and reciprocal: rstd within 32 U.  y adds two products: 34 U."""
import numpy as np
import pytest
import torch

import moe_plain as P

EPS = 1e-6
TOL_RSTD, TOL_Y = 32 * P.U, 34 * P.U
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def test_plain_backward_against_differences():
    g = np.random.default_rng(0)
    h, dy, dh, v = (g.standard_normal((5, 37)) for _ in range(4))
    w, dwv = g.standard_normal(37), g.standard_normal(37)

    def loss(a, b):
        return (P.rmsnorm(a, b, EPS)[1] * dy).sum() + (a * dh).sum()

    rstd, _ = P.rmsnorm(h, w, EPS)
    dx, dw = P.rmsnorm_backward(dy, h, rstd, w, dh)
    t = 1e-5  # (third-order error of the central difference: ~1e-10)
    assert abs((loss(h + t * v, w) - loss(h - t * v, w)) / (2 * t) - (dx * v).sum()) < 1e-6
    assert abs((loss(h, w + t * dwv) - loss(h, w - t * dwv)) / (2 * t) - (dw * dwv).sum()) < 1e-6


# ---------------------------------------------------------------- refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    import bit_block_scaled_quantize_amd.nvfp4 as nv
    return nv


E = dict(OK=0, NULL=1, ENUM=2, SHAPE=3, ALIGN=4, UNSUP=5, WS=6)


def test_rmsnorm_rejects_bad_arguments(lib):
    import ctypes

    def call(x=65536, ldx=64, res=65536, ldr=64, w=65536, wdt=1, dt=1, rows=4, cols=64, eps=1e-6, h=65536, ldh=64,
             y=65536, ldy=64, mx=(4, 64, 0, 65536), rstd=65536):
        t = None if mx is None else lib.CMXTensor(mx[3], 8192, mx[0], mx[1], mx[2])
        return lib.lib.nvfp4_rmsnorm(x, ldx, res, ldr, w, wdt, dt, rows, cols, eps, h, ldh, y, ldy,
                                     None if t is None else ctypes.byref(t), rstd, None)

    assert call(x=None) == E["NULL"]
    assert call(w=None) == E["NULL"]
    assert call(y=None, mx=None) == E["NULL"]
    assert call(mx=(4, 64, 0, None)) == E["NULL"]
    assert call(dt=2) == E["ENUM"]
    assert call(wdt=-1) == E["ENUM"]
    assert call(mx=(4, 64, 2, 65536)) == E["ENUM"]
    assert call(rows=-1) == E["SHAPE"]
    assert call(cols=0) == E["SHAPE"]
    assert call(ldx=63) == E["SHAPE"]
    assert call(ldr=63) == E["SHAPE"]
    assert call(ldh=63) == E["SHAPE"]
    assert call(ldy=63) == E["SHAPE"]
    assert call(cols=48, mx=(4, 48, 0, 65536)) == E["SHAPE"]      # cols % 32 with an MX output
    assert call(mx=(5, 64, 0, 65536)) == E["SHAPE"]
    assert call(x=65537) == E["ALIGN"]
    assert call(w=65537) == E["ALIGN"]
    assert call(dt=0, y=65538) == E["ALIGN"]
    assert call(rstd=65538) == E["ALIGN"]
    assert call(mx=(4, 64, 0, 65544)) == E["ALIGN"]
    assert call(eps=0.0) == E["UNSUP"]
    assert call(eps=float("nan")) == E["UNSUP"]
    big = 32800
    assert call(cols=big, ldx=big, ldr=big, ldh=big, ldy=big, mx=None) == E["UNSUP"]
    assert call(rows=0, x=None, res=None, h=None, mx=None) == E["OK"]


def test_rmsnorm_backward_rejects_bad_arguments(lib):
    need = lib.nvfp4_rmsnorm_backward_workspace_size(4, 64)
    assert need > 0 and lib.nvfp4_rmsnorm_backward_workspace_size(0, 64) == 0
    assert lib.nvfp4_rmsnorm_backward_workspace_size(-1, 64) == 0
    assert lib.nvfp4_rmsnorm_backward_workspace_size(4, 0) == 0

    def call(dy=65536, lddy=64, h=65536, ldh=64, rstd=65536, w=65536, wdt=1, dh=65536, lddh=64, dt=1, rows=4, cols=64,
             dx=65536, lddx=64, dw=65536, ws=65536, ws_bytes=need):
        return lib.lib.nvfp4_rmsnorm_backward(dy, lddy, h, ldh, rstd, w, wdt, dh, lddh, dt, rows, cols, dx, lddx, dw,
                                              ws, ws_bytes, None)

    for k in ("dy", "h", "rstd", "w", "dx", "dw"):
        assert call(**{k: None}) == E["NULL"], k
    assert call(dt=5) == E["ENUM"] and call(wdt=5) == E["ENUM"]
    for k in ("lddy", "ldh", "lddh", "lddx"):
        assert call(**{k: 63}) == E["SHAPE"], k
    assert call(rows=-1) == E["SHAPE"] and call(cols=0) == E["SHAPE"]
    for k in ("dy", "h", "dh", "dx", "w"):
        assert call(**{k: 65537}) == E["ALIGN"], k
    assert call(dw=65538) == E["ALIGN"] and call(ws=65544) == E["ALIGN"]
    assert call(ws=None) == E["WS"] and call(ws_bytes=need - 1) == E["WS"]
    big = 32800
    assert call(cols=big, lddy=big, ldh=big, lddh=big, lddx=big) == E["UNSUP"]


def test_python_refusals(lib):
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError):
        lib.nvfp4_rmsnorm(x, w)                                   # not on a GPU
    with pytest.raises(ValueError):
        lib.nvfp4_rmsnorm(x, torch.ones(63))
    with pytest.raises(TypeError):
        lib.nvfp4_rmsnorm(x.half(), w)
    with pytest.raises(ValueError):
        lib.nvfp4_rmsnorm(x.t(), torch.ones(4))                   # column stride
    with pytest.raises(ValueError):
        lib.nvfp4_rmsnorm(x, w, residual=torch.zeros(4, 32))
    with pytest.raises(TypeError):
        lib.nvfp4_rmsnorm(x, w, residual=torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        lib.nvfp4_rmsnorm_backward(x, x, torch.zeros(3), w)
    with pytest.raises(TypeError):
        lib.nvfp4_rmsnorm_backward(x, x, torch.zeros(4, dtype=torch.float64), w)


# ---------------------------------------------------------------- on the GPU
@pytest.fixture(scope="module")
def nv():
    from parity_utils import require_gpu
    return require_gpu()


def make(seed, rows, cols, dt, ld=None, offset=0):
    """Normal values with a few loud channels; a row stride of ld and a start
    of `offset` elements into the buffer when given."""
    g = np.random.default_rng(seed)
    v = g.standard_normal((rows, cols)) * np.where(g.random(cols) < 0.02, 20.0, 1.0)
    if ld is None:
        return torch.from_numpy(v).to(dt).cuda()
    buf = torch.zeros(rows * ld + offset, dtype=dt, device="cuda")
    view = buf[offset:].view(rows, ld)[:, :cols]
    view.copy_(torch.from_numpy(v).to(dt))
    return view


SIZES = [(1, 32), (1, 7168), (3, 8), (5, 1), (17, 48), (130, 512), (33, 520), (9, 1003), (70, 2048), (4, 5120),
         (2, 8192), (3, 16384), (2, 32768), (2100, 96)]


def check_forward(nv, x, res, w, out, dt, mx_elem):
    hx = P.host(x) + (0.0 if res is None else P.host(res))
    # BF16: a binary32 sum, then one rounding (binary32: the sum alone)
    tol = (P.HALF_STEP[dt] + (P.U if dt == torch.bfloat16 else 0.0)) * np.abs(hx)
    h = P.host(out.h)
    assert (np.abs(h - hx) <= tol).all()
    rstd, y = P.rmsnorm(h, P.host(w), EPS)
    if out.rstd is not None:
        assert (np.abs(P.host(out.rstd) - rstd) <= TOL_RSTD * rstd).all()
    if out.y is not None:
        tol = (TOL_Y + (2.0 ** -8 if dt == torch.bfloat16 else 0.0)) * np.abs(y)
        assert (np.abs(P.host(out.y) - y) <= tol).all()
    if mx_elem is not None:
        r, c = y.shape
        s = out.mx.scales.cpu().numpy().astype(np.int64) - 127
        amax = np.abs(y).reshape(r, c // 32, 32).max(axis=2)
        emax = 8 if mx_elem == nv.NVFP4_MX_E4M3 else 2
        lo, hi = (np.maximum(np.floor(np.log2(np.maximum(amax * f, 1e-300))) - emax, -127) for f in
                  (1 - TOL_Y, 1 + TOL_Y))
        assert ((s >= lo) & (s <= hi)).all()
        v = P.host(nv.nvfp4_mx_dequantize(out.mx, dtype=torch.float32)) / np.repeat(2.0 ** s, 32, axis=1)
        q = y / np.repeat(2.0 ** s, 32, axis=1)
        top, rel, sub = (448.0, 2.0 ** -4, 2.0 ** -10) if emax == 8 else (6.0, 2.0 ** -2, 0.25)
        want = np.clip(q, -top, top)
        assert (np.abs(v - want) <= np.maximum(rel * np.abs(want), sub) + TOL_Y * np.abs(q)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(nv, rows, cols, dtype):
    dt = DT[dtype]
    x, res = make(1, rows, cols, dt), make(2, rows, cols, dt)
    for wdt in (dt, torch.float32):
        w = (1.0 + 0.1 * make(3, 1, cols, torch.float32)[0]).to(wdt)
        for elem in ([nv.NVFP4_MX_E4M3, nv.NVFP4_MX_E2M1] if cols % 32 == 0 else [None]):
            out = nv.nvfp4_rmsnorm(x, w, residual=res, eps=EPS, mx_elem=elem, rstd=True)
            check_forward(nv, x, res, w, out, dt, elem)
        out = nv.nvfp4_rmsnorm(x, w, eps=EPS)
        assert out.h is x and out.rstd is None and out.mx is None
        check_forward(nv, x, None, w, out, dt, None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols,ld,offset", [(96, 97, 1), (1003, 1024, 3), (512, 520, 8), (64, 65, 0)])
def test_strides_and_alignment(nv, cols, ld, offset, dtype):
    dt = DT[dtype]
    x, res = make(4, 37, cols, dt, ld, offset), make(5, 37, cols, dt, ld + 2, 2 * offset)
    w = make(6, 1, cols, dt, cols, offset)[0]
    elem = nv.NVFP4_MX_E4M3 if cols % 32 == 0 else None
    out = nv.nvfp4_rmsnorm(x, w, residual=res, eps=EPS, mx_elem=elem, rstd=True)
    check_forward(nv, x, res, w, out, dt, elem)
    # strided outputs; what lies between their rows stays
    hb, yb = torch.full((37, ld), 7.0, dtype=dt, device="cuda"), torch.full((37, ld), 7.0, dtype=dt, device="cuda")
    o = nv.RMSNormOutput(hb[:, :cols], yb[:, :cols], None, torch.empty(37, device="cuda"))
    nv.nvfp4_rmsnorm(x, w, residual=res, eps=EPS, rstd=True, out=o)
    assert torch.equal(o.h, out.h) and torch.equal(o.y, out.y) and torch.equal(o.rstd, out.rstd)
    assert (hb[:, cols:] == 7).all() and (yb[:, cols:] == 7).all()
    # in place on the residual
    r2 = res.clone()
    o2 = nv.nvfp4_rmsnorm(x, w, residual=r2, eps=EPS, out=nv.RMSNormOutput(r2, torch.empty_like(out.y)))
    assert torch.equal(r2, out.h) and torch.equal(o2.y, out.y)


@pytest.mark.gpu
def test_zero_rows_and_zero_values(nv):
    w = torch.ones(64, device="cuda")
    out = nv.nvfp4_rmsnorm(torch.zeros(0, 64, device="cuda"), w, mx_elem=nv.NVFP4_MX_E4M3, rstd=True)
    assert out.y.shape == (0, 64)
    out = nv.nvfp4_rmsnorm(torch.zeros(3, 64, device="cuda"), w, eps=EPS, mx_elem=nv.NVFP4_MX_E4M3, rstd=True)
    assert (out.y == 0).all() and (out.mx.codes == 0).all() and (out.mx.scales == 0).all()
    assert np.allclose(P.host(out.rstd), 1e3, rtol=TOL_RSTD)
    dx, dw = nv.nvfp4_rmsnorm_backward(torch.zeros(0, 64, device="cuda"), torch.zeros(0, 64, device="cuda"),
                                       torch.zeros(0, device="cuda"), w, dweight=torch.full((64,), 5.0, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_dh", [True, False])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(nv, rows, cols, with_dh, dtype):
    dt = DT[dtype]
    h, dy = make(7, rows, cols, dt), make(8, rows, cols, dt)
    dh = make(9, rows, cols, dt) if with_dh else None
    w = (1.0 + 0.1 * make(10, 1, cols, torch.float32)[0]).to(dt)
    rstd = torch.from_numpy(P.rmsnorm(P.host(h), P.host(w), EPS)[0]).float().cuda()
    dx, dw = nv.nvfp4_rmsnorm_backward(dy, h, rstd, w, dh=dh)
    H, D, R, Wt = P.host(h), P.host(dy), P.host(rstd)[:, None], P.host(w)
    dx64, dw64 = P.rmsnorm_backward(D, H, R[:, 0], Wt, None if dh is None else P.host(dh))
    g, xh = np.abs(D * Wt), np.abs(H * R)
    # the mean: 55 roundings of its terms' absolute sum and 4 more; around it
    # at most 4 roundings of each of the three terms
    mean_abs = (g * xh).mean(axis=1, keepdims=True)
    tol = P.U * (4 * R * g + 63 * R * xh * mean_abs + 2 * np.abs(dx64))
    if dh is not None:
        tol = tol + P.U * 2 * np.abs(P.host(dh))
    tol = tol + (2.0 ** -8 if dt == torch.bfloat16 else 0.0) * (np.abs(dx64) + tol)
    assert (np.abs(P.host(dx) - dx64) <= tol).all()
    # dweight: a group's rows in turn, then its parts by eighths
    groups = nv.nvfp4_rmsnorm_backward_workspace_size(rows, cols) // (4 * cols)
    n = -(-rows // groups) + -(-groups // 8) + 8 + 2
    assert (np.abs(P.host(dw) - dw64) <= n * P.U * (np.abs(D) * xh).sum(axis=0)).all()


@pytest.mark.gpu
def test_backward_against_differences(nv):
    """The kernel's gradients against central differences of the 64-bit
    forward pass in random directions: float32 rounding of the gradients is
    the only error beyond the differences' own."""
    x = make(11, 12, 200, torch.float32)
    w = 1.0 + 0.1 * make(12, 1, 200, torch.float32)[0]
    dy, dh = make(13, 12, 200, torch.float32), make(14, 12, 200, torch.float32)
    out = nv.nvfp4_rmsnorm(x, w, eps=EPS, rstd=True)
    dx, dw = nv.nvfp4_rmsnorm_backward(dy, x, out.rstd, w, dh=dh)
    X, Wt, D, DH = P.host(x), P.host(w), P.host(dy), P.host(dh)

    def loss(a, b):
        return (P.rmsnorm(a, b, EPS)[1] * D).sum() + (a * DH).sum()

    g = np.random.default_rng(15)
    t = 1e-5
    for _ in range(4):
        v, u = g.standard_normal(X.shape), g.standard_normal(Wt.shape)
        got = (P.host(dx) * v).sum()
        assert abs((loss(X + t * v, Wt) - loss(X - t * v, Wt)) / (2 * t) - got) <= 1e-5 * np.abs(P.host(dx) * v).sum()
        got = (P.host(dw) * u).sum()
        assert abs((loss(X, Wt + t * u) - loss(X, Wt - t * u)) / (2 * t) - got) <= 1e-5 * np.abs(P.host(dw) * u).sum()


@pytest.mark.gpu
def test_backward_strides_and_in_place(nv):
    h, dy, dh = (make(s, 41, 99, torch.bfloat16, 105, 3) for s in (16, 17, 18))
    w = make(19, 1, 99, torch.float32)[0]
    rstd = torch.rand(41, device="cuda") + 0.5
    dx, dw = nv.nvfp4_rmsnorm_backward(dy.contiguous(), h.contiguous(), rstd, w, dh=dh.contiguous())
    got, dw2 = nv.nvfp4_rmsnorm_backward(dy, h, rstd, w, dh=dh, dx=dy)
    assert got is dy and torch.equal(dy, dx) and torch.equal(dw, dw2)


@pytest.mark.gpu
def test_offsets_past_32_bits(nv):
    """Two rows over 2^31 elements apart."""
    ld = 2 ** 31 + 32
    bufs = [torch.empty(ld + 96, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    x, res, dh = (b.as_strided((2, 96), (ld, 1)) for b in bufs)
    for i, t in enumerate((x, res, dh)):
        t.copy_(make(30 + i, 2, 96, torch.bfloat16))
    w = torch.ones(96, device="cuda")
    want = nv.nvfp4_rmsnorm(x.contiguous(), w, residual=res.contiguous(), rstd=True)
    grads = nv.nvfp4_rmsnorm_backward(x.contiguous(), want.h, want.rstd, w, dh=dh.contiguous())
    got = nv.nvfp4_rmsnorm(x, w, residual=res, rstd=True, out=nv.RMSNormOutput(res, torch.empty_like(want.y), None,
                                                                             torch.empty_like(want.rstd)))
    assert got.h is res and torch.equal(res, want.h) and torch.equal(got.y, want.y)
    dx, dw = nv.nvfp4_rmsnorm_backward(x, res, got.rstd, w, dh=dh, dx=dh)
    assert torch.equal(dx, grads[0]) and torch.equal(dw, grads[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_row_with_infinity_leaves_the_others(nv, dtype):
    """(The row itself is unspecified.)"""
    x = make(33, 9, 256, DT[dtype])
    w = torch.ones(256, device="cuda")
    want = nv.nvfp4_rmsnorm(x, w, mx_elem=nv.NVFP4_MX_E4M3, rstd=True)
    x2 = x.clone()
    x2[4, 7] = float("inf")
    got = nv.nvfp4_rmsnorm(x2, w, mx_elem=nv.NVFP4_MX_E4M3, rstd=True)
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    for a, b in ((want.y, got.y), (want.rstd, got.rstd), (want.mx.codes, got.mx.codes), (want.mx.scales, got.mx.scales)):
        assert torch.equal(a[keep], b[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(3, 9001), (513, 100), (1100, 2050), (40, 16390), (2049, 640)])
def test_many_rows_and_wide_rows(nv, rows, cols):
    """Row counts around the groups' and widths in which a thread holds
    several chunks, forward and backward, odd strides."""
    for dt in (torch.bfloat16, torch.float32):
        x, res, dh = (make(s, rows, cols, dt, cols + 3, 1) for s in (40, 41, 42))
        w = (1.0 + 0.1 * make(43, 1, cols, torch.float32)[0]).to(dt)
        elem = nv.NVFP4_MX_E2M1 if cols % 32 == 0 else None
        out = nv.nvfp4_rmsnorm(x, w, residual=res, eps=EPS, mx_elem=elem, rstd=True)
        check_forward(nv, x, res, w, out, dt, elem)
        a = nv.nvfp4_rmsnorm_backward(res, x, out.rstd, w, dh=dh)
        b = nv.nvfp4_rmsnorm_backward(res.contiguous(), x.contiguous(), out.rstd, w, dh=dh.contiguous())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        _, dw = P.rmsnorm_backward(P.host(res), P.host(x), P.host(out.rstd), P.host(w), None)
        # (the sums' tolerance as in test_backward)
        groups = nv.nvfp4_rmsnorm_backward_workspace_size(rows, cols) // (4 * cols)
        n = -(-rows // groups) + -(-groups // 8) + 8 + 2
        xh = np.abs(P.host(x) * P.host(out.rstd)[:, None])
        assert (np.abs(P.host(a[1]) - dw) <= n * P.U * (np.abs(P.host(res)) * xh).sum(axis=0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (40, 1003), (9, 5120), (5, 9001), (3, 32768)])
def test_y_is_the_nearest_binary32(nv, rows, cols):
    """Whole numbers up to 1000, whose squares sum in eights without rounding,
    and an eps that is a power of two leave no error before the binary64 part:
    y is within half a step and what a binary32 pair leaves of the product, each
    of its three roundings 2^-24 of a half step."""
    g = np.random.default_rng(50 + cols)
    x = torch.from_numpy(g.integers(-1000, 1001, (rows, cols))).float().cuda()
    w = torch.from_numpy(g.standard_normal(cols)).float().cuda()
    _, y = P.rmsnorm(P.host(x), P.host(w), 2.0 ** -20)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -126))) - 23)
    got = P.host(nv.nvfp4_rmsnorm(x, w, eps=2.0 ** -20).y)
    assert (np.abs(got - y) <= 0.5 * step * (1 + 2.0 ** -20)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_infinite_weight(nv, dtype):
    """y is infinite in its column, of h's sign, and as ever in the others."""
    x = make(34, 6, 256, DT[dtype])
    w = torch.ones(256, device="cuda")
    want = nv.nvfp4_rmsnorm(x, w).y
    w[9], w[200] = float("inf"), float("-inf")
    got = nv.nvfp4_rmsnorm(x, w).y
    assert torch.equal(got[:, 9], torch.sign(x[:, 9]) * float("inf"))
    assert torch.equal(got[:, 200], -torch.sign(x[:, 200]) * float("inf"))
    keep = [c for c in range(256) if c not in (9, 200)]
    assert torch.equal(got[:, keep], want[:, keep])


@pytest.mark.gpu
@pytest.mark.parametrize("elem", ["E4M3", "E2M1"])
def test_codes_at_borders(nv, elem):
    """Codes are those of the exact y, also where its nearest binary32 lies
    halfway between two codes or at a power of two.  Rows of whole numbers with
    rstd's error below 2^-47 (see above); each weight is, to binary32, what puts
    the first row's value at such a place, so that the product falls to either
    side of it by up to 2^-24, and 2^-44 or less in about one of 10^6."""
    code = nv.NVFP4_MX_E4M3 if elem == "E4M3" else nv.NVFP4_MX_E2M1
    g = np.random.default_rng(61)
    cols = 4096
    x = np.abs(g.integers(1, 1001, (2, cols))).astype(np.float64)
    rstd = 1.0 / np.sqrt((x * x).mean(axis=1) + 2.0 ** -20)
    emax, bits = (8, 3) if elem == "E4M3" else (2, 1)
    border = (2 ** (bits + 1) + 2 * g.integers(0, 2 ** bits, cols) + 1) / 2.0 ** (bits + 1)  # halfway in [1, 2)
    border[::32] = np.where(np.arange(cols // 32) % 2, 2.0, 1.75)  # a block's largest: a power of two or below it
    border[1::32] = np.minimum(border[1::32], border[::32] - 0.25)
    border = np.where(np.arange(cols) % 32 == 0, border, 0.5 * border)
    w = torch.from_numpy(border / (x[0] * rstd[0])).float()
    out = nv.nvfp4_rmsnorm(torch.from_numpy(x).float().cuda(), w.cuda(), eps=2.0 ** -20, mx_elem=code)
    y = x * rstd[:, None] * P.host(w)
    amax = np.abs(y).reshape(2, -1, 32).max(axis=2)
    s = np.floor(np.log2(amax)) - emax
    assert np.array_equal(out.mx.scales.cpu().numpy(), (s + 127).astype(np.uint8))
    m = np.abs(y) / np.repeat(2.0 ** s, 32, axis=1)
    low = -6 if elem == "E4M3" else 0
    step = 2.0 ** (np.floor(np.log2(np.maximum(m, 2.0 ** low))) - bits)
    want = np.minimum(np.round(m / step) * step, 448.0 if elem == "E4M3" else 6.0)
    got = P.host(nv.nvfp4_mx_dequantize(out.mx, dtype=torch.float32)) / np.repeat(2.0 ** s, 32, axis=1)
    assert np.array_equal(got, want)
