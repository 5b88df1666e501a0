"""Products of a few rows with 4-bit weights (dense and routed) against the
plain 64-bit forms of moe_plain.py.

Tolerance: the library's for its exact-product GEMMs, 1e-5 sum |x w| of
binary32 accumulation, and half a step of the output's type.  SwiGLU: what
those move it by, and 8 roundings of its own (exponential, sum, quotient, two
products).  A weighted sum adds one rounding a term."""
import ctypes

import numpy as np
import pytest
import torch

import moe_plain as P

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E = dict(OK=0, NULL=1, ENUM=2, SHAPE=3, ALIGN=4, UNSUP=5, WS=6)


# ---------------------------------------------------------------- refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    import bit_block_scaled_quantize_amd.nvfp4 as nv
    return nv


def test_gemv_rejects_bad_arguments(lib):
    def call(x=65536, dt=1, m=4, ldx=64, rows=32, cols=64, mode=0, codes=65536, scales=65537, ts=65536, w=True, y=65536,
             ydt=0, ldy=32, ep=0):
        t = lib.CTensor(codes, scales, ts, rows, cols, mode)
        return lib.lib.nvfp4_gemv(x, dt, m, ldx, ctypes.byref(t) if w else None, y, ydt, ldy, ep, None)

    for kw in (dict(x=None), dict(w=False), dict(codes=None), dict(scales=None), dict(ts=None), dict(y=None)):
        assert call(**kw) == E["NULL"], kw
    for kw in (dict(dt=2), dict(ydt=-1), dict(ep=2), dict(mode=2)):
        assert call(**kw) == E["ENUM"], kw
    for kw in (dict(m=-1), dict(ldx=63), dict(ldy=31), dict(cols=72), dict(mode=1, rows=24), dict(rows=-1),
               dict(ep=1, rows=48), dict(ep=1, rows=33, ldy=64), dict(ep=1, ldy=15)):
        assert call(**kw) == E["SHAPE"], kw
    for kw in (dict(x=65537), dict(dt=0, x=65538), dict(y=65538), dict(codes=65544)):
        assert call(**kw) == E["ALIGN"], kw
    assert call(m=1025) == E["UNSUP"]
    assert call(m=0, x=None, y=None) == E["OK"]
    assert call(rows=0, codes=None, scales=None, y=None, ldy=0) == E["OK"]


def test_mx_gemv_rejects_bad_arguments(lib):
    def call(x=65536, dt=1, m=4, ldx=64, rows=32, cols=64, elem=1, codes=65536, scales=65537, w=True, y=65536, ydt=0,
             ldy=32):
        t = lib.CMXTensor(codes, scales, rows, cols, elem)
        return lib.lib.nvfp4_mx_gemv(x, dt, m, ldx, ctypes.byref(t) if w else None, y, ydt, ldy, None)

    for kw in (dict(x=None), dict(w=False), dict(codes=None), dict(scales=None), dict(y=None)):
        assert call(**kw) == E["NULL"], kw
    for kw in (dict(dt=2), dict(ydt=2), dict(elem=3)):
        assert call(**kw) == E["ENUM"], kw
    for kw in (dict(m=-1), dict(ldx=63), dict(ldy=31), dict(cols=48, ldx=64), dict(rows=-1)):
        assert call(**kw) == E["SHAPE"], kw
    assert call(codes=65544) == E["ALIGN"] and call(y=65538) == E["ALIGN"]
    assert call(elem=0) == E["UNSUP"] and call(m=1025) == E["UNSUP"]
    assert call(m=0, x=None, y=None) == E["OK"]


def test_expert_gemv_rejects_bad_arguments(lib):
    need = lib.nvfp4_expert_gemv_workspace_size(4, 2, 32)
    assert need == 4 * 2 * 32 * 4
    for bad in ((-1, 2, 32), (4, 0, 32), (4, 2, -1), (1025, 1, 32)):
        assert lib.nvfp4_expert_gemv_workspace_size(*bad) == 0

    def call(x=65536, dt=1, xr=4, ldx=64, ids=65536, T=4, k=2, rows=96, cols=64, mode=0, experts=3, weights=65536, y=65536,
             ydt=0, ldy=32, ep=0, ws=65536, ws_bytes=need):
        t = lib.CTensor(65536, 65537, 65536, rows, cols, mode)
        return lib.lib.nvfp4_expert_gemv(x, dt, xr, ldx, ids, T, k, ctypes.byref(t), experts, weights, y, ydt, ldy, ep, ws,
                                         ws_bytes, None)

    for kw in (dict(x=None), dict(ids=None), dict(y=None)):
        assert call(**kw) == E["NULL"], kw
    for kw in (dict(dt=2), dict(ydt=2), dict(ep=2), dict(mode=-1)):
        assert call(**kw) == E["ENUM"], kw
    for kw in (dict(xr=5), dict(T=-1), dict(k=0), dict(experts=0), dict(experts=5), dict(mode=1, rows=72), dict(ldx=63),
               dict(ldy=31), dict(ep=1, rows=3 * 48)):
        assert call(**kw) == E["SHAPE"], kw
    for kw in (dict(x=65537), dict(ids=65538), dict(weights=65537), dict(y=65538), dict(ws=65544)):
        assert call(**kw) == E["ALIGN"], kw
    assert call(T=513, xr=513) == E["UNSUP"]
    assert call(ws=None) == E["WS"] and call(ws_bytes=need - 1) == E["WS"]
    assert call(T=0, xr=0, x=None, ids=None, y=None, ws=None) == E["OK"]


@pytest.mark.parametrize("rows", [2 ** 29, 2 ** 30, 2 ** 33])  # (of SwiGLU a multiple of 32)
def test_more_rows_than_a_grid_holds(lib, rows):
    """More than 2^29 - 32 rows of a matrix are refused: the workgroups of 256 threads
    for each 32 of them would be more than one grid's 2^32 threads."""
    def status(n):
        w = lib.CTensor(65536, 65537, 65536, n, 16, 0)
        yield lib.lib.nvfp4_gemv(65536, 1, 5, 16, ctypes.byref(w), 65536, 1, n, 0, None)
        yield lib.lib.nvfp4_gemv(65536, 1, 5, 16, ctypes.byref(w), 65536, 1, n, 1, None)
        m = lib.CMXTensor(65536, 65537, n, 32, 1)
        yield lib.lib.nvfp4_mx_gemv(65536, 1, 5, 32, ctypes.byref(m), 65536, 1, n, None)
        w = lib.CTensor(65536, 65537, 65536, 2 * n, 16, 0)
        yield lib.lib.nvfp4_expert_gemv(65536, 1, 5, 16, 65536, 5, 1, ctypes.byref(w), 2, None, 65536, 1, n, 0, None, 0,
                                        None)

    assert set(status(rows)) == {E["UNSUP"]}


def test_python_refusals(lib):
    x = torch.zeros(2, 64)
    w = lib.NVFP4Tensor.empty(32, 64, device="cpu")
    with pytest.raises(ValueError):
        lib.nvfp4_gemv(x, w)                                        # not on a GPU
    with pytest.raises(ValueError):
        lib.nvfp4_gemv(x[:, :32], w)
    with pytest.raises(TypeError):
        lib.nvfp4_gemv(x.half(), w)
    with pytest.raises(ValueError):
        lib.nvfp4_gemv(x, lib.NVFP4Tensor(w.codes[:16], w.scales, w.tensor_scale, 32, 64))
    with pytest.raises(TypeError):
        lib.nvfp4_gemv(x, lib.NVFP4Tensor(w.codes.view(torch.int8), w.scales, w.tensor_scale, 32, 64))
    with pytest.raises(ValueError):
        lib.nvfp4_gemv(x, w, out=torch.zeros(2, 31))
    with pytest.raises(ValueError):
        lib.nvfp4_mx_gemv(x, lib.MXTensor.empty(32, 64, device="cpu"))   # E4M3 elements
    ids = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        lib.nvfp4_expert_gemv(torch.zeros(3, 64), ids, w, 1)
    with pytest.raises(TypeError):
        lib.nvfp4_expert_gemv(x, ids.long(), w, 1)
    with pytest.raises(ValueError):
        lib.nvfp4_expert_gemv(x, ids, w, 2)                         # one tensor scale for two matrices


# ---------------------------------------------------------------- on the GPU
@pytest.fixture(scope="module")
def nv():
    from parity_utils import require_gpu
    return require_gpu()


def make_x(seed, rows, cols, dt, ld=None, offset=0):
    g = np.random.default_rng(seed)
    v = g.standard_normal((rows, cols)) * np.where(g.random(cols) < 0.02, 20.0, 1.0)
    if ld is None:
        return torch.from_numpy(v).to(dt).cuda()
    buf = torch.zeros(rows * ld + offset, dtype=dt, device="cuda")
    view = buf[offset:].view(rows, ld)[:, :cols]
    view.copy_(torch.from_numpy(v).to(dt))
    return view


def make_w(nv, seed, rows, cols, fmt, experts=1):
    """Any codes and any ordinary scales: every value of the format."""
    g = np.random.default_rng(seed)
    dev = dict(device="cuda")
    codes = torch.from_numpy(g.integers(0, 256, (rows, cols // 2), dtype=np.uint8)).to(**dev)
    if fmt == "mx":
        return nv.MXTensor(codes, torch.from_numpy(g.integers(118, 130, (rows, cols // 32), dtype=np.uint8)).to(**dev),
                           rows, cols, nv.NVFP4_MX_E2M1)
    two_d = fmt == "nv2d"
    sc = g.integers(0, 127, (rows // 16 if two_d else rows, cols // 16), dtype=np.uint8)
    ts = torch.from_numpy(np.exp(g.standard_normal(experts)).astype(np.float32)).to(**dev)
    return nv.NVFP4Tensor(codes, torch.from_numpy(sc).to(**dev), ts, rows, cols,
                          nv.NVFP4_SCALE_2D if two_d else nv.NVFP4_SCALE_1D)


def call(nv, x, w, **kw):
    return nv.nvfp4_mx_gemv(x, w, **kw) if isinstance(w, nv.MXTensor) else nv.nvfp4_gemv(x, w, **kw)


def values(nv, w, experts=1):
    return P.mx_weight(w) if isinstance(w, nv.MXTensor) else P.nvfp4_weight(w, experts)


def close(got, want, tol):
    # half a step of the type: relative, or that of its subnormals
    half, sub = (2.0 ** -8, 2.0 ** -134) if got.dtype == torch.bfloat16 else (P.U, 2.0 ** -150)
    tol = tol + np.maximum(half * (np.abs(want) + tol), sub)
    bad = np.argwhere(~(np.abs(P.host(got) - want) <= tol))
    assert bad.size == 0, f"{len(bad)} off, first at {bad[0].tolist()}"


def check(nv, x, w, out=None, swiglu=False, out_dtype=None):
    W, X = values(nv, w), P.host(x)
    want, tol = X @ W.T, 1e-5 * (np.abs(X) @ np.abs(W).T)
    kw = {}
    if swiglu:
        want, tol = P.swiglu(want, tol)
        tol = tol + 8 * P.U * np.abs(want)
        kw["epilogue"] = nv.NVFP4_EPI_SWIGLU
    y = call(nv, x, w, out=out, out_dtype=out_dtype, **kw)
    assert y.dtype == (out.dtype if out is not None else out_dtype or x.dtype)
    close(y, want, tol)
    return y


SIZES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (3, 1000, 1056), (5, 33, 128), (15, 64, 160), (16, 48, 288), (17, 40, 512),
         (33, 24, 1024), (1, 4096, 2048), (8, 300, 4128), (4, 70, 20480), (100, 130, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["nv1d", "nv2d", "mx"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemv(nv, m, n, k, fmt, dtype):
    if fmt == "nv2d":
        n = -(-n // 16) * 16
    if fmt != "mx" and m % 2:
        k -= 16  # (odd blocks of 16)
    x = make_x(m + n, m, k, DT[dtype])
    w = make_w(nv, n + k, n, k, fmt)
    y = check(nv, x, w)
    assert torch.equal(y, call(nv, x, w))  # repeats bit for bit
    check(nv, x, w, out_dtype=torch.float32 if dtype == "bf16" else torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["nv1d", "nv2d"])
@pytest.mark.parametrize("m,f,k", [(1, 16, 32), (3, 48, 400), (16, 112, 1040), (18, 512, 256)])
def test_swiglu(nv, m, f, k, fmt, dtype):
    x = 0.05 * make_x(m, m, k, DT[dtype])
    w = make_w(nv, f, 2 * f, k, fmt)
    w.tensor_scale.fill_(0.01)
    check(nv, x, w, swiglu=True)
    check(nv, x, w, swiglu=True, out_dtype=torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_code_and_scale_exactly(nv, dtype):
    """Row n holds scale byte n % 127 and every pair of codes over its columns;
    one-hot rows of x pick single weights, whose product is exact."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").roll(37).repeat(127, 1)
    scales = torch.arange(127, dtype=torch.uint8, device="cuda").view(-1, 1).repeat(1, 32)
    w = nv.NVFP4Tensor(codes, scales, torch.tensor([0.375], device="cuda"), 127, 512)
    x = torch.eye(512, device="cuda").to(DT[dtype])
    y = nv.nvfp4_gemv(x, w, out_dtype=torch.float32)
    assert np.array_equal(P.host(y), P.nvfp4_weight(w).T)
    # MX: every scale byte with a normal weight
    scales = torch.arange(3, 253, dtype=torch.uint8, device="cuda").view(-1, 1).repeat(1, 16)
    w = nv.MXTensor(codes[:1].repeat(250, 1), scales, 250, 512, nv.NVFP4_MX_E2M1)
    y = nv.nvfp4_mx_gemv(x, w, out_dtype=torch.float32)
    assert np.array_equal(P.host(y), P.mx_weight(w).T)
    # zero blocks: byte 0
    w.scales.zero_()
    w.codes.zero_()
    assert (nv.nvfp4_mx_gemv(x, w) == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [4, 16])
@pytest.mark.parametrize("byte", [0, 1, 2, 3, 252, 253, 254])
def test_mx_scale_bytes_at_the_ends(nv, byte, rows):
    """Normal weights are exact, smaller ones exact or zero; of the largest scales
    the weights that binary32 holds (the others are infinite)."""
    top = {253: 3, 254: 2}.get(byte, 7)  # code of the largest magnitude below 2^128 / 2^(byte - 127)
    low = np.arange(256) & 7
    codes = np.arange(256)[(low <= top) & (np.arange(256) >> 4 & 7 <= top)][:64]
    codes = torch.from_numpy(np.resize(codes, 64).astype(np.uint8)).cuda().repeat(16, 1)
    w = nv.MXTensor(codes, torch.full((16, 4), byte, dtype=torch.uint8, device="cuda"), 16, 128, nv.NVFP4_MX_E2M1)
    want = P.mx_weight(w).T
    small = np.abs(want) < 2.0 ** -126
    for dt in DT.values():
        x = torch.eye(128, device="cuda").to(dt)
        got = np.concatenate([P.host(nv.nvfp4_mx_gemv(x[i:i + rows], w, out_dtype=torch.float32)) for i in range(0, 128, rows)])
        assert (((got == want) | (small & (got == 0)))).all()


@pytest.mark.gpu
def test_binary32_x_is_not_rounded(nv):
    """x values that need all 24 bits: each product with a power of two is exact."""
    g = np.random.default_rng(2)
    v = (g.integers(2 ** 23, 2 ** 24, 64).astype(np.float64) * 2.0 ** g.integers(-40, 20, 64)).astype(np.float32)
    x = torch.diag(torch.from_numpy(v)).cuda()
    codes = torch.full((16, 32), 0x22, dtype=torch.uint8, device="cuda")  # all ones
    w = nv.NVFP4Tensor(codes, torch.full((16, 4), 0x38, dtype=torch.uint8, device="cuda"), torch.ones(1, device="cuda"), 16, 64)
    y = nv.nvfp4_gemv(x, w)
    assert torch.equal(y, torch.from_numpy(v).cuda().view(-1, 1).repeat(1, 16))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["nv1d", "nv2d", "mx"])
@pytest.mark.parametrize("ld,offset", [(321, 1), (323, 3), (328, 8)])
def test_strides_and_alignment(nv, ld, offset, fmt, dtype):
    x = make_x(20, 7, 320, DT[dtype], ld, offset)
    w = make_w(nv, 21, 80, 320, fmt)
    if fmt != "mx":  # scale bytes at any address
        buf = torch.zeros(w.scales.numel() + 3, dtype=torch.uint8, device="cuda")
        sc = buf[3:].view(w.scales.shape)
        sc.copy_(w.scales)
        w.scales = sc
    y = check(nv, x, w)
    assert torch.equal(y, call(nv, x.contiguous(), w))
    buf = torch.full((7, 91), 7.0, dtype=DT[dtype], device="cuda")
    check(nv, x, w, out=buf[:, 5:85])
    assert torch.equal(buf[:, 5:85], y) and (buf[:, :5] == 7).all() and (buf[:, 85:] == 7).all()


@pytest.mark.gpu
def test_empty(nv):
    w = make_w(nv, 22, 48, 64, "nv1d")
    assert nv.nvfp4_gemv(torch.zeros(0, 64, device="cuda"), w).shape == (0, 48)
    w0 = nv.NVFP4Tensor.empty(0, 64)
    assert nv.nvfp4_gemv(torch.zeros(3, 64, device="cuda"), w0).shape == (3, 0)
    wk = nv.NVFP4Tensor.empty(48, 0)
    y = nv.nvfp4_gemv(torch.zeros(3, 0, device="cuda"), wk, out=torch.full((3, 48), 5.0, device="cuda"))
    assert (y == 0).all()
    ids = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert nv.nvfp4_expert_gemv(torch.zeros(0, 64, device="cuda"), ids, w, 1).shape == (0, 48)


def expert_reference(nv, x, ids, w, experts, swiglu):
    """Products of all assignments and their tolerances."""
    T, k = ids.shape
    X, I = P.host(x), ids.cpu().numpy()
    W = values(nv, w, experts).reshape(experts, -1, w.cols)
    X = np.repeat(X, k, axis=0) if X.shape[0] == T and k > 1 else X
    want = np.zeros((T * k, W.shape[1]))
    tol = np.zeros_like(want)
    for a, e in enumerate(I.reshape(-1)):
        if 0 <= e < experts:
            want[a], tol[a] = W[e] @ X[a], 1e-5 * (np.abs(W[e]) @ np.abs(X[a]))
    if swiglu:
        want, tol = P.swiglu(want, tol)
        tol = tol + 8 * P.U * np.abs(want)
    return want, tol


EXPERT_SIZES = [  # tokens, top_k, experts, N, K
    (1, 1, 1, 32, 16), (1, 4, 32, 96, 272), (4, 4, 32, 224, 2048), (8, 2, 3, 64, 128), (40, 2, 4, 64, 144),
    (3, 5, 8, 32, 1040), (128, 8, 20, 32, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["nv1d", "nv2d"])
@pytest.mark.parametrize("T,k,experts,n,K", EXPERT_SIZES)
def test_expert_gemv(nv, T, k, experts, n, K, fmt, dtype):
    g = np.random.default_rng(T + K)
    w = make_w(nv, n, experts * n, K, fmt, experts)
    ids = torch.from_numpy(np.stack([g.permutation(max(experts, k))[:k] for _ in range(T)]).astype(np.int32)).cuda()
    wt = torch.from_numpy(g.random((T, k)).astype(np.float32)).cuda()
    for per_assignment in (False, True):
        x = 0.05 * make_x(30, T * k if per_assignment else T, K, DT[dtype])
        for swiglu in (False, True):
            ep = nv.NVFP4_EPI_SWIGLU if swiglu else nv.NVFP4_EPI_NONE
            want, tol = expert_reference(nv, x, ids, w, experts, swiglu)
            close(nv.nvfp4_expert_gemv(x, ids, w, experts, epilogue=ep), want, tol)
            v = P.host(wt).reshape(-1, 1)
            # (a term is rounded as a product and in up to k sums, subnormals by half their step)
            rows = (np.abs(v) * tol + np.maximum(2 * k * P.U * np.abs(v * want), 2.0 ** -149)).reshape(T, k, -1)
            at = (v * want).reshape(T, k, -1)
            y = nv.nvfp4_expert_gemv(x, ids, w, experts, weights=wt, epilogue=ep)
            close(y, at.sum(axis=1), rows.sum(axis=1))
            assert torch.equal(y, nv.nvfp4_expert_gemv(x, ids, w, experts, weights=wt, epilogue=ep))


@pytest.mark.gpu
def test_expert_gemv_foreign_and_repeated_ids(nv):
    """An index out of range is no expert; one that a token names twice counts
    twice."""
    w = make_w(nv, 40, 3 * 48, 160, "nv1d", 3)
    ids = torch.tensor([[0, -1], [3, 2], [1, 1], [7, -9]], dtype=torch.int32, device="cuda")
    wt = torch.tensor([[0.5, 2.0], [1.0, 0.25], [0.75, 0.125], [1.0, 1.0]], device="cuda")
    for rows in (4, 8):
        x = make_x(41, rows, 160, torch.bfloat16)
        want, tol = expert_reference(nv, x, ids, w, 3, False)
        close(nv.nvfp4_expert_gemv(x, ids, w, 3, out=torch.full((8, 48), float("nan"), device="cuda")), want, tol)
        v = P.host(wt).reshape(-1, 1)
        y = nv.nvfp4_expert_gemv(x, ids, w, 3, weights=wt, out=torch.full((4, 48), float("nan"), device="cuda"))
        close(y, (v * want).reshape(4, 2, -1).sum(axis=1), (np.abs(v) * (tol + 4 * P.U * np.abs(want))).reshape(4, 2, -1).sum(axis=1))
        assert (y[3] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("hole", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_weights_without_an_expert(nv, hole):
    """Whatever weight an assignment without an expert has, it adds nothing."""
    w = make_w(nv, 42, 3 * 48, 160, "nv2d", 3)
    ids = torch.tensor([[0, -1, 2], [3, 2, 1], [1, 0, 9], [7, -9, 3]], dtype=torch.int32, device="cuda")
    wt = torch.rand(4, 3, generator=torch.Generator().manual_seed(43)).cuda()
    x = make_x(44, 4, 160, torch.bfloat16)
    want = nv.nvfp4_expert_gemv(x, ids, w, 3, weights=wt)
    holes = torch.where((ids >= 0) & (ids < 3), wt, torch.full_like(wt, hole))
    got = nv.nvfp4_expert_gemv(x, ids, w, 3, weights=holes)
    assert torch.equal(got, want) and (got[3] == 0).all()


@pytest.mark.gpu
def test_offsets_past_32_bits(nv):
    """A stack of experts of over 2^32 bytes of codes: its last one."""
    experts, n, K = 300, 2048, 14336
    codes = torch.zeros((experts * n, K // 2), dtype=torch.uint8, device="cuda")
    last = make_w(nv, 50, n, K, "nv2d")
    codes[-n:] = last.codes
    scales = torch.zeros((experts * n // 16, K // 16), dtype=torch.uint8, device="cuda")
    scales[-n // 16:] = last.scales
    ts = torch.ones(experts, device="cuda")
    ts[-1:] = last.tensor_scale
    w = nv.NVFP4Tensor(codes, scales, ts, experts * n, K, nv.NVFP4_SCALE_2D)
    x = make_x(51, 2, K, torch.bfloat16)
    ids = torch.full((2, 1), experts - 1, dtype=torch.int32, device="cuda")
    assert torch.equal(nv.nvfp4_expert_gemv(x, ids, w, experts), nv.nvfp4_gemv(x, last))
    check(nv, x, last)


@pytest.mark.gpu
def test_streams_and_graphs(nv):
    """On a stream of the caller's, and captured: replays with new inputs give
    what eager calls give."""
    w, wd = make_w(nv, 60, 4 * 64, 160, "nv2d", 4), make_w(nv, 61, 96, 160, "mx")
    ids = torch.tensor([[0, 3], [3, 1], [2, 0]], dtype=torch.int32, device="cuda")
    wt = torch.rand(3, 2, device="cuda")
    x = make_x(62, 3, 160, torch.bfloat16)

    def run(stream=None):
        return (nv.nvfp4_expert_gemv(x, ids, w, 4, weights=wt, stream=stream), nv.nvfp4_mx_gemv(x, wd, stream=stream))

    s = torch.cuda.Stream()
    want = run()
    s.wait_stream(torch.cuda.current_stream())
    got = run(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for seed in range(3):
        x.copy_(make_x(63 + seed, 3, 160, torch.bfloat16))
        ids.copy_((ids + 1) % 4)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(run(), out))
