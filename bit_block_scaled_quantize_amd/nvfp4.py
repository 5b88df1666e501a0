"""Thin binding of libnvfp4.so (include/nvfp4.h): ctypes, and for the operators
of a mixture-of-experts block and of the 4-bit key/value cache the compiled
module _native.

Argument marshalling only: every step of quantize / dequantize / GEMM runs in
the HIP kernels behind the C ABI.  PyTorch supplies device memory (output
tensors are allocated with torch) and the current HIP stream.  If the built
library is missing, importing this module raises -- there is no fallback;
without the compiled module the operators that need it raise.
"""
import contextlib
import ctypes
import functools
import importlib
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")

# enums (include/nvfp4.h)
NVFP4_OK = 0
NVFP4_F32, NVFP4_BF16 = 0, 1
NVFP4_ROW_1D, NVFP4_COL_1D, NVFP4_ROW_COL_1D, NVFP4_BLK_2D = 0, 1, 2, 3
NVFP4_RNE, NVFP4_SR = 0, 1
NVFP4_EPI_NONE, NVFP4_EPI_SWIGLU = 0, 1
NVFP4_SCALE_1D, NVFP4_SCALE_2D = 0, 1
NVFP4_MX_E4M3, NVFP4_MX_E2M1 = 0, 1
NVFP4_MX_ACC_NATIVE, NVFP4_MX_ACC_EXACT = 0, 1
NVFP4_ROUTE_SOFTMAX, NVFP4_ROUTE_SIGMOID = 0, 1
NVFP4_GROUP_MAX, NVFP4_GROUP_TOP2 = 0, 1
NVFP4_KV_NVFP4, NVFP4_KV_MXFP4 = 0, 1

EXPORTED = ["nvfp4_quantize_workspace_size", "nvfp4_quantize", "nvfp4_quantize_noalloc", "nvfp4_requantize",
            "nvfp4_dequantize",
            "nvfp4_gemm", "nvfp4_gemm_workspace_size", "nvfp4_grouped_gemm", "nvfp4_mx_quantize", "nvfp4_mx_dequantize", "nvfp4_mx_gemm",
            "nvfp4_mx_gemm_workspace_size",
            "nvfp4_rmsnorm", "nvfp4_rmsnorm_backward", "nvfp4_rmsnorm_backward_workspace_size",
            "nvfp4_route", "nvfp4_route_workspace_size", "nvfp4_route_backward",
            "nvfp4_gemv", "nvfp4_mx_gemv", "nvfp4_expert_gemv", "nvfp4_expert_gemv_workspace_size",
            "nvfp4_kv_append", "nvfp4_kv_gather", "nvfp4_kv_attention", "nvfp4_kv_attention_workspace_size",
            "nvfp4_status_string", "nvfp4_version"]


class CTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("scale_mode", ctypes.c_int32)]


class CMXTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("elem", ctypes.c_int32)]


class CQuantOpts(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("round", ctypes.c_int32), ("sr_seed", ctypes.c_uint64),
                ("hadamard", ctypes.c_int32), ("hadamard_seed", ctypes.c_uint64),
                ("amax_in", ctypes.c_void_p), ("amax_out", ctypes.c_void_p)]


class CRouteOpts(ctypes.Structure):
    _fields_ = [("top_k", ctypes.c_int32), ("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_score", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("bias", ctypes.c_void_p)]


class CKVCache(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


class CKVPlan(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64), ("width", ctypes.c_int64),
                ("lengths", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("seqs", ctypes.c_int64),
                ("rows", ctypes.c_int64)]


class CKVRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class CKVRope(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run bit_block_scaled_quantize_amd/build.py "
                          "(there is no non-HIP fallback)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    L.nvfp4_quantize_workspace_size.argtypes = [i64, i64, ctypes.POINTER(CQuantOpts)]
    L.nvfp4_quantize_workspace_size.restype = sz
    L.nvfp4_quantize.argtypes = [vp, i32, i64, i64, i64, ctypes.POINTER(CQuantOpts),
                                 ctypes.POINTER(CTensor), vp, sz, vp]
    L.nvfp4_quantize.restype = i32
    L.nvfp4_quantize_noalloc.argtypes = [vp, i32, i64, i64, i64, ctypes.POINTER(CQuantOpts),
                                         ctypes.POINTER(CTensor), vp]
    L.nvfp4_quantize_noalloc.restype = i32
    L.nvfp4_dequantize.argtypes = [ctypes.POINTER(CTensor), vp, i32, i64, vp]
    L.nvfp4_dequantize.restype = i32
    L.nvfp4_requantize.argtypes = [ctypes.POINTER(CTensor), ctypes.POINTER(CQuantOpts),
                                   ctypes.POINTER(CTensor), vp, sz, vp]
    L.nvfp4_requantize.restype = i32
    L.nvfp4_gemm.argtypes = [ctypes.POINTER(CTensor), ctypes.POINTER(CTensor), vp, i32, i64, i32, vp, sz, vp]
    L.nvfp4_gemm.restype = i32
    L.nvfp4_gemm_workspace_size.argtypes = [ctypes.POINTER(CTensor), ctypes.POINTER(CTensor), i32, i32]
    L.nvfp4_gemm_workspace_size.restype = sz
    L.nvfp4_grouped_gemm.argtypes = [i32, ctypes.POINTER(CTensor), vp, ctypes.POINTER(CTensor), vp,
                                     i32, i64, i32, vp, vp, sz, vp]
    L.nvfp4_grouped_gemm.restype = i32
    L.nvfp4_mx_quantize.argtypes = [vp, i32, i64, i64, i64, i32, i32, ctypes.c_uint64,
                                    ctypes.POINTER(CMXTensor), vp]
    L.nvfp4_mx_quantize.restype = i32
    L.nvfp4_mx_dequantize.argtypes = [ctypes.POINTER(CMXTensor), vp, i32, i64, vp]
    L.nvfp4_mx_dequantize.restype = i32
    L.nvfp4_mx_gemm.argtypes = [ctypes.POINTER(CMXTensor), ctypes.POINTER(CMXTensor), vp, i32, i64, i32, vp, sz, vp]
    L.nvfp4_mx_gemm.restype = i32
    L.nvfp4_mx_gemm_workspace_size.argtypes = [ctypes.POINTER(CMXTensor), ctypes.POINTER(CMXTensor), i32, i32]
    L.nvfp4_mx_gemm_workspace_size.restype = sz
    L.nvfp4_rmsnorm.argtypes = [vp, i64, vp, i64, vp, i32, i32, i64, i64, ctypes.c_float, vp, i64, vp, i64,
                                ctypes.POINTER(CMXTensor), vp, vp]
    L.nvfp4_rmsnorm.restype = i32
    L.nvfp4_rmsnorm_backward_workspace_size.argtypes = [i64, i64]
    L.nvfp4_rmsnorm_backward_workspace_size.restype = sz
    L.nvfp4_rmsnorm_backward.argtypes = [vp, i64, vp, i64, vp, vp, i32, vp, i64, i32, i64, i64, vp, i64, vp, vp, sz, vp]
    L.nvfp4_rmsnorm_backward.restype = i32
    L.nvfp4_route_workspace_size.argtypes = [i64, i64]
    L.nvfp4_route_workspace_size.restype = sz
    L.nvfp4_route.argtypes = [vp, i32, i64, i64, i64, ctypes.POINTER(CRouteOpts), vp, vp, vp, vp, vp, vp, sz, vp]
    L.nvfp4_route.restype = i32
    L.nvfp4_route_backward.argtypes = [vp, vp, i32, i64, i64, i64, vp, i32, i32, i32, vp, i64, vp, i64, vp]
    L.nvfp4_route_backward.restype = i32
    L.nvfp4_gemv.argtypes = [vp, i32, i64, i64, ctypes.POINTER(CTensor), vp, i32, i64, i32, vp]
    L.nvfp4_gemv.restype = i32
    L.nvfp4_mx_gemv.argtypes = [vp, i32, i64, i64, ctypes.POINTER(CMXTensor), vp, i32, i64, vp]
    L.nvfp4_mx_gemv.restype = i32
    L.nvfp4_expert_gemv_workspace_size.argtypes = [i64, i32, i64]
    L.nvfp4_expert_gemv_workspace_size.restype = sz
    L.nvfp4_expert_gemv.argtypes = [vp, i32, i64, i64, vp, i64, i32, ctypes.POINTER(CTensor), i32, vp, vp, i32, i64, i32,
                                    vp, sz, vp]
    L.nvfp4_expert_gemv.restype = i32
    kv = [ctypes.POINTER(t) for t in (CKVRows, CKVCache, CKVPlan, CKVRope)]
    L.nvfp4_kv_append.argtypes = [kv[0], kv[0], i32, kv[1], kv[2], kv[3], kv[0], i32, kv[0], vp]
    L.nvfp4_kv_append.restype = i32
    L.nvfp4_kv_gather.argtypes = [kv[1], kv[2], kv[0], kv[0], i32, vp]
    L.nvfp4_kv_gather.restype = i32
    L.nvfp4_kv_attention_workspace_size.argtypes = [i64, i64, i32, i32, i32, i32]
    L.nvfp4_kv_attention_workspace_size.restype = sz
    L.nvfp4_kv_attention.argtypes = [kv[0], i32, i32, kv[1], kv[2], ctypes.c_float, i64, kv[0], vp, vp, sz, vp]
    L.nvfp4_kv_attention.restype = i32
    L.nvfp4_status_string.argtypes = [i32]
    L.nvfp4_status_string.restype = ctypes.c_char_p
    L.nvfp4_version.argtypes = []
    L.nvfp4_version.restype = i32
    return L


lib = _load()


class _NoBinding:
    """In place of _native where it does not load: the operators that go through
    it raise what kept it from loading, the others run."""

    def __init__(self, cause):
        self._cause = cause

    def __getattr__(self, name):
        built = os.path.exists(os.path.join(_HERE, "_native.so"))
        raise ImportError(f"the compiled binding _native.so {'does not load' if built else 'is not built'} "
                          f"({self._cause}); run bit_block_scaled_quantize_amd/build.py") from self._cause


try:
    _native = importlib.import_module("._native", __package__)  # (linked against the library just loaded)
except ImportError as e:
    _native = _NoBinding(e)


class NVFP4Error(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({lib.nvfp4_status_string(status).decode()})")


def _check(fn, status):
    if status != NVFP4_OK:
        raise NVFP4Error(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _on(stream):
    """Context in which a call's outputs and workspace are allocated: the
    stream the kernels run on.  torch's caching allocator hands a freed block
    back only to later allocations on the stream it was allocated on, so a
    workspace released when the call returns cannot be reused by other work
    while the kernels on `stream` still read it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _launches_on_stream(fn):
    """Run the binding function fn with `stream` (keyword) as torch's current
    stream, so that everything it allocates belongs to that stream."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with _on(stream):
            return fn(*args, stream=stream, **kw)
    return call


def _dtype_code(dt):
    if dt == torch.float32:
        return NVFP4_F32
    if dt == torch.bfloat16:
        return NVFP4_BF16
    raise TypeError(f"unsupported dtype {dt}")


@dataclass
class NVFP4Tensor:
    """codes [rows, cols/2] uint8, scales uint8 ([rows, cols/16] or
    [rows/16, cols/16]), tensor_scale float32 [1] (or [G] for grouped
    weights) -- all device tensors."""
    codes: torch.Tensor
    scales: torch.Tensor
    tensor_scale: torch.Tensor
    rows: int
    cols: int
    scale_mode: int = NVFP4_SCALE_1D

    def c(self):
        return CTensor(self.codes.data_ptr(), self.scales.data_ptr(), self.tensor_scale.data_ptr(),
                       self.rows, self.cols, self.scale_mode)

    @staticmethod
    def empty(rows, cols, scale_mode=NVFP4_SCALE_1D, device="cuda", n_scales=1):
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        if scale_mode == NVFP4_SCALE_2D:
            scales = torch.empty((rows // 16, cols // 16), dtype=torch.uint8, device=device)
        else:
            scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=device)
        ts = torch.empty((n_scales,), dtype=torch.float32, device=device)
        return NVFP4Tensor(codes, scales, ts, rows, cols, scale_mode)


def nvfp4_quantize_workspace_size(rows, cols, amax_in=None):
    o = CQuantOpts(0, 0, 0, 0, 0, None if amax_in is None else amax_in.data_ptr(), None)
    return int(lib.nvfp4_quantize_workspace_size(rows, cols, ctypes.byref(o)))


@_launches_on_stream
def nvfp4_quantize(x, layout=NVFP4_ROW_1D, round=NVFP4_RNE, sr_seed=0, hadamard=False,
                   hadamard_seed=0, amax_in=None, out=None, workspace=None, amax_out=None,
                   stream=None):
    """Quantize a 2-D device tensor (float32 or bfloat16, unit column stride).

    Returns an NVFP4Tensor, or (row, col) for NVFP4_ROW_COL_1D.  `out` may
    pass preallocated outputs (one NVFP4Tensor, or a pair for ROW_COL);
    `amax_out` (float32 device tensor) receives the tensor amax used."""
    assert x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else max(cols, x.stride(0))
    dev = x.device
    if out is None:
        if layout == NVFP4_COL_1D:
            outs = [NVFP4Tensor.empty(cols, rows, NVFP4_SCALE_1D, dev)]
        elif layout == NVFP4_BLK_2D:
            outs = [NVFP4Tensor.empty(rows, cols, NVFP4_SCALE_2D, dev)]
        elif layout == NVFP4_ROW_COL_1D:
            outs = [NVFP4Tensor.empty(rows, cols, NVFP4_SCALE_1D, dev),
                    NVFP4Tensor.empty(cols, rows, NVFP4_SCALE_1D, dev)]
        else:
            outs = [NVFP4Tensor.empty(rows, cols, NVFP4_SCALE_1D, dev)]
    else:
        outs = list(out) if isinstance(out, (list, tuple)) else [out]
    arr = (CTensor * 2)()
    for i, t in enumerate(outs):
        arr[i] = t.c()
    opts = CQuantOpts(layout, round, sr_seed, int(bool(hadamard)), hadamard_seed,
                      None if amax_in is None else amax_in.data_ptr(),
                      None if amax_out is None else amax_out.data_ptr())
    need = int(lib.nvfp4_quantize_workspace_size(rows, cols, ctypes.byref(opts)))
    if workspace is None and need:
        workspace = torch.empty((need + 15) // 16 * 4, dtype=torch.float32, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.nvfp4_quantize(ctypes.c_void_p(x.data_ptr()), _dtype_code(x.dtype), rows, cols, ld,
                            ctypes.byref(opts), arr, _ptr(workspace), ws_bytes, _stream(stream))
    _check("nvfp4_quantize", st)
    return tuple(outs) if layout == NVFP4_ROW_COL_1D else outs[0]


def nvfp4_quantize_noalloc(x, out, layout=NVFP4_ROW_1D, round=NVFP4_RNE, sr_seed=0, hadamard=False,
                           hadamard_seed=0, amax_in=None, amax_out=None, stream=None):
    """nvfp4_quantize into preallocated outputs (`out`: one NVFP4Tensor, or a
    pair for NVFP4_ROW_COL_1D) with no workspace: the library's static
    device scratch holds the amax partials, so neither the library nor this
    wrapper allocates anything."""
    assert x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else max(cols, x.stride(0))
    outs = list(out) if isinstance(out, (list, tuple)) else [out]
    arr = (CTensor * 2)()
    for i, t in enumerate(outs):
        arr[i] = t.c()
    opts = CQuantOpts(layout, round, sr_seed, int(bool(hadamard)), hadamard_seed,
                      None if amax_in is None else amax_in.data_ptr(),
                      None if amax_out is None else amax_out.data_ptr())
    st = lib.nvfp4_quantize_noalloc(ctypes.c_void_p(x.data_ptr()), _dtype_code(x.dtype), rows, cols, ld,
                                    ctypes.byref(opts), arr, _stream(stream))
    _check("nvfp4_quantize_noalloc", st)
    return tuple(outs) if layout == NVFP4_ROW_COL_1D else outs[0]


@_launches_on_stream
def nvfp4_requantize(q, round=NVFP4_RNE, sr_seed=0, hadamard=False, hadamard_seed=0, amax_in=None,
                     out=None, workspace=None, amax_out=None, stream=None):
    """COL_1D re-quantization of a row-blocked NVFP4Tensor q (rows x cols):
    returns the cols x rows NVFP4Tensor that quantizing q's binary32
    dequantization along columns gives."""
    dev = q.codes.device
    if out is None:
        out = NVFP4Tensor.empty(q.cols, q.rows, NVFP4_SCALE_1D, dev)
    opts = CQuantOpts(NVFP4_COL_1D, round, sr_seed, int(bool(hadamard)), hadamard_seed,
                      None if amax_in is None else amax_in.data_ptr(),
                      None if amax_out is None else amax_out.data_ptr())
    need = int(lib.nvfp4_quantize_workspace_size(q.rows, q.cols, ctypes.byref(opts)))
    if workspace is None and need:
        workspace = torch.empty((need + 15) // 16 * 4, dtype=torch.float32, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    ci, co = q.c(), out.c()
    st = lib.nvfp4_requantize(ctypes.byref(ci), ctypes.byref(opts), ctypes.byref(co), _ptr(workspace),
                              ws_bytes, _stream(stream))
    _check("nvfp4_requantize", st)
    return out


@_launches_on_stream
def nvfp4_dequantize(q, dtype=torch.float32, out=None, stream=None):
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.codes.device)
    assert out.stride(1) == 1
    ld = out.stride(0) if q.rows > 1 else max(q.cols, out.stride(0))
    ct = q.c()
    st = lib.nvfp4_dequantize(ctypes.byref(ct), ctypes.c_void_p(out.data_ptr()), _dtype_code(out.dtype),
                              ld, _stream(stream))
    _check("nvfp4_dequantize", st)
    return out


def nvfp4_gemm_workspace_size(A, B, out_dtype=torch.float32, epilogue=NVFP4_EPI_NONE):
    """Bytes of workspace with which nvfp4_gemm splits a last partial round
    of tiles on the current device (0: no split)."""
    ca, cb = A.c(), B.c()
    return int(lib.nvfp4_gemm_workspace_size(ctypes.byref(ca), ctypes.byref(cb), _dtype_code(out_dtype),
                                             epilogue))


@_launches_on_stream
def nvfp4_gemm(A, B, out_dtype=torch.float32, out=None, epilogue=NVFP4_EPI_NONE, workspace=None,
               stream=None):
    """C = A B^T (A: M x K, B: N x K NVFP4 tensors); with NVFP4_EPI_SWIGLU
    (N = 2F, bfloat16 output) C = gate * sigmoid(gate) * up, M x F.
    workspace: None allocates what nvfp4_gemm_workspace_size asks for (a
    split of a last partial round of tiles; often nothing); False passes
    none; a device tensor is passed as is."""
    ncols = B.rows // 2 if epilogue == NVFP4_EPI_SWIGLU else B.rows
    if out is None:
        out = torch.empty((A.rows, ncols), dtype=out_dtype, device=A.codes.device)
    assert out.stride(1) == 1
    ldc = out.stride(0) if A.rows > 1 else max(ncols, out.stride(0))
    ca, cb = A.c(), B.c()
    if workspace is None:
        need = int(lib.nvfp4_gemm_workspace_size(ctypes.byref(ca), ctypes.byref(cb), _dtype_code(out.dtype),
                                                 epilogue))
        workspace = torch.empty((need + 15) // 16 * 4, dtype=torch.float32, device=out.device) if need else False
    if workspace is False:
        workspace = None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.nvfp4_gemm(ctypes.byref(ca), ctypes.byref(cb), ctypes.c_void_p(out.data_ptr()),
                        _dtype_code(out.dtype), ldc, epilogue, _ptr(workspace), ws_bytes, _stream(stream))
    _check("nvfp4_gemm", st)
    return out


@_launches_on_stream
def nvfp4_grouped_gemm(A, offsets, B, groups, epilogue=NVFP4_EPI_NONE, out_dtype=torch.bfloat16,
                       out=None, amax_out=None, stream=None):
    """Per group g: rows offsets[g]..offsets[g+1]-1 of A times B_g^T (B stacks
    `groups` weight matrices).  offsets: int64 device tensor [groups+1]."""
    assert offsets.dtype == torch.int64 and offsets.is_cuda
    ng = B.rows // groups
    ncols = ng // 2 if epilogue == NVFP4_EPI_SWIGLU else ng
    if out is None:
        out = torch.empty((A.rows, ncols), dtype=out_dtype, device=A.codes.device)
    assert out.stride(1) == 1
    ldc = out.stride(0) if A.rows > 1 else max(ncols, out.stride(0))
    ca, cb = A.c(), B.c()
    st = lib.nvfp4_grouped_gemm(groups, ctypes.byref(ca), ctypes.c_void_p(offsets.data_ptr()),
                                ctypes.byref(cb), ctypes.c_void_p(out.data_ptr()),
                                _dtype_code(out.dtype), ldc, epilogue, _ptr(amax_out), None, 0,
                                _stream(stream))
    _check("nvfp4_grouped_gemm", st)
    return out


# ---------------------------------------------------------------- MX formats
@dataclass
class MXTensor:
    """codes uint8 ([rows, cols] for E4M3, [rows, cols/2] for E2M1) and E8M0
    scales uint8 [rows, cols/32] -- device tensors."""
    codes: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int
    elem: int = NVFP4_MX_E4M3

    def c(self):
        return CMXTensor(self.codes.data_ptr(), self.scales.data_ptr(), self.rows, self.cols, self.elem)

    @staticmethod
    def empty(rows, cols, elem=NVFP4_MX_E4M3, device="cuda"):
        codes = torch.empty((rows, cols if elem == NVFP4_MX_E4M3 else cols // 2), dtype=torch.uint8,
                            device=device)
        scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=device)
        return MXTensor(codes, scales, rows, cols, elem)


@_launches_on_stream
def nvfp4_mx_quantize(x, layout=NVFP4_ROW_1D, elem=NVFP4_MX_E4M3, round=NVFP4_RNE, sr_seed=0, out=None,
                      stream=None):
    """MX-quantize a 2-D device tensor (float32 or bfloat16, unit column
    stride) along rows (ROW_1D) or columns (COL_1D; the result describes the
    transpose)."""
    assert x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else max(cols, x.stride(0))
    if out is None:
        r, c = (cols, rows) if layout == NVFP4_COL_1D else (rows, cols)
        out = MXTensor.empty(r, c, elem, x.device)
    ct = out.c()
    st = lib.nvfp4_mx_quantize(ctypes.c_void_p(x.data_ptr()), _dtype_code(x.dtype), rows, cols, ld, layout,
                               round, sr_seed, ctypes.byref(ct), _stream(stream))
    _check("nvfp4_mx_quantize", st)
    return out


@_launches_on_stream
def nvfp4_mx_dequantize(q, dtype=torch.float32, out=None, stream=None):
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.codes.device)
    assert out.stride(1) == 1
    ld = out.stride(0) if q.rows > 1 else max(q.cols, out.stride(0))
    ct = q.c()
    st = lib.nvfp4_mx_dequantize(ctypes.byref(ct), ctypes.c_void_p(out.data_ptr()), _dtype_code(out.dtype), ld,
                                 _stream(stream))
    _check("nvfp4_mx_dequantize", st)
    return out


def nvfp4_mx_gemm_workspace_size(A, B, out_dtype=torch.float32, accum=NVFP4_MX_ACC_NATIVE):
    """Bytes of workspace with which nvfp4_mx_gemm splits a last partial
    round of tiles on the current device (0: no split)."""
    ca, cb = A.c(), B.c()
    return int(lib.nvfp4_mx_gemm_workspace_size(ctypes.byref(ca), ctypes.byref(cb), _dtype_code(out_dtype),
                                                accum))


@_launches_on_stream
def nvfp4_mx_gemm(A, B, out_dtype=torch.float32, out=None, accum=NVFP4_MX_ACC_NATIVE, workspace=None,
                  stream=None):
    """C = A B^T (A: M x K, B: N x K MX tensors of one element format);
    accum NVFP4_MX_ACC_NATIVE (scaled matrix cores) or NVFP4_MX_ACC_EXACT
    (exact products, binary32 sums).  workspace as for nvfp4_gemm."""
    if out is None:
        out = torch.empty((A.rows, B.rows), dtype=out_dtype, device=A.codes.device)
    assert out.stride(1) == 1
    ldc = out.stride(0) if A.rows > 1 else max(B.rows, out.stride(0))
    ca, cb = A.c(), B.c()
    if workspace is None:
        need = int(lib.nvfp4_mx_gemm_workspace_size(ctypes.byref(ca), ctypes.byref(cb), _dtype_code(out.dtype),
                                                    accum))
        workspace = torch.empty((need + 15) // 16 * 4, dtype=torch.float32, device=out.device) if need else False
    if workspace is False:
        workspace = None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.nvfp4_mx_gemm(ctypes.byref(ca), ctypes.byref(cb), ctypes.c_void_p(out.data_ptr()),
                           _dtype_code(out.dtype), ldc, accum, _ptr(workspace), ws_bytes, _stream(stream))
    _check("nvfp4_mx_gemm", st)
    return out


# ---------------------------------------------------------------- MoE-block operators
# (checks, allocation and the calls themselves in csrc/binding.cpp)
if not isinstance(_native, _NoBinding):
    # (a torch without a GPU build has neither function, and no tensor that asks for them)
    _native.setup(NVFP4Error, getattr(torch._C, "_cuda_getDevice", None),
                  getattr(torch._C, "_cuda_getCurrentRawStream", None))


def _handle(stream):
    return None if stream is None else stream.cuda_stream


@dataclass
class RMSNormOutput:
    """h (the sum with the residual; x itself without one), y, mx (MXTensor)
    and rstd, each None when not asked for."""
    h: torch.Tensor
    y: torch.Tensor = None
    mx: MXTensor = None
    rstd: torch.Tensor = None


@_launches_on_stream
def nvfp4_rmsnorm(x, weight, residual=None, eps=1e-6, y=True, mx_elem=None, rstd=False, out=None, stream=None):
    """RMS norm of h = x + residual (rows x cols, float32 or bfloat16): y =
    h / sqrt(mean(h^2) + eps) * weight as a tensor of x's dtype (y=True), as
    an MXTensor (mx_elem=NVFP4_MX_E4M3 or NVFP4_MX_E2M1), or both; rstd=True
    returns 1 / sqrt(mean(h^2) + eps) per row for the backward pass.  out: an
    RMSNormOutput of preallocated tensors for what is asked for (out.h may be
    residual or x)."""
    oh = oy = codes = scales = orstd = None
    if out is not None:
        oh, oy, orstd = out.h, out.y, out.rstd
        if mx_elem is not None and out.mx is not None:
            if out.mx.elem != mx_elem:
                raise ValueError("out.mx has another element format than mx_elem")
            codes, scales = out.mx.codes, out.mx.scales
    h, oy, codes, scales, orstd = _native.rmsnorm(x, weight, residual, eps, y, -1 if mx_elem is None else mx_elem, rstd,
                                                  oh, oy, codes, scales, orstd, _handle(stream))
    mx = None if codes is None else MXTensor(codes, scales, x.shape[0], x.shape[1], mx_elem)
    return RMSNormOutput(x if residual is None else h, oy, mx, orstd)


@_launches_on_stream
def nvfp4_rmsnorm_backward(dy, h, rstd, weight, dh=None, dx=None, dweight=None, workspace=None, stream=None):
    """(dx, dweight) of nvfp4_rmsnorm from the h and rstd it gave: dx (h's
    dtype) is the gradient of x and of residual alike, dh (optional) the
    gradient that reaches h by the residual stream, dweight float32.  dx,
    dweight and workspace (nvfp4_rmsnorm_backward_workspace_size) may be
    preallocated."""
    return _native.rmsnorm_backward(dy, h, rstd, weight, dh, dx, dweight, workspace, _handle(stream))


def nvfp4_rmsnorm_backward_workspace_size(rows, cols):
    """Bytes of workspace of nvfp4_rmsnorm_backward."""
    return int(lib.nvfp4_rmsnorm_backward_workspace_size(rows, cols))


@dataclass
class RouteOutput:
    """ids int32 and weights float32 [tokens, top_k]; with the dispatch plan
    offsets int64 [experts + 1], order and position int32 [tokens * top_k]."""
    ids: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor = None
    order: torch.Tensor = None
    position: torch.Tensor = None


def nvfp4_route_workspace_size(tokens, experts):
    """Bytes of workspace of nvfp4_route with the dispatch plan."""
    return int(lib.nvfp4_route_workspace_size(tokens, experts))


@_launches_on_stream
def nvfp4_route(logits, top_k, bias=None, score=NVFP4_ROUTE_SOFTMAX, groups=1, top_groups=1,
                group_score=NVFP4_GROUP_TOP2, renorm=True, plan=True, out=None, workspace=None, stream=None):
    """Route tokens to experts by their logits (tokens x experts, float32 or
    bfloat16): the top_k experts of the largest score + bias (bias float32
    [experts]) within the top_groups groups of the largest group score, and
    their weights.  plan=True also sorts the tokens * top_k assignments by
    expert (offsets feed nvfp4_grouped_gemm; order // top_k are the tokens to
    gather).  out: a RouteOutput of preallocated tensors for some or all of what
    is asked for; the result holds them and new ones for the others."""
    o = (None,) * 5 if out is None else (out.ids, out.weights, out.offsets, out.order, out.position)
    r = _native.route(logits, top_k, bias, score, groups, top_groups, group_score, renorm, plan, *o, workspace,
                      _handle(stream))
    return RouteOutput(*r)


@_launches_on_stream
def nvfp4_route_backward(dweights, logits, ids, score=NVFP4_ROUTE_SOFTMAX, renorm=True, dscores=None, out=None,
                         stream=None):
    """Gradient of the logits from that of the chosen weights (float32
    [tokens, top_k]) and, optionally, of all scores (dscores float32 [tokens,
    experts], as of an auxiliary balance loss)."""
    return _native.route_backward(dweights, logits, ids, score, renorm, dscores, out, _handle(stream))


def _code(dtype):
    return -1 if dtype is None else _dtype_code(dtype)


@_launches_on_stream
def nvfp4_gemv(x, w, epilogue=NVFP4_EPI_NONE, out_dtype=None, out=None, stream=None):
    """x W^T of a few rows x (m x K, bfloat16 or float32, not quantized) and an
    NVFP4Tensor w (N x K): m x N in out_dtype (x's unless given); with
    NVFP4_EPI_SWIGLU (N = 2F) gate * sigmoid(gate) * up, m x F."""
    return _native.gemv(x, w.codes, w.scales, w.tensor_scale, w.rows, w.cols, w.scale_mode, epilogue, _code(out_dtype),
                        out, _handle(stream))


@_launches_on_stream
def nvfp4_mx_gemv(x, w, out_dtype=None, out=None, stream=None):
    """nvfp4_gemv for an MXFP4 weight (MXTensor with E2M1 elements)."""
    return _native.mx_gemv(x, w.codes, w.scales, w.rows, w.cols, w.elem, _code(out_dtype), out, _handle(stream))


def nvfp4_expert_gemv_workspace_size(tokens, top_k, n):
    """Bytes of workspace of nvfp4_expert_gemv with weights (n output columns)."""
    return int(lib.nvfp4_expert_gemv_workspace_size(tokens, top_k, n))


@_launches_on_stream
def nvfp4_expert_gemv(x, ids, w, experts, weights=None, epilogue=NVFP4_EPI_NONE, out_dtype=None, out=None,
                      workspace=None, stream=None):
    """Routed nvfp4_gemv: ids (int32 [tokens, top_k]) names the expert of each
    assignment, w stacks `experts` matrices (tensor_scale [experts]).  x has a
    row for each token or for each assignment (tokens * top_k).  Without
    weights: a row of the result for each assignment; with weights (float32
    [tokens, top_k]): each token's weighted sum of its products."""
    return _native.expert_gemv(x, ids, w.codes, w.scales, w.tensor_scale, w.rows, w.cols, w.scale_mode, experts, weights,
                               epilogue, _code(out_dtype), out, workspace, _handle(stream))


# ---------------------------------------------------------------- the 4-bit key/value cache
@dataclass
class NVFP4KVCache:
    """Pages of keys and values: codes uint8 [pages, kv_heads, page_size,
    head_dim/2] and scales uint8 [pages, kv_heads, page_size, head_dim/16]
    (NVFP4; with k_scale and v_scale, float32 [kv_heads], as the heads' tensor
    scales) or [..., head_dim/32] (MXFP4) -- contiguous device tensors."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor
    k_scale: torch.Tensor = None
    v_scale: torch.Tensor = None
    format: int = NVFP4_KV_NVFP4

    def args(self):
        return (self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.k_scale, self.v_scale, self.format)

    @staticmethod
    def empty(pages, kv_heads, head_dim, page_size=64, format=NVFP4_KV_NVFP4, k_scale=1.0, v_scale=1.0, device="cuda"):
        """A cache with nothing in it.  k_scale and v_scale (NVFP4): what every
        head's values are divided by before their blocks' E4M3 scales (largest
        2688 times that) are found; the largest magnitude expected / 2688, or 1
        for values of ordinary size (block maxima from 2^-9 * 6 to 2688)."""
        per = 32 if format == NVFP4_KV_MXFP4 else 16
        new = [torch.empty((pages, kv_heads, page_size, w), dtype=torch.uint8, device=device)
               for w in (head_dim // 2, head_dim // per) * 2]
        s = [None] * 2 if per == 32 else [torch.full((kv_heads,), float(x), device=device) for x in (k_scale, v_scale)]
        return NVFP4KVCache(*new, *s, format)


@_launches_on_stream
def nvfp4_kv_append(k, v, cache, page_table, lengths, offsets=None, q=None, rope=None, interleaved=False, out=None,
                    stream=None):
    """Append k and v (rows x kv_heads x head_dim, float32 or bfloat16, unit
    stride in the last dimension) to an NVFP4KVCache, k rotated by its
    position, and return q (rows x q_heads x head_dim, optional) rotated alike
    (into `out`, which may be q).  page_table int32 [seqs, width]; lengths
    int32 [seqs]: the sequences' positions with the new ones; offsets int32
    [seqs + 1]: rows offsets[s] .. offsets[s+1]-1 are the last ones of sequence s
    (None: one row a sequence).  rope float32 [positions, dim]: each position's
    dim / 2 cosines, then sines; the first dim elements of a head are rotated
    in halves, or interleaved in pairs."""
    return _native.kv_append(k, v, *cache.args(), page_table, lengths, offsets, rope, interleaved, q, out,
                             _handle(stream))


@_launches_on_stream
def nvfp4_kv_gather(cache, page_table, lengths, offsets=None, rows=None, dtype=torch.bfloat16, out=None, stream=None):
    """(k, v), each rows x kv_heads x head_dim, of the cache's positions that
    the plan names (as nvfp4_kv_append); rows: their number (without offsets one
    a sequence; with offsets that of out unless given).  out: a pair of tensors
    to fill."""
    if out is not None:
        dtype = out[0].dtype
    if rows is None:
        if offsets is not None and out is None:
            raise ValueError("rows must be given where offsets are")  # (they lie on the device)
        rows = page_table.shape[0] if offsets is None else out[0].shape[0]
    return _native.kv_gather(*cache.args(), page_table, lengths, offsets, rows,
                             _dtype_code(dtype), *((None, None) if out is None else out), _handle(stream))


def nvfp4_kv_attention_workspace_size(rows, seqs, q_heads, kv_heads, head_dim, dtype=torch.bfloat16):
    """Bytes of workspace of nvfp4_kv_attention for rows of q in seqs sequences."""
    return int(lib.nvfp4_kv_attention_workspace_size(rows, seqs, q_heads, kv_heads, head_dim, _dtype_code(dtype)))


@_launches_on_stream
def nvfp4_kv_attention(q, cache, page_table, lengths, offsets=None, scale=None, window=0, lse=False, out=None,
                       out_lse=None, workspace=None, stream=None):
    """Attention of q (rows x q_heads x head_dim, float32 or bfloat16) over the
    cache: a row at position p of its sequence (plan as for nvfp4_kv_append,
    after the append) sees the positions up to p, with window > 0 the last
    `window` of them.  scale: head_dim ** -0.5 unless given.  Returns a tensor
    like q, with lse=True also the float32 logarithms of the softmax's sums
    [rows, q_heads].  out, out_lse and workspace
    (nvfp4_kv_attention_workspace_size) may be preallocated."""
    o, l = _native.kv_attention(q, *cache.args(), page_table, lengths, offsets,
                                q.shape[-1] ** -0.5 if scale is None else scale, window, lse, out, out_lse, workspace,
                                _handle(stream))
    return (o, l) if lse else o
