// C ABI of the NVFP4 library (declared in include/nvfp4.h): host-side argument
// validation, then dispatch to the kernel launchers.  No entry point allocates
// memory or keeps state; every error is reported before anything is enqueued.
#include "nvfp4.h"

#include <hip/hip_runtime.h>

#include <mutex>

#include "launch.hpp"

using namespace nvfp4;

// Scratch of nvfp4_quantize_noalloc: the amax pass's per-workgroup partial
// maxima (at most kMaxPartials floats for a tensor of any size, 2 KiB).  Each
// device the library runs on holds its own copy until the process ends.  In
// host code `scratch` names a host-side stand-in, not device memory: kernels
// get the device address that hipGetSymbolAddress returns for the device.
static __device__ __align__(256) float scratch[kMaxPartials];

namespace {

constexpr int64_t kMaxGridY = 65535;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

size_t dtype_size(int dt) { return dt == NVFP4_BF16 ? 2 : 4; }

bool valid_dtype(int dt) { return dt == NVFP4_F32 || dt == NVFP4_BF16; }

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The output tensor a layout implies for an input of rows x cols.
nvfp4_status check_out(const nvfp4_tensor* t, int64_t r, int64_t c, int mode) {
    if (!t->tensor_scale) return NVFP4_ERR_NULL;
    if (r > 0 && c > 0 && (!t->codes || !t->scales)) return NVFP4_ERR_NULL;
    if (t->rows != r || t->cols != c || t->scale_mode != mode) return NVFP4_ERR_SHAPE;
    if (!aligned(t->codes, 16)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

// A GEMM operand: shape, scale layout, pointers, alignment.
nvfp4_status check_operand(const nvfp4_tensor* t) {
    if (!t) return NVFP4_ERR_NULL;
    if (t->rows < 0 || t->cols < 0) return NVFP4_ERR_SHAPE;
    if (t->scale_mode != NVFP4_SCALE_1D && t->scale_mode != NVFP4_SCALE_2D) return NVFP4_ERR_ENUM;
    if (t->cols % 16) return NVFP4_ERR_SHAPE;
    if (t->scale_mode == NVFP4_SCALE_2D && t->rows % 16) return NVFP4_ERR_SHAPE;
    if (t->rows > 0 && t->cols > 0 && (!t->codes || !t->scales)) return NVFP4_ERR_NULL;
    if (!t->tensor_scale) return NVFP4_ERR_NULL;
    if (!aligned(t->codes, 16)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

Operand as_operand(const nvfp4_tensor* t) {
    return Operand{t->codes, t->scales, t->tensor_scale, t->scale_mode == NVFP4_SCALE_2D ? 1 : 0};
}

}  // namespace

extern "C" {

size_t nvfp4_quantize_workspace_size(int64_t rows, int64_t cols, const nvfp4_quant_opts* opts) {
    (void)rows;
    (void)cols;
    if (opts && opts->amax_in) return 0;
    return kQuantWorkspaceBytes;
}

}  // extern "C"

namespace {

// Argument checks of nvfp4_quantize other than the workspace; NVFP4_OK when
// the request can be launched.
nvfp4_status check_quantize(const void* x, int32_t dt /* nvfp4_dtype */, int64_t rows, int64_t cols, int64_t ld,
                            const nvfp4_quant_opts* opts, nvfp4_tensor* out) {
    if (!opts || !out) return NVFP4_ERR_NULL;
    if (!valid_dtype(dt)) return NVFP4_ERR_ENUM;
    const int layout = opts->layout;
    if (layout < NVFP4_ROW_1D || layout > NVFP4_BLK_2D) return NVFP4_ERR_ENUM;
    if (opts->round != NVFP4_RNE && opts->round != NVFP4_SR) return NVFP4_ERR_ENUM;
    if (rows < 0 || cols < 0 || ld < cols) return NVFP4_ERR_SHAPE;
    const bool row_blocks = layout == NVFP4_ROW_1D || layout == NVFP4_ROW_COL_1D || layout == NVFP4_BLK_2D;
    const bool col_blocks = layout == NVFP4_COL_1D || layout == NVFP4_ROW_COL_1D || layout == NVFP4_BLK_2D;
    if (row_blocks && cols % 16) return NVFP4_ERR_SHAPE;
    if (col_blocks && rows % 16) return NVFP4_ERR_SHAPE;
    if (opts->hadamard && layout == NVFP4_BLK_2D) return NVFP4_ERR_UNSUPPORTED;
    const bool empty = rows == 0 || cols == 0;
    if (!empty && !x) return NVFP4_ERR_NULL;
    if (!aligned(x, 16) || (ld * (int64_t)dtype_size(dt)) % 16) return NVFP4_ERR_ALIGN;

    nvfp4_status st;
    switch (layout) {
        case NVFP4_ROW_1D: st = check_out(&out[0], rows, cols, NVFP4_SCALE_1D); break;
        case NVFP4_COL_1D: st = check_out(&out[0], cols, rows, NVFP4_SCALE_1D); break;
        case NVFP4_BLK_2D: st = check_out(&out[0], rows, cols, NVFP4_SCALE_2D); break;
        default:
            st = check_out(&out[0], rows, cols, NVFP4_SCALE_1D);
            if (st == NVFP4_OK) st = check_out(&out[1], cols, rows, NVFP4_SCALE_1D);
    }
    if (st != NVFP4_OK) return st;

    // grid-size limits of the launches (y counts row tiles / row bands)
    if (cdiv(cols, 128) > 0x7FFFFFFF) return NVFP4_ERR_UNSUPPORTED;
    if ((layout == NVFP4_COL_1D || layout == NVFP4_ROW_COL_1D) && cdiv(rows, 256) > kMaxGridY)
        return NVFP4_ERR_UNSUPPORTED;
    if (layout == NVFP4_BLK_2D && cdiv(rows, 64) > kMaxGridY) return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

nvfp4_status launch_checked_quantize(const void* x, int32_t dt /* nvfp4_dtype */, int64_t rows, int64_t cols,
                                     int64_t ld, const nvfp4_quant_opts* opts, nvfp4_tensor* out,
                                     float* ws, void* stream) {
    const int layout = opts->layout;
    QOut o[2];
    o[0] = QOut{out[0].codes, out[0].scales, out[0].tensor_scale};
    if (layout == NVFP4_ROW_COL_1D) o[1] = QOut{out[1].codes, out[1].scales, out[1].tensor_scale};
    else o[1] = QOut{nullptr, nullptr, nullptr};
    hipError_t e = launch_quantize(x, dt == NVFP4_BF16, rows, cols, ld, layout, opts->round == NVFP4_SR,
                                   opts->sr_seed, opts->hadamard != 0, opts->hadamard_seed,
                                   opts->amax_in, opts->amax_out, o, ws, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
float* g_scratch_ptr[kMaxDevices] = {};

// The device address of `scratch` on the device `stream` belongs to, looked up
// once per device with that device current; NULL on failure.
float* scratch_on_device_of(hipStream_t stream) {
    int dev = -1;
    if (stream) {
        if (hipStreamGetDevice(stream, &dev) != hipSuccess) return nullptr;
    } else if (hipGetDevice(&dev) != hipSuccess) {
        return nullptr;
    }
    if (dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        int cur = -1;
        if (hipGetDevice(&cur) != hipSuccess) return nullptr;
        if (cur != dev && hipSetDevice(dev) != hipSuccess) return nullptr;
        void* p = nullptr;
        const hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (cur != dev) (void)hipSetDevice(cur);
        if (e != hipSuccess || !p) return nullptr;
        g_scratch_ptr[dev] = static_cast<float*>(p);
    }
    return g_scratch_ptr[dev];
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_quantize(const void* x, int32_t dt /* nvfp4_dtype */, int64_t rows, int64_t cols, int64_t ld,
                            const nvfp4_quant_opts* opts, nvfp4_tensor* out, void* ws,
                            size_t ws_bytes, void* stream) {
    nvfp4_status st = check_quantize(x, dt, rows, cols, ld, opts, out);
    if (st != NVFP4_OK) return st;
    if (rows > 0 && cols > 0 && !opts->amax_in) {
        if (!ws) return NVFP4_ERR_WORKSPACE;
        if (ws_bytes < kQuantWorkspaceBytes) return NVFP4_ERR_WORKSPACE;
        if (!aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    }
    return launch_checked_quantize(x, dt, rows, cols, ld, opts, out, static_cast<float*>(ws), stream);
}

nvfp4_status nvfp4_quantize_noalloc(const void* x, int32_t dt /* nvfp4_dtype */, int64_t rows, int64_t cols, int64_t ld,
                                    const nvfp4_quant_opts* opts, nvfp4_tensor* out, void* stream) {
    nvfp4_status st = check_quantize(x, dt, rows, cols, ld, opts, out);
    if (st != NVFP4_OK) return st;
    // the amax pass writes at most kMaxPartials partials whatever the size, so
    // no request needs more scratch than the array holds
    static_assert(sizeof(scratch) >= kQuantWorkspaceBytes, "scratch smaller than the quantize workspace");
    float* ws = nullptr;
    if (rows > 0 && cols > 0 && !opts->amax_in) {
        ws = scratch_on_device_of(static_cast<hipStream_t>(stream));
        if (!ws) return NVFP4_ERR_HIP;
    }
    return launch_checked_quantize(x, dt, rows, cols, ld, opts, out, ws, stream);
}

nvfp4_status nvfp4_requantize(const nvfp4_tensor* in, const nvfp4_quant_opts* opts, nvfp4_tensor* out,
                              void* ws, size_t ws_bytes, void* stream) {
    if (!in || !opts || !out) return NVFP4_ERR_NULL;
    if (opts->layout < NVFP4_ROW_1D || opts->layout > NVFP4_BLK_2D) return NVFP4_ERR_ENUM;
    if (opts->round != NVFP4_RNE && opts->round != NVFP4_SR) return NVFP4_ERR_ENUM;
    nvfp4_status st = check_operand(in);
    if (st != NVFP4_OK) return st;
    if (in->scale_mode != NVFP4_SCALE_1D) return NVFP4_ERR_UNSUPPORTED;
    if (opts->layout != NVFP4_COL_1D) return NVFP4_ERR_UNSUPPORTED;
    const int64_t rows = in->rows, cols = in->cols;
    if (rows % 16) return NVFP4_ERR_SHAPE;
    st = check_out(out, cols, rows, NVFP4_SCALE_1D);
    if (st != NVFP4_OK) return st;
    if (cdiv(rows, 256) > kMaxGridY) return NVFP4_ERR_UNSUPPORTED;
    const bool empty = rows == 0 || cols == 0;
    if (!empty && !opts->amax_in) {
        if (!ws) return NVFP4_ERR_WORKSPACE;
        if (ws_bytes < kQuantWorkspaceBytes) return NVFP4_ERR_WORKSPACE;
        if (!aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    }
    const QOut o{out->codes, out->scales, out->tensor_scale};
    hipError_t e = launch_requantize(in->codes, in->scales, in->tensor_scale, rows, cols,
                                     opts->round == NVFP4_SR, opts->sr_seed, opts->hadamard != 0,
                                     opts->hadamard_seed, opts->amax_in, opts->amax_out, &o,
                                     static_cast<float*>(ws), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

nvfp4_status nvfp4_dequantize(const nvfp4_tensor* q, void* y, int32_t dt /* nvfp4_dtype */, int64_t ld,
                              void* stream) {
    if (!q) return NVFP4_ERR_NULL;
    if (!valid_dtype(dt)) return NVFP4_ERR_ENUM;
    nvfp4_status st = check_operand(q);
    if (st != NVFP4_OK) return st;
    if (ld < q->cols) return NVFP4_ERR_SHAPE;
    const bool empty = q->rows == 0 || q->cols == 0;
    if (!empty && !y) return NVFP4_ERR_NULL;
    if (!aligned(y, 16) || (ld * (int64_t)dtype_size(dt)) % 16) return NVFP4_ERR_ALIGN;
    hipError_t e = launch_dequantize(q->codes, q->scales, q->tensor_scale, q->rows, q->cols,
                                     q->scale_mode == NVFP4_SCALE_2D, y, dt == NVFP4_BF16, ld,
                                     static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

size_t nvfp4_gemm_workspace_size(const nvfp4_tensor* A, const nvfp4_tensor* B, int32_t c_dt /* nvfp4_dtype */,
                                 int32_t ep /* nvfp4_epilogue */) {
    if (!A || !B || !valid_dtype(c_dt) || ep != NVFP4_EPI_NONE) return 0;
    if (A->rows < 0 || B->rows < 0 || A->cols != B->cols) return 0;
    int cus = 0;
    if (device_cus(cus) != hipSuccess) return 0;
    const GemmSplit sp = gemm_split_plan(A->rows, B->rows, A->cols, false, cus);
    return sp.split > 1 ? (size_t)sp.bytes : 0;
}

nvfp4_status nvfp4_gemm(const nvfp4_tensor* A, const nvfp4_tensor* B, void* C, int32_t c_dt /* nvfp4_dtype */,
                        int64_t ldc, int32_t ep /* nvfp4_epilogue */, void* ws, size_t ws_bytes, void* stream) {
    if (!A || !B) return NVFP4_ERR_NULL;
    if (!valid_dtype(c_dt)) return NVFP4_ERR_ENUM;
    if (ep != NVFP4_EPI_NONE && ep != NVFP4_EPI_SWIGLU) return NVFP4_ERR_ENUM;
    nvfp4_status st = check_operand(A);
    if (st != NVFP4_OK) return st;
    st = check_operand(B);
    if (st != NVFP4_OK) return st;
    if (A->cols != B->cols) return NVFP4_ERR_SHAPE;
    const int64_t M = A->rows, N = B->rows, K = A->cols;
    const bool swiglu = ep == NVFP4_EPI_SWIGLU;
    if (swiglu) {
        if (N % 2 || (N / 2) % 16) return NVFP4_ERR_SHAPE;
        if (c_dt != NVFP4_BF16) return NVFP4_ERR_UNSUPPORTED;
    }
    const int64_t ncols = swiglu ? N / 2 : N;
    if (ldc < ncols) return NVFP4_ERR_SHAPE;
    if (M > 0 && ncols > 0 && !C) return NVFP4_ERR_NULL;
    if (!aligned(C, dtype_size(c_dt))) return NVFP4_ERR_ALIGN;
    if (cdiv(M, 128) > kMaxGridY) return NVFP4_ERR_UNSUPPORTED;
    if (ws && !aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    hipError_t e = launch_gemm(as_operand(A), as_operand(B), M, N, K, C, c_dt == NVFP4_BF16, ldc, swiglu,
                               ws, ws ? ws_bytes : 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

nvfp4_status nvfp4_grouped_gemm(int32_t G, const nvfp4_tensor* A, const int64_t* offsets,
                                const nvfp4_tensor* B, void* C, int32_t c_dt /* nvfp4_dtype */, int64_t ldc,
                                int32_t ep /* nvfp4_epilogue */, float* amax_out, void* ws, size_t ws_bytes,
                                void* stream) {
    (void)ws;
    (void)ws_bytes;
    if (!A || !B || !offsets) return NVFP4_ERR_NULL;
    if (!valid_dtype(c_dt)) return NVFP4_ERR_ENUM;
    if (ep != NVFP4_EPI_NONE && ep != NVFP4_EPI_SWIGLU) return NVFP4_ERR_ENUM;
    if (G < 1) return NVFP4_ERR_SHAPE;
    nvfp4_status st = check_operand(A);
    if (st != NVFP4_OK) return st;
    st = check_operand(B);
    if (st != NVFP4_OK) return st;
    if (A->scale_mode != NVFP4_SCALE_1D) return NVFP4_ERR_UNSUPPORTED;
    if (A->cols != B->cols) return NVFP4_ERR_SHAPE;
    if (B->rows % G) return NVFP4_ERR_SHAPE;
    const int64_t Ng = B->rows / G, K = A->cols, total = A->rows;
    if (B->scale_mode == NVFP4_SCALE_2D && Ng % 16) return NVFP4_ERR_SHAPE;
    const bool swiglu = ep == NVFP4_EPI_SWIGLU;
    if (swiglu) {
        if (Ng % 2 || (Ng / 2) % 16) return NVFP4_ERR_SHAPE;
        if (c_dt != NVFP4_BF16) return NVFP4_ERR_UNSUPPORTED;
    } else if (amax_out) {
        return NVFP4_ERR_UNSUPPORTED;
    }
    const int64_t ncols = swiglu ? Ng / 2 : Ng;
    if (ldc < ncols) return NVFP4_ERR_SHAPE;
    if (total > 0 && ncols > 0 && !C) return NVFP4_ERR_NULL;
    if (!aligned(C, dtype_size(c_dt))) return NVFP4_ERR_ALIGN;
    if (cdiv(total, 128) + G > kMaxGridY) return NVFP4_ERR_UNSUPPORTED;
    hipError_t e = launch_grouped_gemm(G, as_operand(A), offsets, total, as_operand(B), Ng, K, C,
                                       c_dt == NVFP4_BF16, ldc, swiglu, amax_out,
                                       static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

// ---------------------------------------------------------------- MX formats
nvfp4_status nvfp4_mx_quantize(const void* x, int32_t dt /* nvfp4_dtype */, int64_t rows, int64_t cols, int64_t ld,
                               int32_t layout /* nvfp4_layout */, int32_t round /* nvfp4_round */, uint64_t sr_seed,
                               nvfp4_mx_tensor* out, void* stream) {
    if (!out) return NVFP4_ERR_NULL;
    if (!valid_dtype(dt)) return NVFP4_ERR_ENUM;
    if (layout < NVFP4_ROW_1D || layout > NVFP4_BLK_2D) return NVFP4_ERR_ENUM;
    if (round != NVFP4_RNE && round != NVFP4_SR) return NVFP4_ERR_ENUM;
    if (out->elem != NVFP4_MX_E4M3 && out->elem != NVFP4_MX_E2M1) return NVFP4_ERR_ENUM;
    if (layout != NVFP4_ROW_1D && layout != NVFP4_COL_1D) return NVFP4_ERR_UNSUPPORTED;
    if (rows < 0 || cols < 0 || ld < cols) return NVFP4_ERR_SHAPE;
    const bool col = layout == NVFP4_COL_1D;
    if ((col ? rows : cols) % 32) return NVFP4_ERR_SHAPE;
    const int64_t orows = col ? cols : rows, ocols = col ? rows : cols;
    if (out->rows != orows || out->cols != ocols) return NVFP4_ERR_SHAPE;
    const bool empty = rows == 0 || cols == 0;
    if (!empty && (!x || !out->codes || !out->scales)) return NVFP4_ERR_NULL;
    if (!aligned(x, 16) || (ld * (int64_t)dtype_size(dt)) % 16 || !aligned(out->codes, 16))
        return NVFP4_ERR_ALIGN;
    if (col ? cdiv(rows, 256) > kMaxGridY : cdiv(cols, 512) > 0x7FFFFFFF) return NVFP4_ERR_UNSUPPORTED;
    hipError_t e = launch_mx_quantize(x, dt == NVFP4_BF16, rows, cols, ld, col ? kLayoutCol : kLayoutRow,
                                      out->elem == NVFP4_MX_E4M3 ? kMxE4M3 : kMxE2M1, round == NVFP4_SR,
                                      sr_seed, out->codes, out->scales, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

nvfp4_status nvfp4_mx_dequantize(const nvfp4_mx_tensor* q, void* y, int32_t dt /* nvfp4_dtype */, int64_t ld,
                                 void* stream) {
    if (!q) return NVFP4_ERR_NULL;
    if (!valid_dtype(dt)) return NVFP4_ERR_ENUM;
    if (q->elem != NVFP4_MX_E4M3 && q->elem != NVFP4_MX_E2M1) return NVFP4_ERR_ENUM;
    if (q->rows < 0 || q->cols < 0 || q->cols % 32 || ld < q->cols) return NVFP4_ERR_SHAPE;
    const bool empty = q->rows == 0 || q->cols == 0;
    if (!empty && (!y || !q->codes || !q->scales)) return NVFP4_ERR_NULL;
    if (!aligned(y, 16) || (ld * (int64_t)dtype_size(dt)) % 16 || !aligned(q->codes, 16))
        return NVFP4_ERR_ALIGN;
    if (cdiv(q->cols / 8, 64) > 0x7FFFFFFF) return NVFP4_ERR_UNSUPPORTED;
    hipError_t e = launch_mx_dequantize(q->codes, q->scales, q->elem == NVFP4_MX_E4M3 ? kMxE4M3 : kMxE2M1,
                                        q->rows, q->cols, y, dt == NVFP4_BF16, ld,
                                        static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

size_t nvfp4_mx_gemm_workspace_size(const nvfp4_mx_tensor* A, const nvfp4_mx_tensor* B, int32_t c_dt /* nvfp4_dtype */,
                                    int32_t accum) {
    if (!A || !B || !valid_dtype(c_dt)) return 0;
    if (accum != NVFP4_MX_ACC_NATIVE && accum != NVFP4_MX_ACC_EXACT) return 0;
    if (A->rows < 0 || B->rows < 0 || A->cols != B->cols) return 0;
    int cus = 0;
    if (device_cus(cus) != hipSuccess) return 0;
    const GemmSplit sp =
        mx_gemm_split_plan(A->rows, B->rows, A->cols, mx_split_tile_us(A->elem == NVFP4_MX_E4M3 ? kMxE4M3 : kMxE2M1, accum == NVFP4_MX_ACC_EXACT), cus);
    return sp.split > 1 ? (size_t)sp.bytes : 0;
}

nvfp4_status nvfp4_mx_gemm(const nvfp4_mx_tensor* A, const nvfp4_mx_tensor* B, void* C, int32_t c_dt /* nvfp4_dtype */,
                           int64_t ldc, int32_t accum, void* ws, size_t ws_bytes, void* stream) {
    if (!A || !B) return NVFP4_ERR_NULL;
    if (!valid_dtype(c_dt)) return NVFP4_ERR_ENUM;
    if (accum != NVFP4_MX_ACC_NATIVE && accum != NVFP4_MX_ACC_EXACT) return NVFP4_ERR_ENUM;
    for (const nvfp4_mx_tensor* t : {A, B}) {
        if (t->elem != NVFP4_MX_E4M3 && t->elem != NVFP4_MX_E2M1) return NVFP4_ERR_ENUM;
        if (t->rows < 0 || t->cols < 0 || t->cols % 32) return NVFP4_ERR_SHAPE;
    }
    if (A->cols != B->cols) return NVFP4_ERR_SHAPE;
    if (A->elem != B->elem) return NVFP4_ERR_UNSUPPORTED;
    const int64_t M = A->rows, N = B->rows, K = A->cols;
    if (K % 64) return NVFP4_ERR_UNSUPPORTED;
    // the kernels keep per-lane byte offsets inside a 256-row tile in 32 bits
    const uint64_t row_bytes = (uint64_t)(A->elem == NVFP4_MX_E4M3 ? K : K / 2);
    if (256 * row_bytes >= ((uint64_t)1 << 32)) return NVFP4_ERR_UNSUPPORTED;
    if (ldc < N) return NVFP4_ERR_SHAPE;
    if (M > 0 && N > 0) {
        if (!C) return NVFP4_ERR_NULL;
        if (K > 0 && (!A->codes || !A->scales || !B->codes || !B->scales)) return NVFP4_ERR_NULL;
    }
    if (!aligned(C, dtype_size(c_dt)) || !aligned(A->codes, 16) || !aligned(B->codes, 16) ||
        !aligned(A->scales, 2) || !aligned(B->scales, 2))
        return NVFP4_ERR_ALIGN;
    if (cdiv(M, 256) > kMaxGridY) return NVFP4_ERR_UNSUPPORTED;
    if (ws && !aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    hipError_t e = launch_mx_gemm(A->codes, A->scales, B->codes, B->scales,
                                  A->elem == NVFP4_MX_E4M3 ? kMxE4M3 : kMxE2M1, M, N, K, C, c_dt == NVFP4_BF16,
                                  ldc, accum == NVFP4_MX_ACC_EXACT, ws, ws ? ws_bytes : 0,
                                  static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

// ---------------------------------------------------------------- RMS norm
namespace {

// A matrix argument of the row operators: any element alignment and stride.
nvfp4_status check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dt) {
    if (ld < cols) return NVFP4_ERR_SHAPE;
    if (rows > 0 && !p) return NVFP4_ERR_NULL;
    return aligned(p, dtype_size(dt)) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

}  // namespace

nvfp4_status nvfp4_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                           int32_t w_dt /* nvfp4_dtype */, int32_t dt /* nvfp4_dtype */, int64_t rows, int64_t cols,
                           float eps, void* h, int64_t ldh, void* y, int64_t ldy, nvfp4_mx_tensor* mx, float* rstd,
                           void* stream) {
    if (!valid_dtype(dt) || !valid_dtype(w_dt)) return NVFP4_ERR_ENUM;
    if (mx && mx->elem != NVFP4_MX_E4M3 && mx->elem != NVFP4_MX_E2M1) return NVFP4_ERR_ENUM;
    if (rows < 0 || cols < 1) return NVFP4_ERR_SHAPE;
    if (!y && !mx) return NVFP4_ERR_NULL;
    if (!weight) return NVFP4_ERR_NULL;
    if (!aligned(weight, dtype_size(w_dt)) || !aligned(rstd, 4)) return NVFP4_ERR_ALIGN;
    nvfp4_status st = check_matrix(x, rows, cols, ldx, dt);
    if (st == NVFP4_OK && residual) st = check_matrix(residual, rows, cols, ldr, dt);
    if (st == NVFP4_OK && h) st = check_matrix(h, rows, cols, ldh, dt);
    if (st == NVFP4_OK && y) st = check_matrix(y, rows, cols, ldy, dt);
    if (st != NVFP4_OK) return st;
    if (mx) {
        if (cols % 32 || mx->rows != rows || mx->cols != cols) return NVFP4_ERR_SHAPE;
        if (rows > 0 && (!mx->codes || !mx->scales)) return NVFP4_ERR_NULL;
        if (!aligned(mx->codes, 16)) return NVFP4_ERR_ALIGN;
    }
    if (!(eps > 0.0f) || cols > kMaxNormCols || rows > 0x7FFFFFFF) return NVFP4_ERR_UNSUPPORTED;
    RmsNorm n = {x, residual, weight, dt == NVFP4_BF16, w_dt == NVFP4_BF16, rows, cols, ldx, ldr, ldh, ldy, eps, h, y,
                 mx ? mx->codes : nullptr, mx ? mx->scales : nullptr,
                 mx && mx->elem == NVFP4_MX_E2M1 ? kMxE2M1 : kMxE4M3, rstd};
    return launch_rmsnorm(n, static_cast<hipStream_t>(stream)) == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

size_t nvfp4_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols) {
    if (rows < 0 || rows > 0x7FFFFFFF || cols < 1 || cols > kMaxNormCols) return 0;
    return (size_t)rmsnorm_backward_workspace_floats(rows, cols) * sizeof(float);
}

nvfp4_status nvfp4_rmsnorm_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh, const float* rstd,
                                    const void* weight, int32_t w_dt /* nvfp4_dtype */, const void* dh, int64_t lddh,
                                    int32_t dt /* nvfp4_dtype */, int64_t rows, int64_t cols, void* dx, int64_t lddx,
                                    float* dweight, void* ws, size_t ws_bytes, void* stream) {
    if (!valid_dtype(dt) || !valid_dtype(w_dt)) return NVFP4_ERR_ENUM;
    if (rows < 0 || cols < 1) return NVFP4_ERR_SHAPE;
    if (!weight || !dweight || (rows > 0 && !rstd)) return NVFP4_ERR_NULL;
    if (!aligned(weight, dtype_size(w_dt)) || !aligned(rstd, 4) || !aligned(dweight, 4)) return NVFP4_ERR_ALIGN;
    nvfp4_status st = check_matrix(dy, rows, cols, lddy, dt);
    if (st == NVFP4_OK) st = check_matrix(h, rows, cols, ldh, dt);
    if (st == NVFP4_OK && dh) st = check_matrix(dh, rows, cols, lddh, dt);
    if (st == NVFP4_OK) st = check_matrix(dx, rows, cols, lddx, dt);
    if (st != NVFP4_OK) return st;
    if (cols > kMaxNormCols || rows > 0x7FFFFFFF) return NVFP4_ERR_UNSUPPORTED;
    if (rows > 0) {
        if (!ws || ws_bytes < nvfp4_rmsnorm_backward_workspace_size(rows, cols)) return NVFP4_ERR_WORKSPACE;
        if (!aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    }
    RmsNormBackward n = {dy, h, dh, rstd, weight, dt == NVFP4_BF16, w_dt == NVFP4_BF16, rows, cols, lddy, ldh, lddh,
                         lddx, dx, dweight, static_cast<float*>(ws)};
    return launch_rmsnorm_backward(n, static_cast<hipStream_t>(stream)) == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

// ---------------------------------------------------------------- routing
size_t nvfp4_route_workspace_size(int64_t tokens, int64_t experts) {
    if (tokens < 0 || tokens > 0x7FFFFFFF || experts < 1 || experts > kMaxExperts) return 0;
    return route_workspace_bytes(tokens, (int)experts);
}

nvfp4_status nvfp4_route(const void* logits, int32_t dt /* nvfp4_dtype */, int64_t tokens, int64_t experts, int64_t ld,
                         const nvfp4_route_opts* opts, int32_t* ids, float* weights, int64_t* offsets, int32_t* order,
                         int32_t* position, void* ws, size_t ws_bytes, void* stream) {
    if (!opts) return NVFP4_ERR_NULL;
    if (!valid_dtype(dt)) return NVFP4_ERR_ENUM;
    if (opts->score != NVFP4_ROUTE_SOFTMAX && opts->score != NVFP4_ROUTE_SIGMOID) return NVFP4_ERR_ENUM;
    if (opts->group_score != NVFP4_GROUP_MAX && opts->group_score != NVFP4_GROUP_TOP2) return NVFP4_ERR_ENUM;
    const int64_t G = opts->groups, k = opts->top_k;
    if (tokens < 0 || experts < 1 || G < 1 || experts % G || opts->top_groups < 1 || opts->top_groups > G || k < 1 ||
        k > opts->top_groups * (experts / G))
        return NVFP4_ERR_SHAPE;
    nvfp4_status st = check_matrix(logits, tokens, experts, ld, dt);
    if (st != NVFP4_OK) return st;
    if (tokens > 0 && (!ids || !weights)) return NVFP4_ERR_NULL;
    if ((order || position) && !offsets) return NVFP4_ERR_NULL;
    if (offsets && tokens > 0 && (!order || !position)) return NVFP4_ERR_NULL;
    if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(offsets, 8) || !aligned(order, 4) ||
        !aligned(position, 4) || !aligned(opts->bias, 4))
        return NVFP4_ERR_ALIGN;
    if (experts > kMaxExperts || k > kMaxTopK || !route_shape_fits((int)experts, (int)G) || tokens > 0x7FFFFFFF / k)
        return NVFP4_ERR_UNSUPPORTED;
    const size_t need = offsets ? nvfp4_route_workspace_size(tokens, experts) : 0;
    if (need) {
        if (!ws || ws_bytes < need) return NVFP4_ERR_WORKSPACE;
        if (!aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    }
    RouteArgs a;
    a.logits = logits;
    a.bf16 = dt == NVFP4_BF16;
    a.tokens = tokens;
    a.ld = ld;
    a.bias = opts->bias;
    a.shape = RouteShape{(int)experts, (int)G, (int)(experts / G), opts->top_groups, opts->top_k, 0,
                         opts->group_score == NVFP4_GROUP_TOP2};
    a.sigmoid = opts->score == NVFP4_ROUTE_SIGMOID;
    a.renorm = opts->renorm != 0;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.order = order;
    a.position = position;
    a.counts = static_cast<uint8_t*>(ws);
    a.span = 0;
    a.group = 0;
    return launch_route(a, static_cast<hipStream_t>(stream)) == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

nvfp4_status nvfp4_route_backward(const float* dweights, const void* logits, int32_t dt /* nvfp4_dtype */,
                                  int64_t tokens, int64_t experts, int64_t ld, const int32_t* ids, int32_t top_k,
                                  int32_t score /* nvfp4_route_score */, int32_t renorm, const float* dscores,
                                  int64_t ldds, void* dlogits, int64_t lddl, void* stream) {
    if (!valid_dtype(dt)) return NVFP4_ERR_ENUM;
    if (score != NVFP4_ROUTE_SOFTMAX && score != NVFP4_ROUTE_SIGMOID) return NVFP4_ERR_ENUM;
    if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts) return NVFP4_ERR_SHAPE;
    nvfp4_status st = check_matrix(logits, tokens, experts, ld, dt);
    if (st == NVFP4_OK && dscores) st = check_matrix(dscores, tokens, experts, ldds, NVFP4_F32);
    if (st == NVFP4_OK) st = check_matrix(dlogits, tokens, experts, lddl, dt);
    if (st != NVFP4_OK) return st;
    if (tokens > 0 && (!dweights || !ids)) return NVFP4_ERR_NULL;
    if (!aligned(dweights, 4) || !aligned(ids, 4)) return NVFP4_ERR_ALIGN;
    if (experts > kMaxExperts || top_k > kMaxTopK || tokens > 0x7FFFFFFF) return NVFP4_ERR_UNSUPPORTED;
    const RouteBackward a = {dweights, logits, ids, dscores, dlogits, tokens, ld, ldds, lddl, (int)experts, top_k,
                             score == NVFP4_ROUTE_SIGMOID, renorm != 0};
    return launch_route_backward(a, dt == NVFP4_BF16, static_cast<hipStream_t>(stream)) == hipSuccess ? NVFP4_OK
                                                                                                     : NVFP4_ERR_HIP;
}

// ---------------------------------------------------------------- products of a few rows
namespace {

// Arguments that nvfp4_gemv and its MX and routed forms share: the output
// columns of one matrix of N rows, x and y.
nvfp4_status check_gemv(const void* x, int32_t dt, int64_t x_rows, int64_t ldx, int64_t N, int64_t K, const void* y,
                        int32_t y_dt, int64_t y_rows, int64_t ldy, int32_t ep) {
    const bool swiglu = ep == NVFP4_EPI_SWIGLU;
    if (swiglu && (N % 2 || (N / 2) % 16)) return NVFP4_ERR_SHAPE;
    if (x_rows < 0) return NVFP4_ERR_SHAPE;
    const int64_t outs = swiglu ? N / 2 : N;
    nvfp4_status st = check_matrix(x, K > 0 ? x_rows : 0, K, ldx, dt);
    if (st == NVFP4_OK) st = check_matrix(y, outs > 0 ? y_rows : 0, outs, ldy, y_dt);
    if (st != NVFP4_OK) return st;
    if (N > kMaxGemvCols) return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

}  // namespace

nvfp4_status nvfp4_gemv(const void* x, int32_t dt /* nvfp4_dtype */, int64_t m, int64_t ldx, const nvfp4_tensor* W,
                        void* y, int32_t y_dt /* nvfp4_dtype */, int64_t ldy, int32_t ep /* nvfp4_epilogue */,
                        void* stream) {
    if (!W) return NVFP4_ERR_NULL;
    if (!valid_dtype(dt) || !valid_dtype(y_dt)) return NVFP4_ERR_ENUM;
    if (ep != NVFP4_EPI_NONE && ep != NVFP4_EPI_SWIGLU) return NVFP4_ERR_ENUM;
    nvfp4_status st = check_operand(W);
    if (st == NVFP4_OK) st = check_gemv(x, dt, m, ldx, W->rows, W->cols, y, y_dt, m, ldy, ep);
    if (st != NVFP4_OK) return st;
    if (m > kMaxGemvRows) return NVFP4_ERR_UNSUPPORTED;
    GemvArgs p = {x, m, ldx, W->codes, W->scales, W->tensor_scale, W->rows, W->cols, y, ldy, nullptr, 0, 1, 0, false,
                  dt == NVFP4_BF16, y_dt == NVFP4_BF16, W->scale_mode == NVFP4_SCALE_2D, false, 0};
    const hipError_t e = launch_gemv(p, ep == NVFP4_EPI_SWIGLU, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

nvfp4_status nvfp4_mx_gemv(const void* x, int32_t dt /* nvfp4_dtype */, int64_t m, int64_t ldx,
                           const nvfp4_mx_tensor* W, void* y, int32_t y_dt /* nvfp4_dtype */, int64_t ldy,
                           void* stream) {
    if (!W) return NVFP4_ERR_NULL;
    if (!valid_dtype(dt) || !valid_dtype(y_dt)) return NVFP4_ERR_ENUM;
    if (W->elem != NVFP4_MX_E4M3 && W->elem != NVFP4_MX_E2M1) return NVFP4_ERR_ENUM;
    if (W->rows < 0 || W->cols < 0 || W->cols % 32) return NVFP4_ERR_SHAPE;
    if (W->rows > 0 && W->cols > 0 && (!W->codes || !W->scales)) return NVFP4_ERR_NULL;
    if (!aligned(W->codes, 16)) return NVFP4_ERR_ALIGN;
    const nvfp4_status st = check_gemv(x, dt, m, ldx, W->rows, W->cols, y, y_dt, m, ldy, NVFP4_EPI_NONE);
    if (st != NVFP4_OK) return st;
    if (W->elem != NVFP4_MX_E2M1 || m > kMaxGemvRows) return NVFP4_ERR_UNSUPPORTED;
    GemvArgs p = {x, m, ldx, W->codes, W->scales, nullptr, W->rows, W->cols, y, ldy, nullptr, 0, 1, 0, false,
                  dt == NVFP4_BF16, y_dt == NVFP4_BF16, false, true, 0};
    const hipError_t e = launch_gemv(p, false, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

size_t nvfp4_expert_gemv_workspace_size(int64_t tokens, int32_t top_k, int64_t n) {
    if (tokens < 0 || top_k < 1 || n < 0 || tokens > kMaxGemvAssignments / top_k) return 0;
    if (n > (int64_t)1 << 40) return 0;
    return (size_t)(tokens * top_k * n) * sizeof(float);
}

nvfp4_status nvfp4_expert_gemv(const void* x, int32_t dt /* nvfp4_dtype */, int64_t x_rows, int64_t ldx,
                               const int32_t* ids, int64_t tokens, int32_t top_k, const nvfp4_tensor* W,
                               int32_t experts, const float* weights, void* y, int32_t y_dt /* nvfp4_dtype */,
                               int64_t ldy, int32_t ep /* nvfp4_epilogue */, void* ws, size_t ws_bytes, void* stream) {
    if (!W) return NVFP4_ERR_NULL;
    if (!valid_dtype(dt) || !valid_dtype(y_dt)) return NVFP4_ERR_ENUM;
    if (ep != NVFP4_EPI_NONE && ep != NVFP4_EPI_SWIGLU) return NVFP4_ERR_ENUM;
    if (experts < 1 || tokens < 0 || top_k < 1) return NVFP4_ERR_SHAPE;
    nvfp4_status st = check_operand(W);
    if (st != NVFP4_OK) return st;
    if (W->rows % experts) return NVFP4_ERR_SHAPE;
    const int64_t N = W->rows / experts;
    if (W->scale_mode == NVFP4_SCALE_2D && N % 16) return NVFP4_ERR_SHAPE;
    if (tokens > kMaxGemvAssignments / top_k) return NVFP4_ERR_UNSUPPORTED;
    const int64_t assignments = tokens * top_k;
    if (x_rows != tokens && x_rows != assignments) return NVFP4_ERR_SHAPE;
    st = check_gemv(x, dt, x_rows, ldx, N, W->cols, y, y_dt, weights ? tokens : assignments, ldy, ep);
    if (st != NVFP4_OK) return st;
    if (tokens > 0 && !ids) return NVFP4_ERR_NULL;
    if (!aligned(ids, 4) || !aligned(weights, 4)) return NVFP4_ERR_ALIGN;
    const size_t need = weights ? nvfp4_expert_gemv_workspace_size(tokens, top_k, ep == NVFP4_EPI_SWIGLU ? N / 2 : N) : 0;
    if (need) {
        if (!ws || ws_bytes < need) return NVFP4_ERR_WORKSPACE;
        if (!aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    }
    GemvArgs p = {x, x_rows, ldx, W->codes, W->scales, W->tensor_scale, N, W->cols, y, ldy, ids, (int)assignments, top_k,
                  experts, x_rows != tokens, dt == NVFP4_BF16, y_dt == NVFP4_BF16, W->scale_mode == NVFP4_SCALE_2D, false, 0};
    const hipError_t e = launch_expert_gemv(p, ep == NVFP4_EPI_SWIGLU, weights, static_cast<float*>(ws),
                                            static_cast<hipStream_t>(stream));
    return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

// ---------------------------------------------------------------- the 4-bit cache
namespace {

constexpr int64_t kMaxKvRows = (int64_t)1 << 30;

nvfp4_status check_cache(const nvfp4_kv_cache* c, const nvfp4_kv_plan* p) {
    if (!c || !p) return NVFP4_ERR_NULL;
    if (c->format != NVFP4_KV_NVFP4 && c->format != NVFP4_KV_MXFP4) return NVFP4_ERR_ENUM;
    if (c->pages < 0 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1) return NVFP4_ERR_SHAPE;
    if (p->rows < 0 || p->seqs < 0 || p->width < 0 || p->ld_table < p->width) return NVFP4_ERR_SHAPE;
    if (!p->offsets && p->rows != p->seqs) return NVFP4_ERR_SHAPE;
    const bool mx = c->format == NVFP4_KV_MXFP4;
    if (c->pages > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)) return NVFP4_ERR_NULL;
    if (!mx && (!c->k_scale || !c->v_scale)) return NVFP4_ERR_NULL;
    if (p->seqs > 0 && (!p->lengths || (p->width > 0 && !p->page_table))) return NVFP4_ERR_NULL;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
        !aligned(p->page_table, 4) || !aligned(p->lengths, 4) || !aligned(p->offsets, 4))
        return NVFP4_ERR_ALIGN;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NVFP4_ERR_UNSUPPORTED;
    if (c->page_size < 16 || (c->page_size & (c->page_size - 1))) return NVFP4_ERR_UNSUPPORTED;
    if (c->page_size > kMaxKvRows || p->width > kMaxKvRows / c->page_size || p->rows > kMaxKvRows ||
        p->seqs > kMaxKvSeqs || c->pages > 0x7FFFFFFF)
        return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

// Rows x heads of a call (written: heads that do not overlap).
nvfp4_status check_heads(const nvfp4_kv_rows* r, int64_t rows, int64_t heads, int64_t dim, int32_t dt, bool written) {
    if (!r) return NVFP4_ERR_NULL;
    if (r->row_stride < 0 || r->head_stride < 0) return NVFP4_ERR_SHAPE;
    if (rows > 0 && !r->data) return NVFP4_ERR_NULL;
    if (written && rows > 0) {
        // `inner` pieces of dim, `stride` apart, end before the next one of `outer`
        const auto apart = [dim](int64_t inner, int64_t stride, int64_t outer, int64_t outer_stride) {
            if (inner > 1 && stride < dim) return false;
            if (outer == 1) return true;
            return outer_stride >= dim && (inner == 1 || (outer_stride - dim) / stride >= inner - 1);
        };
        const bool by_row = apart(heads, r->head_stride, rows, r->row_stride);
        const bool by_head = apart(rows, r->row_stride, heads, r->head_stride);
        if (!by_row && !by_head) return NVFP4_ERR_SHAPE;
    }
    return aligned(r->data, dtype_size(dt)) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

KvCache kv_cache_of(const nvfp4_kv_cache* c) {
    const bool mx = c->format == NVFP4_KV_MXFP4;
    return KvCache{c->k_codes, c->k_scales, c->v_codes, c->v_scales, mx ? nullptr : c->k_scale, mx ? nullptr : c->v_scale,
                   (int)c->pages, c->kv_heads, c->head_dim, mx};
}

KvPlan kv_plan_of(const nvfp4_kv_cache* c, const nvfp4_kv_plan* p) {
    return KvPlan{p->page_table, p->ld_table, p->lengths, p->offsets, (int)p->width, __builtin_ctzll(c->page_size),
                  (int)p->seqs, (int)p->rows};
}

KvRows kv_rows_of(const nvfp4_kv_rows* r) { return KvRows{r->data, r->row_stride, r->head_stride}; }

}  // namespace

nvfp4_status nvfp4_kv_append(const nvfp4_kv_rows* k, const nvfp4_kv_rows* v, int32_t dt /* nvfp4_dtype */,
                             const nvfp4_kv_cache* cache, const nvfp4_kv_plan* plan, const nvfp4_kv_rope* rope,
                             const nvfp4_kv_rows* q, int32_t q_heads, nvfp4_kv_rows* q_out, void* stream) {
    if (!valid_dtype(dt)) return NVFP4_ERR_ENUM;
    nvfp4_status st = check_cache(cache, plan);
    if (st != NVFP4_OK) return st;
    const int64_t rows = plan->rows, dim = cache->head_dim;
    if (q_heads < 0 || (q ? q_heads < 1 : q_heads > 0)) return NVFP4_ERR_SHAPE;
    st = check_heads(k, rows, cache->kv_heads, dim, dt, false);
    if (st == NVFP4_OK) st = check_heads(v, rows, cache->kv_heads, dim, dt, false);
    if (st == NVFP4_OK && q) st = check_heads(q, rows, q_heads, dim, dt, false);
    if (st == NVFP4_OK && q) st = check_heads(q_out, rows, q_heads, dim, dt, true);
    if (st != NVFP4_OK) return st;
    KvAppend a = {};
    a.rope_rows = 0x7FFFFFFF;
    if (rope) {
        if (rope->positions < 0 || rope->dim < 1 || rope->ld < rope->dim) return NVFP4_ERR_SHAPE;
        if (rope->positions > 0 && !rope->table) return NVFP4_ERR_NULL;
        if (!aligned(rope->table, 4)) return NVFP4_ERR_ALIGN;
        if (rope->dim < 32 || rope->dim > dim || (rope->dim & (rope->dim - 1))) return NVFP4_ERR_UNSUPPORTED;
        a.rope = rope->table;
        a.rope_ld = rope->ld;
        a.rope_rows = (int)(rope->positions < 0x7FFFFFFF ? rope->positions : 0x7FFFFFFF);
        a.rot = rope->dim;
        a.interleaved = rope->interleaved != 0;
    }
    a.cache = kv_cache_of(cache);
    a.plan = kv_plan_of(cache, plan);
    a.k = kv_rows_of(k);
    a.v = kv_rows_of(v);
    if (q) {
        a.q = kv_rows_of(q);
        a.q_out = {q_out->data, q_out->row_stride, q_out->head_stride};
        a.q_heads = q_heads;
    }
    a.bf16 = dt == NVFP4_BF16;
    if (q_heads > 0x3FFFFFFF - 2 * (int64_t)cache->kv_heads) return NVFP4_ERR_UNSUPPORTED;
    return launch_kv_append(a, static_cast<hipStream_t>(stream)) == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

nvfp4_status nvfp4_kv_gather(const nvfp4_kv_cache* cache, const nvfp4_kv_plan* plan, nvfp4_kv_rows* k,
                             nvfp4_kv_rows* v, int32_t dt /* nvfp4_dtype */, void* stream) {
    if (!valid_dtype(dt)) return NVFP4_ERR_ENUM;
    nvfp4_status st = check_cache(cache, plan);
    if (st == NVFP4_OK) st = check_heads(k, plan->rows, cache->kv_heads, cache->head_dim, dt, true);
    if (st == NVFP4_OK) st = check_heads(v, plan->rows, cache->kv_heads, cache->head_dim, dt, true);
    if (st != NVFP4_OK) return st;
    if (cache->kv_heads > 0x1FFFFFFF) return NVFP4_ERR_UNSUPPORTED;
    const KvGather g = {kv_cache_of(cache), kv_plan_of(cache, plan), kv_rows_of(k), kv_rows_of(v), dt == NVFP4_BF16, 0, 0};
    return launch_kv_gather(g, static_cast<hipStream_t>(stream)) == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

size_t nvfp4_kv_attention_workspace_size(int64_t rows, int64_t seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                         int32_t dt /* nvfp4_dtype */) {
    if (rows < 0 || seqs < 0 || seqs > kMaxKvSeqs || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || !valid_dtype(dt)) return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    if (rows > kMaxKvQueries / q_heads) return 0;
    return kv_attention_workspace_bytes(rows, seqs, q_heads, kv_heads, head_dim, dt == NVFP4_BF16);
}

nvfp4_status nvfp4_kv_attention(const nvfp4_kv_rows* q, int32_t dt /* nvfp4_dtype */, int32_t q_heads,
                                const nvfp4_kv_cache* cache, const nvfp4_kv_plan* plan, float scale, int64_t window,
                                nvfp4_kv_rows* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    if (!valid_dtype(dt)) return NVFP4_ERR_ENUM;
    nvfp4_status st = check_cache(cache, plan);
    if (st != NVFP4_OK) return st;
    if (q_heads < 1 || q_heads % cache->kv_heads || window < 0) return NVFP4_ERR_SHAPE;
    const int64_t rows = plan->rows, dim = cache->head_dim;
    st = check_heads(q, rows, q_heads, dim, dt, false);
    if (st == NVFP4_OK) st = check_heads(out, rows, q_heads, dim, dt, true);
    if (st != NVFP4_OK) return st;
    if (!aligned(lse, 4)) return NVFP4_ERR_ALIGN;
    if (rows > kMaxKvQueries / q_heads) return NVFP4_ERR_UNSUPPORTED;
    const size_t need = nvfp4_kv_attention_workspace_size(rows, plan->seqs, q_heads, cache->kv_heads, cache->head_dim, dt);
    if (need) {
        if (!ws || ws_bytes < need) return NVFP4_ERR_WORKSPACE;
        if (!aligned(ws, 16)) return NVFP4_ERR_ALIGN;
    }
    KvAttention a = {};
    a.cache = kv_cache_of(cache);
    a.plan = kv_plan_of(cache, plan);
    a.q = kv_rows_of(q);
    a.out = {out->data, out->row_stride, out->head_stride};
    a.lse = lse;
    a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    // (a window as long as the longest sequence hides nothing)
    a.window = window < plan->width * cache->page_size ? (int)window : 0;
    a.scale = scale;
    a.bf16 = dt == NVFP4_BF16;
    a.ws = static_cast<float*>(ws);
    return launch_kv_attention(a, static_cast<hipStream_t>(stream)) == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

const char* nvfp4_status_string(int32_t s /* nvfp4_status */) {
    switch (s) {
        case NVFP4_OK: return "ok";
        case NVFP4_ERR_NULL: return "a required pointer is NULL";
        case NVFP4_ERR_ENUM: return "an enum argument is out of range";
        case NVFP4_ERR_SHAPE: return "invalid or inconsistent shape";
        case NVFP4_ERR_ALIGN: return "pointer or leading dimension misaligned";
        case NVFP4_ERR_UNSUPPORTED: return "unsupported combination";
        case NVFP4_ERR_WORKSPACE: return "workspace missing or too small";
        case NVFP4_ERR_HIP: return "HIP launch error";
    }
    return "unknown status";
}

int32_t nvfp4_version(void) { return 100; }

}  // extern "C"
