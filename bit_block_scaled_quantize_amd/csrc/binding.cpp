// Python entry points of the MoE-block operators over the C ABI
// (include/nvfp4.h): argument checks, output and workspace allocation with
// torch, and the call.  nvfp4.py gives them their names, defaults and result
// types.  These operators are called once or more for every layer and token;
// marshalled in Python (ctypes, torch.empty), a call costs the host 10 to 18 us
// where its kernels take 3 to 8.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "nvfp4.h"

namespace {

PyObject* g_error = nullptr;           // NVFP4Error
PyObject* g_current_device = nullptr;  // torch._C._cuda_getDevice
PyObject* g_current_stream = nullptr;  // torch._C._cuda_getCurrentRawStream

// A Python exception is set.
struct Raised : python_error {
    Raised() { persist(); }
};

const at::Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}

int32_t small(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, " is out of range");
    return (int32_t)v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v != 0;
}

bool given(PyObject* o) { return o != Py_None; }

int32_t code_of(at::ScalarType t) {
    TORCH_CHECK_TYPE(t == at::kFloat || t == at::kBFloat16, "unsupported dtype ", t);
    return t == at::kFloat ? NVFP4_F32 : NVFP4_BF16;
}

void same_device(const char* name, const at::Tensor& t, const at::Tensor& like) {
    TORCH_CHECK_VALUE(t.device() == like.device(), name, " is on ", t.device(), ", expected ", like.device());
}

// Leading dimension of a 2-D tensor with unit column stride.
int64_t matrix(const char* name, const at::Tensor& t) {
    TORCH_CHECK_VALUE(t.dim() == 2 && (t.stride(1) == 1 || t.size(1) <= 1), name,
                      " must be a matrix with unit column stride");
    return t.size(0) > 1 ? t.stride(0) : std::max(t.size(1), t.stride(0));
}

int64_t matrix(const char* name, const at::Tensor& t, int64_t rows, int64_t cols, at::ScalarType dtype,
               const at::Tensor& like) {
    const int64_t ld = matrix(name, t);
    TORCH_CHECK_VALUE(t.size(0) == rows && t.size(1) == cols, name, " is ", t.size(0), " x ", t.size(1), ", expected ",
                      rows, " x ", cols);
    TORCH_CHECK_TYPE(t.scalar_type() == dtype, name, " has dtype ", t.scalar_type(), ", expected ", dtype);
    same_device(name, t, like);
    return ld;
}

// Address of a contiguous tensor of n elements.
void* flat(const char* name, const at::Tensor& t, int64_t n, at::ScalarType dtype, const at::Tensor& like) {
    TORCH_CHECK_VALUE(t.numel() == n && t.is_contiguous(), name, " must be contiguous with ", n, " elements");
    TORCH_CHECK_TYPE(t.scalar_type() == dtype, name, " has dtype ", t.scalar_type(), ", expected ", dtype);
    same_device(name, t, like);
    return t.data_ptr();
}

template <typename T>
T* flat(PyObject* o, const char* name, int64_t n, at::ScalarType dtype, const at::Tensor& like) {
    return given(o) ? static_cast<T*>(flat(name, tensor(o, name), n, dtype, like)) : nullptr;
}

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype, const at::Tensor& like) {
    return at::empty(sizes, like.options().dtype(dtype));
}

// The tensor given, or a new one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef sizes, at::ScalarType dtype, const at::Tensor& like) {
    return given(o) ? tensor(o, name) : empty(sizes, dtype, like);
}

// Handle of the stream a call on the tensors of t's device runs on: that given
// (an integer), or torch's current one.
void* stream_of(const at::Tensor& t, PyObject* stream) {
    TORCH_CHECK_VALUE(t.is_cuda(), "the tensors must be on the current GPU, got ", t.device());
    PyObject* current = PyObject_CallNoArgs(g_current_device);
    if (!current) throw Raised();
    const long dev = PyLong_AsLong(current);
    Py_DECREF(current);
    TORCH_CHECK_VALUE(t.get_device() == dev, "the tensors must be on the current GPU, got ", t.device());
    if (given(stream)) return reinterpret_cast<void*>(integer(stream));
    PyObject* index = PyLong_FromLong(dev);
    PyObject* handle = index ? PyObject_CallOneArg(g_current_stream, index) : nullptr;
    Py_XDECREF(index);
    if (!handle) throw Raised();
    void* s = reinterpret_cast<void*>(integer(handle));
    Py_DECREF(handle);
    return s;
}

void check(const char* fn, nvfp4_status st) {
    if (st == NVFP4_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "si", fn, (int)st);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised();
}

// A workspace: the tensor given, or `need` bytes of a new one (kept alive by
// `hold`).
struct Workspace {
    void* ptr = nullptr;
    size_t bytes = 0;
    at::Tensor hold;
    Workspace(PyObject* o, size_t need, const at::Tensor& like) {
        if (given(o)) {
            hold = tensor(o, "workspace");
            same_device("workspace", hold, like);
            TORCH_CHECK_VALUE(hold.is_contiguous(), "workspace must be contiguous");
        } else if (need) {
            hold = empty({(int64_t)need}, at::kByte, like);
        } else {
            return;
        }
        ptr = hold.data_ptr();
        bytes = hold.nbytes();
    }
};

PyObject* wrapped(const at::Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

template <int N>
PyObject* tuple(const at::Tensor (&t)[N]) {
    PyObject* r = PyTuple_New(N);
    if (!r) throw Raised();
    for (int i = 0; i < N; ++i) {
        PyObject* o = wrapped(t[i]);
        if (!o) {
            Py_DECREF(r);
            throw Raised();
        }
        PyTuple_SET_ITEM(r, i, o);
    }
    return r;
}

void expect(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// (x, weight, residual, eps, y, mx_elem or -1, rstd, h, y, codes, scales, rstd
// to fill, stream) -> (h, y, codes, scales, rstd)
PyObject* rmsnorm(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 13);
    const at::Tensor& x = tensor(v[0], "x");
    const int64_t ldx = matrix("x", x), rows = x.size(0), cols = x.size(1);
    const at::ScalarType dt = x.scalar_type();
    const int32_t code = code_of(dt);
    const at::Tensor& weight = tensor(v[1], "weight");
    const int32_t w_code = code_of(weight.scalar_type());
    void* w = flat("weight", weight, cols, weight.scalar_type(), x);
    const at::Tensor* residual = given(v[2]) ? &tensor(v[2], "residual") : nullptr;
    const int64_t ldr = residual ? matrix("residual", *residual, rows, cols, dt, x) : 0;
    const double eps = PyFloat_AsDouble(v[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised();
    const int32_t elem = small(v[5], "mx_elem");
    void* s = stream_of(x, v[12]);
    at::Tensor out[5];
    int64_t ldh = 0, ldy = 0;
    if (residual) {
        out[0] = output(v[7], "out.h", {rows, cols}, dt, x);
        ldh = matrix("out.h", out[0], rows, cols, dt, x);
    } else {
        out[0] = x;
    }
    if (truth(v[4])) {
        out[1] = output(v[8], "out.y", {rows, cols}, dt, x);
        ldy = matrix("out.y", out[1], rows, cols, dt, x);
    }
    nvfp4_mx_tensor mx = {nullptr, nullptr, rows, cols, elem};
    if (elem != -1) {
        const int64_t width = elem == NVFP4_MX_E2M1 ? cols / 2 : cols;
        out[2] = output(v[9], "out.mx.codes", {rows, width}, at::kByte, x);
        out[3] = output(v[10], "out.mx.scales", {rows, cols / 32}, at::kByte, x);
        mx.codes = static_cast<uint8_t*>(flat("out.mx.codes", out[2], rows * width, at::kByte, x));
        mx.scales = static_cast<uint8_t*>(flat("out.mx.scales", out[3], rows * (cols / 32), at::kByte, x));
    }
    float* rstd = nullptr;
    if (truth(v[6])) {
        out[4] = output(v[11], "out.rstd", {rows}, at::kFloat, x);
        rstd = static_cast<float*>(flat("out.rstd", out[4], rows, at::kFloat, x));
    }
    check("nvfp4_rmsnorm",
          nvfp4_rmsnorm(x.data_ptr(), ldx, residual ? residual->data_ptr() : nullptr, ldr, w, w_code, code, rows, cols,
                        (float)eps, residual ? out[0].data_ptr() : nullptr, ldh,
                        out[1].defined() ? out[1].data_ptr() : nullptr, ldy, elem != -1 ? &mx : nullptr, rstd, s));
    return tuple(out);
    END_HANDLE_TH_ERRORS
}

// (dy, h, rstd, weight, dh, dx, dweight, workspace, stream) -> (dx, dweight)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 9);
    const at::Tensor& h = tensor(v[1], "h");
    const int64_t ldh = matrix("h", h), rows = h.size(0), cols = h.size(1);
    const at::ScalarType dt = h.scalar_type();
    const int32_t code = code_of(dt);
    const at::Tensor &dy = tensor(v[0], "dy"), &weight = tensor(v[3], "weight");
    const int64_t lddy = matrix("dy", dy, rows, cols, dt, h);
    const float* rstd = static_cast<float*>(flat("rstd", tensor(v[2], "rstd"), rows, at::kFloat, h));
    const int32_t w_code = code_of(weight.scalar_type());
    void* w = flat("weight", weight, cols, weight.scalar_type(), h);
    const at::Tensor* dh = given(v[4]) ? &tensor(v[4], "dh") : nullptr;
    const int64_t lddh = dh ? matrix("dh", *dh, rows, cols, dt, h) : 0;
    void* s = stream_of(h, v[8]);
    const at::Tensor out[2] = {output(v[5], "dx", {rows, cols}, dt, h), output(v[6], "dweight", {cols}, at::kFloat, h)};
    const int64_t lddx = matrix("dx", out[0], rows, cols, dt, h);
    float* dweight = static_cast<float*>(flat("dweight", out[1], cols, at::kFloat, h));
    const Workspace ws(v[7], nvfp4_rmsnorm_backward_workspace_size(rows, cols), h);
    check("nvfp4_rmsnorm_backward",
          nvfp4_rmsnorm_backward(dy.data_ptr(), lddy, h.data_ptr(), ldh, rstd, w, w_code, dh ? dh->data_ptr() : nullptr,
                                 lddh, code, rows, cols, out[0].data_ptr(), lddx, dweight, ws.ptr, ws.bytes, s));
    return tuple(out);
    END_HANDLE_TH_ERRORS
}

// (logits, top_k, bias, score, groups, top_groups, group_score, renorm, plan,
// ids, weights, offsets, order, position to fill, workspace, stream) -> (ids,
// weights, offsets, order, position)
PyObject* route(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 16);
    const at::Tensor& l = tensor(v[0], "logits");
    const int64_t ld = matrix("logits", l), tokens = l.size(0), experts = l.size(1);
    const int32_t code = code_of(l.scalar_type()), top_k = small(v[1], "top_k");
    TORCH_CHECK_VALUE(top_k >= 0, "top_k is negative");
    const int64_t a = tokens * top_k;
    nvfp4_route_opts o = {};
    o.top_k = top_k;
    o.score = small(v[3], "score");
    o.groups = small(v[4], "groups");
    o.top_groups = small(v[5], "top_groups");
    o.group_score = small(v[6], "group_score");
    o.renorm = truth(v[7]);
    o.bias = flat<float>(v[2], "bias", experts, at::kFloat, l);
    const bool plan = truth(v[8]);
    void* s = stream_of(l, v[15]);
    at::Tensor out[5];
    out[0] = output(v[9], "out.ids", {tokens, top_k}, at::kInt, l);
    out[1] = output(v[10], "out.weights", {tokens, top_k}, at::kFloat, l);
    int32_t* ids = static_cast<int32_t*>(flat("out.ids", out[0], a, at::kInt, l));
    float* weights = static_cast<float*>(flat("out.weights", out[1], a, at::kFloat, l));
    int64_t* offsets = nullptr;
    int32_t *order = nullptr, *position = nullptr;
    if (plan) {
        out[2] = output(v[11], "out.offsets", {experts + 1}, at::kLong, l);
        out[3] = output(v[12], "out.order", {a}, at::kInt, l);
        out[4] = output(v[13], "out.position", {a}, at::kInt, l);
        offsets = static_cast<int64_t*>(flat("out.offsets", out[2], experts + 1, at::kLong, l));
        order = static_cast<int32_t*>(flat("out.order", out[3], a, at::kInt, l));
        position = static_cast<int32_t*>(flat("out.position", out[4], a, at::kInt, l));
    }
    const Workspace ws(v[14], plan ? nvfp4_route_workspace_size(tokens, experts) : 0, l);
    check("nvfp4_route", nvfp4_route(l.data_ptr(), code, tokens, experts, ld, &o, ids, weights, offsets, order, position,
                                     ws.ptr, ws.bytes, s));
    return tuple(out);
    END_HANDLE_TH_ERRORS
}

// (dweights, logits, ids, score, renorm, dscores, out, stream) -> dlogits
PyObject* route_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 8);
    const at::Tensor &l = tensor(v[1], "logits"), &ids = tensor(v[2], "ids");
    const int64_t ld = matrix("logits", l), tokens = l.size(0), experts = l.size(1);
    TORCH_CHECK_VALUE(ids.dim() == 2, "ids must be tokens x top_k");
    const int64_t top_k = ids.size(1);
    TORCH_CHECK_VALUE(top_k <= INT32_MAX, "top_k is out of range");
    const int32_t code = code_of(l.scalar_type());
    const int32_t* pi = static_cast<int32_t*>(flat("ids", ids, tokens * top_k, at::kInt, l));
    const float* pw = static_cast<float*>(flat("dweights", tensor(v[0], "dweights"), tokens * top_k, at::kFloat, l));
    const at::Tensor* ds = given(v[5]) ? &tensor(v[5], "dscores") : nullptr;
    const int64_t ldds = ds ? matrix("dscores", *ds, tokens, experts, at::kFloat, l) : 0;
    const int32_t score = small(v[3], "score");
    const bool renorm = truth(v[4]);
    void* s = stream_of(l, v[7]);
    const at::Tensor out = output(v[6], "out", {tokens, experts}, l.scalar_type(), l);
    const int64_t lddl = matrix("out", out, tokens, experts, l.scalar_type(), l);
    check("nvfp4_route_backward",
          nvfp4_route_backward(pw, l.data_ptr(), code, tokens, experts, ld, pi, (int32_t)top_k, score, renorm,
                               ds ? static_cast<float*>(ds->data_ptr()) : nullptr, ldds, out.data_ptr(), lddl, s));
    return wrapped(out);
    END_HANDLE_TH_ERRORS
}

// A 4-bit weight's arrays: (codes, scales, tensor_scale, rows, cols,
// scale_mode) from v; n_scales tensor scales.
nvfp4_tensor weight_of(PyObject* const* v, int64_t n_scales, const at::Tensor& x) {
    nvfp4_tensor w = {};
    w.rows = integer(v[3]);
    w.cols = integer(v[4]);
    w.scale_mode = small(v[5], "scale_mode");
    const int64_t scale_rows = w.scale_mode == NVFP4_SCALE_2D ? w.rows / 16 : w.rows;
    w.codes = flat<uint8_t>(v[0], "codes", w.rows * (w.cols / 2), at::kByte, x);
    w.scales = flat<uint8_t>(v[1], "scales", scale_rows * (w.cols / 16), at::kByte, x);
    w.tensor_scale = flat<float>(v[2], "tensor_scale", n_scales, at::kFloat, x);
    return w;
}

// Leading dimension of the rows that a weight of `cols` columns multiplies.
int64_t input(const at::Tensor& x, int64_t cols) {
    const int64_t ld = matrix("x", x);
    TORCH_CHECK_VALUE(x.size(1) == cols, "x is ", x.size(0), " x ", x.size(1), ", expected ", cols, " columns");
    return ld;
}

// Output of rows x cols: given, or new in the dtype of `code` (-1: x's).
at::Tensor product(PyObject* o, int64_t rows, int64_t cols, int64_t code, const at::Tensor& x, int64_t& ld) {
    const at::Tensor out =
        output(o, "out", {rows, cols}, code < 0 ? x.scalar_type() : code == NVFP4_F32 ? at::kFloat : at::kBFloat16, x);
    ld = matrix("out", out, rows, cols, out.scalar_type(), x);
    return out;
}

// (x, codes, scales, tensor_scale, rows, cols, scale_mode, epilogue, dtype code
// or -1, out, stream) -> y
PyObject* gemv(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 11);
    const at::Tensor& x = tensor(v[0], "x");
    const int64_t ldx = input(x, integer(v[5]));
    const int32_t code = code_of(x.scalar_type()), ep = small(v[7], "epilogue");
    const nvfp4_tensor w = weight_of(v + 1, 1, x);
    void* s = stream_of(x, v[10]);
    int64_t ldy;
    const at::Tensor y = product(v[9], x.size(0), ep == NVFP4_EPI_SWIGLU ? w.rows / 2 : w.rows, integer(v[8]), x, ldy);
    check("nvfp4_gemv",
          nvfp4_gemv(x.data_ptr(), code, x.size(0), ldx, &w, y.data_ptr(), code_of(y.scalar_type()), ldy, ep, s));
    return wrapped(y);
    END_HANDLE_TH_ERRORS
}

// (x, codes, scales, rows, cols, elem, dtype code or -1, out, stream) -> y
PyObject* mx_gemv(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 9);
    const at::Tensor& x = tensor(v[0], "x");
    nvfp4_mx_tensor w = {};
    w.rows = integer(v[3]);
    w.cols = integer(v[4]);
    w.elem = small(v[5], "elem");
    const int64_t ldx = input(x, w.cols);
    const int32_t code = code_of(x.scalar_type());
    TORCH_CHECK_VALUE(w.elem == NVFP4_MX_E2M1, "the weight must have E2M1 elements");
    w.codes = flat<uint8_t>(v[1], "codes", w.rows * (w.cols / 2), at::kByte, x);
    w.scales = flat<uint8_t>(v[2], "scales", w.rows * (w.cols / 32), at::kByte, x);
    void* s = stream_of(x, v[8]);
    int64_t ldy;
    const at::Tensor y = product(v[7], x.size(0), w.rows, integer(v[6]), x, ldy);
    check("nvfp4_mx_gemv",
          nvfp4_mx_gemv(x.data_ptr(), code, x.size(0), ldx, &w, y.data_ptr(), code_of(y.scalar_type()), ldy, s));
    return wrapped(y);
    END_HANDLE_TH_ERRORS
}

// (x, ids, codes, scales, tensor_scale, rows, cols, scale_mode, experts,
// weights, epilogue, dtype code or -1, out, workspace, stream) -> y
PyObject* expert_gemv(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 15);
    const at::Tensor &x = tensor(v[0], "x"), &ids = tensor(v[1], "ids");
    TORCH_CHECK_VALUE(ids.dim() == 2, "ids must be tokens x top_k");
    const int64_t tokens = ids.size(0), top_k = ids.size(1), a = tokens * top_k, ldx = input(x, integer(v[6]));
    TORCH_CHECK_VALUE(x.size(0) == tokens || x.size(0) == a, "x must have a row for each token or for each assignment");
    TORCH_CHECK_VALUE(top_k <= INT32_MAX, "top_k is out of range");
    const int32_t code = code_of(x.scalar_type()), experts = small(v[8], "experts"), ep = small(v[10], "epilogue");
    TORCH_CHECK_VALUE(experts > 0, "experts must be positive");
    const nvfp4_tensor w = weight_of(v + 2, experts, x);
    const int32_t* pi = static_cast<int32_t*>(flat("ids", ids, a, at::kInt, x));
    const float* pw = flat<float>(v[9], "weights", a, at::kFloat, x);
    void* s = stream_of(x, v[14]);
    const int64_t cols = w.rows / experts / (ep == NVFP4_EPI_SWIGLU ? 2 : 1);
    int64_t ldy;
    const at::Tensor y = product(v[12], pw ? tokens : a, cols, integer(v[11]), x, ldy);
    const Workspace ws(v[13], pw ? nvfp4_expert_gemv_workspace_size(tokens, (int32_t)top_k, cols) : 0, x);
    check("nvfp4_expert_gemv",
          nvfp4_expert_gemv(x.data_ptr(), code, x.size(0), ldx, pi, tokens, (int32_t)top_k, &w, experts, pw, y.data_ptr(),
                            code_of(y.scalar_type()), ldy, ep, ws.ptr, ws.bytes, s));
    return wrapped(y);
    END_HANDLE_TH_ERRORS
}

// (NVFP4Error, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
PyObject* setup(PyObject*, PyObject* const* v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 3);
    PyObject** slots[3] = {&g_error, &g_current_device, &g_current_stream};
    for (int i = 0; i < 3; ++i) {
        Py_INCREF(v[i]);
        Py_XDECREF(*slots[i]);
        *slots[i] = v[i];
    }
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define NVFP4_ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {NVFP4_ENTRY(setup),          NVFP4_ENTRY(rmsnorm), NVFP4_ENTRY(rmsnorm_backward),
                         NVFP4_ENTRY(route),          NVFP4_ENTRY(route_backward), NVFP4_ENTRY(gemv),
                         NVFP4_ENTRY(mx_gemv),        NVFP4_ENTRY(expert_gemv),    {nullptr, nullptr, 0, nullptr}};
#undef NVFP4_ENTRY

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
