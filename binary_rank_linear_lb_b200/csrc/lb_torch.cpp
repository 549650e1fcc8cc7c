// Argument marshalling of the dense path for torch tensors: checks, outputs, the
// current stream, the call into liblb.so.  In C++ because a one-token call is as
// short as its marshalling: the same in Python took 8 us of the 13 us of a call
// (three outputs at 1.5 us, checks, ctypes), here about 2.
//
// The functions take their arguments by position (None where optional) and launch
// on the current stream of the tensors' device; the package's functions give them
// their keywords and the stream argument.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "lb.h"

namespace {

PyObject* g_error = nullptr;                       // LbError

using at::Tensor;

const Tensor& tensor(PyObject* o, const char* what) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a tensor");
    return THPVariable_Unpack(o);
}
Tensor optional(PyObject* o, const char* what) { return o == Py_None ? Tensor() : tensor(o, what); }

struct Rows {
    int64_t rows, cols, ld;
};
// A matrix whose rows are contiguous.
Rows rows_of(const Tensor& t, const char* what) {
    TORCH_CHECK_VALUE(t.dim() == 2, what, " must be a matrix with unit stride along its columns");
    const int64_t rows = t.size(0), cols = t.size(1);
    if (t.is_contiguous()) return {rows, cols, cols};
    TORCH_CHECK_VALUE(t.stride(1) == 1 || cols == 1, what, " must be a matrix with unit stride along its columns");
    return {rows, cols, rows > 1 ? t.stride(0) : cols};
}
lb_dtype dtype_of(at::ScalarType t, const char* what) {
    switch (t) {
        case at::kHalf: return LB_F16;
        case at::kBFloat16: return LB_BF16;
        case at::kFloat: return LB_F32;
        default: TORCH_CHECK_VALUE(false, "unsupported ", what, " dtype ", t);
    }
}
void check_vector(const Tensor& t, int64_t n, const char* what) {
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == n && t.is_contiguous(), what, " must be a contiguous vector of ", n,
                      " elements");
}
void check_type(const Tensor& t, at::ScalarType s, const char* what) {
    TORCH_CHECK_VALUE(t.scalar_type() == s, what, " must be ", s);
}

// The GPU that the tensors share, entered; its current stream.
struct Place {
    c10::Device device;
    c10::cuda::OptionalCUDAGuard guard;
    explicit Place(const Tensor& t) : device(t.device()) {
        TORCH_CHECK_VALUE(t.is_cuda(), "all tensors must be on one CUDA device, got ", t.device());
        guard.set_index(device.index());
    }
    void with(const Tensor& t) const {
        TORCH_CHECK_VALUE(!t.defined() || t.device() == device, "all tensors must be on one CUDA device, got ",
                          t.device(), " and ", device);
    }
    Tensor matrix(int64_t rows, int64_t cols, int64_t ld, at::ScalarType t) const {
        const int64_t size[2] = {rows, cols}, stride[2] = {ld, 1};
        return at::detail::empty_strided_cuda(size, stride, t, device);
    }
    Tensor vector(int64_t n, at::ScalarType t) const {
        const int64_t size[1] = {n}, stride[1] = {1};
        return at::detail::empty_strided_cuda(size, stride, t, device);
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
};

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// nullptr with LbError set; `what` is the entry point.
PyObject* fail(lb_status s, const char* what) {
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)s, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}
bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}
PyObject* wrap(const Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
// A tuple of tensors (undefined: None).
PyObject* pack(std::initializer_list<Tensor> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) {
        PyObject* o = wrap(t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// Codes and scales, checked, or new; a new q has a pitch of whole 16-byte pieces,
// which lb_linear_int8's fast kernels read.
int64_t codes(const Place& at_, Tensor& q, Tensor& scale, int64_t rows, int64_t cols) {
    int64_t ldq = (cols + 15) / 16 * 16;
    if (q.defined()) {
        at_.with(q);
        check_type(q, at::kChar, "q");
        const Rows m = rows_of(q, "q");
        TORCH_CHECK_VALUE(m.rows == rows && m.cols == cols, "q must be an int8 matrix of ", rows, " x ", cols);
        ldq = m.ld;
    } else {
        q = at_.matrix(rows, cols, ldq, at::kChar);
    }
    if (scale.defined()) {
        at_.with(scale);
        check_type(scale, at::kFloat, "scale");
        check_vector(scale, rows, "scale");
    } else {
        scale = at_.vector(rows, at::kFloat);
    }
    return ldq;
}

// (x, q, scale) -> (q, scale)
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 3)) return nullptr;
    const Tensor& x = tensor(a[0], "x");
    Tensor q = optional(a[1], "q"), scale = optional(a[2], "scale");
    const Rows m = rows_of(x, "x");
    const lb_dtype dt = dtype_of(x.scalar_type(), "x");
    const Place at_(x);
    const int64_t ldq = codes(at_, q, scale, m.rows, m.cols);
    const lb_status s = lb_quantize_rows(ptr(x), dt, m.rows, m.cols, m.ld, (int8_t*)ptr(q), ldq, (float*)ptr(scale),
                                         at_.stream());
    return s == LB_OK ? pack({q, scale}) : fail(s, "lb_quantize_rows");
    END_HANDLE_TH_ERRORS
}

// (x, weight, residual, eps, sum_out, q, scale) -> (q, scale, sum)
PyObject* rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 7)) return nullptr;
    const Tensor& x = tensor(a[0], "x");
    const Tensor weight = optional(a[1], "weight"), residual = optional(a[2], "residual");
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    Tensor sum = optional(a[4], "sum_out"), q = optional(a[5], "q"), scale = optional(a[6], "scale");
    const Rows m = rows_of(x, "x");
    const lb_dtype dt = dtype_of(x.scalar_type(), "x");
    const Place at_(x);
    lb_dtype wdt = LB_F32;
    if (weight.defined()) {
        at_.with(weight);
        check_vector(weight, m.cols, "weight");
        wdt = dtype_of(weight.scalar_type(), "weight");
    }
    int64_t ldr = 0, lds = 0;
    auto like_x = [&](const Tensor& t, const char* what) {
        at_.with(t);
        const Rows r = rows_of(t, what);
        TORCH_CHECK_VALUE(r.rows == m.rows && r.cols == m.cols && t.scalar_type() == x.scalar_type(), what,
                          " must have x's shape and dtype");
        return r.ld;
    };
    if (residual.defined()) {
        ldr = like_x(residual, "residual");
        if (sum.defined()) {
            lds = like_x(sum, "sum_out");
        } else {
            lds = m.cols;
            sum = at_.matrix(m.rows, m.cols, m.cols, x.scalar_type());
        }
    } else {
        TORCH_CHECK_VALUE(!sum.defined(), "sum_out needs a residual");
    }
    const int64_t ldq = codes(at_, q, scale, m.rows, m.cols);
    const lb_status s =
        lb_rmsnorm_quantize(ptr(x), dt, m.rows, m.cols, m.ld, ptr(residual), ldr, ptr(sum), lds, ptr(weight), wdt,
                            (float)eps, (int8_t*)ptr(q), ldq, (float*)ptr(scale), at_.stream());
    return s == LB_OK ? pack({q, scale, sum}) : fail(s, "lb_rmsnorm_quantize");
    END_HANDLE_TH_ERRORS
}

// (xq, xs, wq, ws, y, dtype) -> y
PyObject* linear_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 6)) return nullptr;
    const Tensor &xq = tensor(a[0], "xq"), &xs = tensor(a[1], "xs"), &wq = tensor(a[2], "wq"), &ws = tensor(a[3], "ws");
    Tensor y = optional(a[4], "y");
    const Rows x = rows_of(xq, "xq"), w = rows_of(wq, "wq");
    TORCH_CHECK_VALUE(xq.scalar_type() == at::kChar && wq.scalar_type() == at::kChar && x.cols == w.cols,
                      "xq and wq must be int8 matrices with the same number of columns");
    check_type(xs, at::kFloat, "xs");
    check_type(ws, at::kFloat, "ws");
    check_vector(xs, x.rows, "xs");
    check_vector(ws, w.rows, "ws");
    const Place at_(xq);
    at_.with(xs);
    at_.with(wq);
    at_.with(ws);
    int64_t ldy = w.rows;
    if (y.defined()) {
        at_.with(y);
        const Rows m = rows_of(y, "y");
        TORCH_CHECK_VALUE(m.rows == x.rows && m.cols == w.rows, "y must be ", x.rows, " x ", w.rows);
        ldy = m.ld;
        dtype_of(y.scalar_type(), "y");
    } else {
        TORCH_CHECK_TYPE(THPDtype_Check(a[5]), "dtype must be a torch.dtype");
        const at::ScalarType t = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
        dtype_of(t, "y");
        y = at_.matrix(x.rows, w.rows, w.rows, t);
    }
    const lb_status s = lb_linear_int8((const int8_t*)ptr(xq), x.ld, (const float*)ptr(xs), x.rows,
                                       (const int8_t*)ptr(wq), w.ld, (const float*)ptr(ws), x.cols, w.rows, ptr(y),
                                       dtype_of(y.scalar_type(), "y"), ldy, at_.stream());
    return s == LB_OK ? wrap(y) : fail(s, "lb_linear_int8");
    END_HANDLE_TH_ERRORS
}

// (logits, tokens, top) -> (logprob, entropy, top_id, top_logprob)
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arity(n, 3)) return nullptr;
    const Tensor& x = tensor(a[0], "logits");
    const Tensor tokens = optional(a[1], "tokens");
    const long top = PyLong_AsLong(a[2]);
    if (top == -1 && PyErr_Occurred()) return nullptr;
    const Rows m = rows_of(x, "logits");
    const lb_dtype dt = dtype_of(x.scalar_type(), "logits");
    TORCH_CHECK_VALUE(top >= 0 && top <= 32 && (top <= m.cols || m.cols == 0), "top must be 0 .. ",
                      std::min<int64_t>(32, m.cols));
    const Place at_(x);
    Tensor logprob, top_id, top_lp;
    if (tokens.defined()) {
        at_.with(tokens);
        check_type(tokens, at::kLong, "tokens");
        check_vector(tokens, m.rows, "tokens");
        logprob = at_.vector(m.rows, at::kFloat);
    }
    const Tensor entropy = at_.vector(m.rows, at::kFloat);
    if (top > 0) {
        top_id = at_.matrix(m.rows, top, top, at::kLong);
        top_lp = at_.matrix(m.rows, top, top, at::kFloat);
    }
    const lb_status s = lb_token_logprobs(ptr(x), dt, m.rows, m.cols, m.ld, (const int64_t*)ptr(tokens),
                                          (float*)ptr(logprob), (float*)ptr(entropy), (int)top, (int64_t*)ptr(top_id),
                                          (float*)ptr(top_lp), at_.stream());
    return s == LB_OK ? pack({logprob, entropy, top_id, top_lp}) : fail(s, "lb_token_logprobs");
    END_HANDLE_TH_ERRORS
}

// The class that a call raises when the library refuses it: error(status, entry point).
PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

#define LB_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {
    {"quantize_rows", LB_FAST(quantize_rows)},       {"rmsnorm_quantize", LB_FAST(rmsnorm_quantize)},
    {"linear_int8", LB_FAST(linear_int8)},           {"token_logprobs", LB_FAST(token_logprobs)},
    {"set_error", set_error, METH_O, nullptr},       {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "lb_torch", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit_lb_torch() { return PyModule_Create(&g_module); }
