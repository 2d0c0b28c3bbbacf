// Torch-facing calls of the MXFP4, Newton-Schulz, 8-bit integer and gated entry points: argument
// checks on tensors, outputs and scratch from torch's allocator on the current
// stream, one call of the C-ABI each.
//
// Written against the CPython and ATen interfaces because these calls are
// short: quantising one token's activations takes the GPU about 2 us, and the
// same checks and allocations made from Python take the host 14 us a call
// (ctypes with 20 arguments, five tensor attributes per operand), from here
// 4 to 5 us, launch included (gemm_mxfp4_dyn, one token, 4096 x 4096: 3.9 to 4.5 us a
// call in a row of them, about what its kernel takes).
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/hip/HIPStream.h>

#include <cstring>
#include <string>

#include "mpgemm.h"

namespace {

// A Python exception has been set.
struct Raised {};

[[noreturn]] void fail(PyObject *type, const std::string &what) {
    PyErr_SetString(type, what.c_str());
    throw Raised();
}

PyObject *package() {
    static PyObject *m = PyImport_ImportModule("precision_dense_gemm_tiled_amd");
    if (!m)
        throw Raised();
    return m;
}

void check(int status, const char *what) {
    if (status == MPGEMM_OK)
        return;
    PyObject *cls = PyObject_GetAttrString(package(), "MpgemmError");
    if (!cls)
        throw Raised();
    PyObject *e = PyObject_CallFunction(cls, "is", status, what);
    if (e) {
        PyErr_SetObject(cls, e);
        Py_DECREF(e);
    }
    Py_DECREF(cls);
    throw Raised();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o))
        fail(PyExc_TypeError, std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}

// The calls that return floating-point results take no part in autograd: a gradient or a tangent
// (of forward mode, which no_grad does not end) that the caller would miss is an error, as it is for torch's own out= forms.
void no_gradient(const at::Tensor &t, const char *name) {
    if (c10::GradMode::is_enabled() && t.requires_grad())
        fail(PyExc_RuntimeError, std::string(name) + " requires grad, but this call takes no part in autograd: "
                                                     "detach it, call under torch.no_grad() or from an autograd.Function");
    if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
        fail(PyExc_RuntimeError, std::string(name) + " has a tangent, but this call takes no part in autograd: "
                                                     "unpack the dual tensor or call from an autograd.Function");
}

int type_of(at::ScalarType t, const char *name, bool f32 = true) {
    if (t == at::kHalf)
        return MPGEMM_TYPE_F16;
    if (t == at::kBFloat16)
        return MPGEMM_TYPE_BF16;
    if (t == at::kFloat && f32)
        return MPGEMM_TYPE_F32;
    fail(PyExc_TypeError, std::string(name) + ": expected float16, bfloat16" + (f32 ? " or float32" : "") + ", got " +
                              c10::toString(t));
}

// Row stride of a 2-D device tensor with contiguous rows.
int64_t rows_of(const at::Tensor &t, at::ScalarType type, const char *name) {
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, std::string(name) + ": expected " + c10::toString(type) + ", got " +
                                  c10::toString(t.scalar_type()));
    if (t.dim() != 2)
        fail(PyExc_ValueError, std::string(name) + ": expected a 2-D tensor");
    if (!t.is_cuda())
        fail(PyExc_ValueError, std::string(name) + ": expected a device tensor");
    if (t.size(1) > 1 && t.stride(1) != 1)
        fail(PyExc_ValueError, std::string(name) + ": rows must be contiguous (stride(1) == 1)");
    return t.size(0) > 1 ? t.stride(0) : std::max<int64_t>(t.size(1), 1);
}

int64_t blocks_of(int64_t k) { return (k + 31) / 32; }

// (torch.empty without its way through the dispatcher)
at::Tensor empty(at::IntArrayRef size, at::ScalarType type, const at::Device &dev) {
    return at::Tensor(at::detail::empty_cuda(size, type, dev, std::nullopt));
}

// Codes and scales of rows of k elements, and their row strides in bytes.
struct Held {
    uint8_t *q = nullptr, *s = nullptr;
    int64_t ldq = 0, lds = 0, rows = 0;
    at::Tensor padded;   // the scales' copy, where there is one
};

Held held(PyObject *oq, PyObject *os, int64_t k, const char *name, const at::Device &dev) {
    const at::Tensor &q = tensor(oq, name), &s = tensor(os, name);
    Held h;
    h.ldq = rows_of(q, at::kByte, name);
    h.lds = rows_of(s, at::kByte, name);
    h.rows = q.size(0);
    const int64_t nb = blocks_of(k);
    if (q.size(1) != 16 * nb || s.size(1) != nb || s.size(0) != h.rows)
        fail(PyExc_ValueError, std::string(name) + ": codes of " + std::to_string(h.rows) + " x " +
                                   std::to_string(q.size(1)) + " and scales of " + std::to_string(s.size(0)) + " x " +
                                   std::to_string(s.size(1)) + " for rows of " + std::to_string(k) + " elements");
    if (q.device() != dev || s.device() != dev)
        fail(PyExc_ValueError, std::string(name) + ": not on " + dev.str());
    if (h.rows <= 1)   // (a row stride that is not used)
        h.lds = (h.lds + 15) / 16 * 16;
    h.q = static_cast<uint8_t *>(q.data_ptr());
    h.s = static_cast<uint8_t *>(s.data_ptr());
    // Copies of the scales that a call returned (clone, contiguous, to the host and back) have
    // lost the padding of their rows: they get it again here, in a launch of its own.
    if (h.rows > 0 && nb > 0 && (h.lds % 16 != 0 || (reinterpret_cast<uintptr_t>(h.s) & 15) != 0)) {
        h.lds = (nb + 15) / 16 * 16;
        h.padded = empty({h.rows, h.lds}, at::kByte, dev);
        h.padded.narrow(1, 0, nb).copy_(s);
        h.s = static_cast<uint8_t *>(h.padded.data_ptr());
    }
    return h;
}

const void *bias_of(PyObject *o, int64_t n, at::ScalarType type, const at::Device &dev) {
    if (o == Py_None)
        return nullptr;
    const at::Tensor &b = tensor(o, "bias");
    no_gradient(b, "bias");
    if (b.scalar_type() != type || b.dim() != 1 || b.size(0) != n || !b.is_contiguous() || b.device() != dev)
        fail(PyExc_ValueError, "bias: expected " + std::to_string(n) + " contiguous " + c10::toString(type) +
                                   " values on " + dev.str());
    return b.data_ptr();
}

// The result (new, or the caller's) and its row stride.
at::Tensor result(PyObject *out, int64_t rows, int64_t cols, at::ScalarType type, const at::Device &dev, int64_t &ld) {
    if (out == Py_None) {
        ld = std::max<int64_t>(cols, 1);
        return empty({rows, cols}, type, dev);
    }
    const at::Tensor &t = tensor(out, "out");
    no_gradient(t, "out");
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || t.device() != dev)
        fail(PyExc_ValueError, "out: expected " + std::to_string(rows) + " x " + std::to_string(cols) + " on " + dev.str());
    ld = rows_of(t, type, "out");
    return t;
}

// New codes and scales, in one allocation; the scale rows are padded to 16 bytes.
struct NewHeld {
    at::Tensor q, s;
    NewHeld(int64_t rows, int64_t k, const at::Device &dev) {
        const int64_t nb = blocks_of(k), lds = (nb + 15) / 16 * 16;
        q = empty({rows * (16 * nb + lds)}, at::kByte, dev);
        s = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(q.storage()), q.key_set(), q.dtype());
        q.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef{rows, 16 * nb}, at::IntArrayRef{16 * nb, 1});
        s.unsafeGetTensorImpl()->set_storage_offset(rows * 16 * nb);
        s.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef{rows, nb}, at::IntArrayRef{lds, 1});
    }
};

at::Tensor scratch(int64_t bytes, const at::Device &dev, const char *what) {
    if (bytes < 0)
        check(MPGEMM_ERR_UNSUPPORTED, what);
    return bytes ? empty({bytes}, at::kByte, dev) : at::Tensor();
}

void *pointer(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

void *stream_of(const at::Device &dev) { return c10::hip::getCurrentHIPStream(dev.index()).stream(); }

constexpr int kMaxDevices = 64;

int cu_count(const at::Device &dev) {
    static int known[kMaxDevices];
    const int i = dev.index();
    if (i < 0 || i >= kMaxDevices)
        fail(PyExc_ValueError, "device " + dev.str() + " out of range");
    if (!known[i]) {
        PyObject *n = PyObject_CallMethod(package(), "_cu_count", "i", i);
        if (!n)
            throw Raised();
        known[i] = (int)PyLong_AsLong(n);
        Py_DECREF(n);
    }
    return known[i];
}

// The caller's handle, or the device's default one.
mpgemm_handle_t handle_of(PyObject *o, const at::Device &dev) {
    if (o != Py_None) {
        void *h = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred())
            throw Raised();
        return static_cast<mpgemm_handle_t>(h);
    }
    static mpgemm_handle_t known[kMaxDevices];
    const int i = dev.index();
    if (i < 0 || i >= kMaxDevices)
        fail(PyExc_ValueError, "device " + dev.str() + " out of range");
    if (!known[i]) {
        PyObject *h = PyObject_CallMethod(package(), "default_handle", "i", i);
        if (!h)
            throw Raised();
        known[i] = static_cast<mpgemm_handle_t>(PyLong_AsVoidPtr(h));
        Py_DECREF(h);
    }
    return known[i];
}

at::ScalarType dtype_of(PyObject *o, PyObject *out) {
    if (o != Py_None) {
        if (!THPDtype_Check(o))
            fail(PyExc_TypeError, "dtype: expected a torch.dtype");
        return reinterpret_cast<THPDtype *>(o)->scalar_type;
    }
    return out == Py_None ? at::kFloat : tensor(out, "out").scalar_type();
}

int64_t integer(PyObject *o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised();
    return v;
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised();
    return v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised();
    return v != 0;
}

PyObject *wrap(at::Tensor t) { return t.defined() ? THPVariable_Wrap(std::move(t)) : (Py_INCREF(Py_None), Py_None); }

PyObject *tuple(std::initializer_list<at::Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts)
        PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}

// (X, both, handle) -> codes and scales, along rows or along both axes
PyObject *quantize(PyObject *const *a) {
    const at::Tensor &X = tensor(a[0], "X");
    const int type = type_of(X.scalar_type(), "X");
    const int64_t ldx = rows_of(X, X.scalar_type(), "X");
    const bool both = truth(a[1]);
    const int64_t M = X.size(0), K = X.size(1);
    const at::Device dev = X.device();
    const NewHeld r(M, K, dev);
    const mpgemm_handle_t h = handle_of(a[2], dev);
    auto u8 = [](const at::Tensor &t) { return static_cast<uint8_t *>(t.data_ptr()); };
    // (tensors without elements have no stride to speak of; the call does nothing then)
    const int64_t lds = (blocks_of(K) + 15) / 16 * 16, ldst = (blocks_of(M) + 15) / 16 * 16;
    if (!both) {
        check(mpgemm_quantize_mxfp4(h, M, K, type, X.data_ptr(), ldx, u8(r.q), 16 * blocks_of(K), u8(r.s), lds, nullptr, 0,
                                    nullptr, 0, stream_of(dev)), "mpgemm_quantize_mxfp4");
        return tuple({r.q, r.s});
    }
    const NewHeld c(K, M, dev);
    check(mpgemm_quantize_mxfp4(h, M, K, type, X.data_ptr(), ldx, u8(r.q), 16 * blocks_of(K), u8(r.s), lds, u8(c.q),
                                16 * blocks_of(M), u8(c.s), ldst, stream_of(dev)), "mpgemm_quantize_mxfp4");
    return tuple({r.q, r.s, c.q, c.s});
}

// (q, s, K, dtype, out, handle) -> values
PyObject *dequantize(PyObject *const *a) {
    const at::ScalarType dt = dtype_of(a[3], a[4]);
    const int type = type_of(dt, "dtype");
    const at::Device dev = tensor(a[0], "q").device();
    const int64_t K = integer(a[2]);
    const Held m = held(a[0], a[1], K, "q", dev);
    int64_t ldy;
    at::Tensor Y = result(a[4], m.rows, K, dt, dev, ldy);
    check(mpgemm_dequantize_mxfp4(handle_of(a[5], dev), m.rows, K, m.q, m.ldq, m.s, m.lds, type, Y.data_ptr(), ldy,
                                  stream_of(dev)), "mpgemm_dequantize_mxfp4");
    return wrap(Y);
}

// (Aq, As, Bq, Bs, K, bias, dtype, out, handle) -> C
PyObject *gemm(PyObject *const *a) {
    const at::ScalarType dt = dtype_of(a[6], a[7]);
    const int type = type_of(dt, "dtype");
    const at::Device dev = tensor(a[0], "A").device();
    const int64_t K = integer(a[4]);
    const Held A = held(a[0], a[1], K, "A", dev), B = held(a[2], a[3], K, "B", dev);
    const void *bias = bias_of(a[5], B.rows, dt, dev);
    int64_t ldc;
    at::Tensor C = result(a[7], A.rows, B.rows, dt, dev, ldc);
    const int64_t n = mpgemm_run_mxfp4_workspace(A.rows, B.rows, K, cu_count(dev));
    const at::Tensor ws = scratch(n, dev, "mpgemm_run_mxfp4");
    check(mpgemm_run_mxfp4(handle_of(a[8], dev), A.rows, B.rows, K, A.q, A.ldq, A.s, A.lds, B.q, B.ldq, B.s, B.lds, bias,
                           type, C.data_ptr(), ldc, pointer(ws), n, stream_of(dev)), "mpgemm_run_mxfp4");
    return wrap(C);
}

// (X, Wq, Ws, bias, out, handle) -> Y
PyObject *dyn(PyObject *const *a) {
    const at::Tensor &X = tensor(a[0], "X");
    no_gradient(X, "X");
    const at::ScalarType dt = X.scalar_type();
    const int type = type_of(dt, "X");
    const int64_t ldx = rows_of(X, dt, "X");
    const at::Device dev = X.device();
    const int64_t M = X.size(0), K = X.size(1);
    const Held W = held(a[1], a[2], K, "W", dev);
    const void *bias = bias_of(a[3], W.rows, dt, dev);
    int64_t ldy;
    at::Tensor Y = result(a[4], M, W.rows, dt, dev, ldy);
    const int64_t n = mpgemm_run_mxfp4_dyn_workspace(M, W.rows, K, cu_count(dev));
    const at::Tensor ws = scratch(n, dev, "mpgemm_run_mxfp4_dyn");
    check(mpgemm_run_mxfp4_dyn(handle_of(a[5], dev), M, W.rows, K, type, X.data_ptr(), ldx, W.q, W.ldq, W.s, W.lds, bias,
                               Y.data_ptr(), ldy, pointer(ws), n, stream_of(dev)), "mpgemm_run_mxfp4_dyn");
    return wrap(Y);
}

// (dY, WTq, WTs, XTq, XTs, need_dx, need_dw, handle) -> (dX, dW)
PyObject *backward(PyObject *const *a) {
    const at::Tensor &dY = tensor(a[0], "dY");
    no_gradient(dY, "dY");
    const at::ScalarType dt = dY.scalar_type();
    const int type = type_of(dt, "dY");
    const int64_t lddy = rows_of(dY, dt, "dY");
    const at::Device dev = dY.device();
    const int64_t M = dY.size(0), N = dY.size(1);
    const bool need_dx = truth(a[5]), need_dw = truth(a[6]);
    if (!need_dx && !need_dw)
        return tuple({at::Tensor(), at::Tensor()});
    Held WT, XT;
    if (need_dx)
        WT = held(a[1], a[2], N, "W^T", dev);
    if (need_dw)
        XT = held(a[3], a[4], M, "X^T", dev);
    const int64_t K = need_dx ? WT.rows : XT.rows, ld = std::max<int64_t>(K, 1);
    if (need_dx && need_dw && XT.rows != K)
        fail(PyExc_ValueError, "W^T and X^T disagree on K");
    const at::Tensor dX = need_dx ? empty({M, K}, dt, dev) : at::Tensor();
    const at::Tensor dW = need_dw ? empty({N, K}, at::kFloat, dev) : at::Tensor();
    const int64_t n = mpgemm_run_mxfp4_backward_workspace(M, N, K, cu_count(dev));
    const at::Tensor ws = scratch(n, dev, "mpgemm_run_mxfp4_backward");
    check(mpgemm_run_mxfp4_backward(handle_of(a[7], dev), M, N, K, type, dY.data_ptr(), lddy, WT.q, WT.ldq, WT.s, WT.lds,
                                    XT.q, XT.ldq, XT.s, XT.lds, pointer(dX), ld, static_cast<float *>(pointer(dW)), ld,
                                    pointer(ws), n, stream_of(dev)), "mpgemm_run_mxfp4_backward");
    return tuple({dX, dW});
}

// Row and matrix strides of one matrix or a batch.
void strides_of(const at::Tensor &t, at::ScalarType type, const char *name, int64_t &ld, int64_t &stride) {
    const int64_t d = t.dim(), rows = t.size(d - 2), cols = t.size(d - 1);
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, std::string(name) + ": expected " + c10::toString(type) + ", got " +
                                  c10::toString(t.scalar_type()));
    if (!t.is_cuda())
        fail(PyExc_ValueError, std::string(name) + ": expected a device tensor");
    if (cols > 1 && t.stride(d - 1) != 1)
        fail(PyExc_ValueError, std::string(name) + ": rows must be contiguous (their last stride 1)");
    ld = rows > 1 ? t.stride(d - 2) : std::max<int64_t>(cols, 1);
    stride = d == 3 && t.size(0) > 1 ? t.stride(0) : 0;
}

// (G, steps, coeffs, eps, out, handle) -> Y
PyObject *newton_schulz(PyObject *const *a) {
    const at::Tensor &G = tensor(a[0], "G");
    no_gradient(G, "G");
    if (a[4] != Py_None)
        no_gradient(tensor(a[4], "out"), "out");
    const at::ScalarType dt = G.scalar_type();
    const int type = type_of(dt, "G", false);
    if (G.dim() != 2 && G.dim() != 3)
        fail(PyExc_ValueError, "G: expected a matrix or a batch of matrices");
    const int64_t steps = integer(a[1]);
    PyObject *seq = PySequence_Fast(a[2], "coeffs: expected three numbers");
    if (!seq)
        throw Raised();
    float k[3];
    const bool three = PySequence_Fast_GET_SIZE(seq) == 3;
    bool numbers = three;
    for (int i = 0; i < 3 && numbers; ++i) {
        k[i] = (float)PyFloat_AsDouble(PySequence_Fast_GET_ITEM(seq, i));
        numbers = !PyErr_Occurred();
    }
    Py_DECREF(seq);
    if (!three)
        fail(PyExc_ValueError, "coeffs: expected three numbers");
    if (!numbers)
        throw Raised();
    const float eps = (float)number(a[3]);
    const at::Device dev = G.device();
    const int64_t B = G.dim() == 2 ? 1 : G.size(0), M = G.size(-2), N = G.size(-1);
    int64_t ldg, sg, ldy, sy;
    strides_of(G, dt, "G", ldg, sg);
    if (steps < 0 || steps > 1 << 20)
        check(MPGEMM_ERR_INVALID_ARG, "mpgemm_run_newton_schulz");
    at::Tensor Y = a[4] == Py_None ? empty(G.sizes(), dt, dev) : tensor(a[4], "out");
    if (Y.sizes() != G.sizes() || Y.device() != dev)
        fail(PyExc_ValueError, "out: expected a tensor of G's shape on " + dev.str());
    strides_of(Y, dt, "out", ldy, sy);
    const int64_t n = mpgemm_run_newton_schulz_workspace(B, M, N);
    const at::Tensor ws = scratch(n, dev, "mpgemm_run_newton_schulz");
    check(mpgemm_run_newton_schulz(handle_of(a[5], dev), B, M, N, type, G.data_ptr(), ldg, sg, (int)steps, k, eps,
                                   Y.data_ptr(), ldy, sy, pointer(ws), n, stream_of(dev)), "mpgemm_run_newton_schulz");
    return wrap(Y);
}

// ---- 8-bit integers: codes (R x K int8, any row stride) and R fp32 scales

struct I8Held {
    const int8_t *q = nullptr;
    const float *s = nullptr;
    int64_t ld = 0, rows = 0, k = 0;
};

I8Held i8_held(PyObject *oq, PyObject *os, const char *name, const at::Device &dev) {
    const at::Tensor &q = tensor(oq, name), &s = tensor(os, name);
    no_gradient(s, name);
    I8Held h;
    h.ld = rows_of(q, at::kChar, name);
    h.rows = q.size(0);
    h.k = q.size(1);
    if (s.scalar_type() != at::kFloat || s.dim() != 1 || s.size(0) != h.rows || !s.is_contiguous())
        fail(PyExc_ValueError, std::string(name) + ": expected " + std::to_string(h.rows) + " contiguous float32 scales");
    if (q.device() != dev || s.device() != dev)
        fail(PyExc_ValueError, std::string(name) + ": not on " + dev.str());
    h.q = static_cast<const int8_t *>(q.data_ptr());
    h.s = static_cast<const float *>(s.data_ptr());
    return h;
}

void same_k(int64_t k, int64_t other, const char *what) {
    if (k != other)
        fail(PyExc_ValueError, std::string(what) + " disagree on K (" + std::to_string(k) + " and " + std::to_string(other) + ")");
}

// Whether rows start at multiples of 16 bytes, not too far apart for one offset.
bool rows_aligned(const void *p, int64_t ld, int64_t rows, int size) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (rows <= 1 || (ld * size % 16 == 0 && ld * size < (1 << 23)));
}

int act_of(PyObject *o) {
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    if (s && !strcmp(s, "silu"))
        return MPGEMM_ACT_SILU;
    if (s && !strcmp(s, "gelu"))
        return MPGEMM_ACT_GELU;
    if (s && !strcmp(s, "gelu_tanh"))
        return MPGEMM_ACT_GELU_TANH;
    fail(PyExc_ValueError, "act: expected 'silu', 'gelu' or 'gelu_tanh'");
}

// A 16-bit matrix of the block's type on its device, for the product named.
const at::Tensor &block(PyObject *o, const char *name, at::ScalarType type, const at::Device &dev, int64_t &ld) {
    const at::Tensor &t = tensor(o, name);
    no_gradient(t, name);
    ld = rows_of(t, type, name);
    if (t.device() != dev)
        fail(PyExc_ValueError, std::string(name) + ": not on " + dev.str());
    return t;
}

void shape_is(const at::Tensor &t, int64_t rows, int64_t cols, const char *name) {
    if (t.size(0) != rows || t.size(1) != cols)
        fail(PyExc_ValueError, std::string(name) + ": expected " + std::to_string(rows) + " x " + std::to_string(cols) + ", got " +
                                   std::to_string(t.size(0)) + " x " + std::to_string(t.size(1)));
}

// (X, handle) -> codes (rows padded to 16 bytes), scales
PyObject *quantize_i8(PyObject *const *a) {
    const at::Tensor &X = tensor(a[0], "X");
    no_gradient(X, "X");
    const int type = type_of(X.scalar_type(), "X");
    const int64_t ldx = rows_of(X, X.scalar_type(), "X"), M = X.size(0), K = X.size(1), ld = std::max<int64_t>((K + 15) / 16 * 16, 16);
    const at::Device dev = X.device();
    // (an allocation each: tensors of two types over one storage cannot be saved)
    at::Tensor q = empty({M, ld}, at::kChar, dev), s = empty({M}, at::kFloat, dev);
    q.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef{M, K}, at::IntArrayRef{ld, 1});
    if (K == 0)
        s.zero_();
    check(mpgemm_quantize_i8(handle_of(a[1], dev), M, K, type, X.data_ptr(), ldx, static_cast<int8_t *>(q.data_ptr()), ld,
                             static_cast<float *>(s.data_ptr()), stream_of(dev)), "mpgemm_quantize_i8");
    return tuple({q, s});
}

// (q, s, dtype, out, handle) -> values
PyObject *dequantize_i8(PyObject *const *a) {
    const at::ScalarType dt = dtype_of(a[2], a[3]);
    const int type = type_of(dt, "dtype");
    const at::Device dev = tensor(a[0], "q").device();
    const I8Held m = i8_held(a[0], a[1], "q", dev);
    int64_t ldy;
    at::Tensor Y = result(a[3], m.rows, m.k, dt, dev, ldy);
    check(mpgemm_dequantize_i8(handle_of(a[4], dev), m.rows, m.k, m.q, m.ld, m.s, type, Y.data_ptr(), ldy, stream_of(dev)),
          "mpgemm_dequantize_i8");
    return wrap(Y);
}

// (Aq, As, Bq, Bs, bias, dtype, out, handle) -> C
PyObject *gemm_w8a8(PyObject *const *a) {
    const at::ScalarType dt = dtype_of(a[5], a[6]);
    const int type = type_of(dt, "dtype");
    const at::Device dev = tensor(a[0], "A").device();
    const I8Held A = i8_held(a[0], a[1], "A", dev), B = i8_held(a[2], a[3], "B", dev);
    same_k(A.k, B.k, "A and B");
    const void *bias = bias_of(a[4], B.rows, dt, dev);
    int64_t ldc;
    at::Tensor C = result(a[6], A.rows, B.rows, dt, dev, ldc);
    const bool al = rows_aligned(A.q, A.ld, A.rows, 1) && rows_aligned(B.q, B.ld, B.rows, 1);
    const int64_t n = mpgemm_run_w8a8_workspace(A.rows, B.rows, A.k, al, cu_count(dev));
    const at::Tensor ws = scratch(n, dev, "mpgemm_run_w8a8");
    check(mpgemm_run_w8a8(handle_of(a[7], dev), A.rows, B.rows, A.k, A.q, A.ld, A.s, B.q, B.ld, B.s, bias, type, C.data_ptr(), ldc,
                          pointer(ws), n, stream_of(dev)), "mpgemm_run_w8a8");
    return wrap(C);
}

// (X, Wq, Ws, bias, out, handle) -> Y
PyObject *w8a8_dyn(PyObject *const *a) {
    const at::Tensor &X = tensor(a[0], "X");
    no_gradient(X, "X");
    const at::ScalarType dt = X.scalar_type();
    const int type = type_of(dt, "X");
    const int64_t ldx = rows_of(X, dt, "X"), M = X.size(0), K = X.size(1);
    const at::Device dev = X.device();
    const I8Held W = i8_held(a[1], a[2], "W", dev);
    same_k(K, W.k, "X and W");
    const void *bias = bias_of(a[3], W.rows, dt, dev);
    int64_t ldy;
    at::Tensor Y = result(a[4], M, W.rows, dt, dev, ldy);
    const int64_t n = mpgemm_run_w8a8_dyn_workspace(M, W.rows, K, rows_aligned(W.q, W.ld, W.rows, 1), cu_count(dev));
    const at::Tensor ws = scratch(n, dev, "mpgemm_run_w8a8_dyn");
    check(mpgemm_run_w8a8_dyn(handle_of(a[5], dev), M, W.rows, K, type, X.data_ptr(), ldx, W.q, W.ld, W.s, bias, Y.data_ptr(), ldy,
                              pointer(ws), n, stream_of(dev)), "mpgemm_run_w8a8_dyn");
    return wrap(Y);
}

// (X, Wg, Wu, act, keep, out, handle) -> H or (H, G, U)
PyObject *gated(PyObject *const *a) {
    const at::Tensor &X = tensor(a[0], "X");
    no_gradient(X, "X");
    const at::ScalarType dt = X.scalar_type();
    const int type = type_of(dt, "X", false), act = act_of(a[3]);
    const int64_t ldx = rows_of(X, dt, "X"), M = X.size(0), K = X.size(1);
    const at::Device dev = X.device();
    int64_t ldg, ldu, ldh;
    const at::Tensor &Wg = block(a[1], "Wg", dt, dev, ldg), &Wu = block(a[2], "Wu", dt, dev, ldu);
    const int64_t N = Wg.size(0);
    shape_is(Wg, N, K, "Wg");
    shape_is(Wu, N, K, "Wu");
    const bool keep = truth(a[4]);
    at::Tensor H = result(a[5], M, N, dt, dev, ldh);
    const at::Tensor G = keep ? empty({M, N}, dt, dev) : at::Tensor(), U = keep ? empty({M, N}, dt, dev) : at::Tensor();
    const bool al = rows_aligned(X.data_ptr(), ldx, M, 2) && rows_aligned(Wg.data_ptr(), ldg, N, 2) && rows_aligned(Wu.data_ptr(), ldu, N, 2);
    const int64_t n = mpgemm_run_gated_workspace(M, N, K, al, cu_count(dev)), ld = std::max<int64_t>(N, 1);
    const at::Tensor ws = scratch(n, dev, "mpgemm_run_gated");
    check(mpgemm_run_gated(handle_of(a[6], dev), M, N, K, type, act, X.data_ptr(), ldx, Wg.data_ptr(), ldg, Wu.data_ptr(), ldu,
                           H.data_ptr(), ldh, pointer(G), ld, pointer(U), ld, pointer(ws), n, stream_of(dev)), "mpgemm_run_gated");
    if (!keep)
        return wrap(H);
    return tuple({H, G, U});
}

// (dH, X, Wg, Wu, G, U, act, need_dx, need_dw, handle) -> (dX, dWg, dWu)
PyObject *gated_backward(PyObject *const *a) {
    const at::Tensor &dH = tensor(a[0], "dH");
    no_gradient(dH, "dH");
    const at::ScalarType dt = dH.scalar_type();
    const int type = type_of(dt, "dH", false), act = act_of(a[6]);
    const int64_t lddh = rows_of(dH, dt, "dH"), M = dH.size(0), N = dH.size(1);
    const at::Device dev = dH.device();
    const bool need_dx = truth(a[7]), need_dw = truth(a[8]);
    if (!need_dx && !need_dw)
        return tuple({at::Tensor(), at::Tensor(), at::Tensor()});
    int64_t ldx = 0, ldwg = 0, ldwu = 0, ldg, ldu, K = 0;
    at::Tensor X, Wg, Wu;
    if (need_dw) {
        X = block(a[1], "X", dt, dev, ldx);
        K = X.size(1);
        shape_is(X, M, K, "X");
    }
    if (need_dx) {
        Wg = block(a[2], "Wg", dt, dev, ldwg);
        Wu = block(a[3], "Wu", dt, dev, ldwu);
        if (!need_dw)
            K = Wg.size(1);
        shape_is(Wg, N, K, "Wg");
        shape_is(Wu, N, K, "Wu");
    }
    const at::Tensor &G = block(a[4], "G", dt, dev, ldg), &U = block(a[5], "U", dt, dev, ldu);
    shape_is(G, M, N, "G");
    shape_is(U, M, N, "U");
    const at::Tensor dX = need_dx ? empty({M, K}, dt, dev) : at::Tensor();
    const at::Tensor dWg = need_dw ? empty({N, K}, dt, dev) : at::Tensor(), dWu = need_dw ? empty({N, K}, dt, dev) : at::Tensor();
    const bool al = (!need_dw || rows_aligned(X.data_ptr(), ldx, M, 2)) &&
                    (!need_dx || (rows_aligned(Wg.data_ptr(), ldwg, N, 2) && rows_aligned(Wu.data_ptr(), ldwu, N, 2) && (ldwg == ldwu || N <= 1)));
    const int64_t n = mpgemm_run_gated_backward_workspace(M, N, K, al, cu_count(dev)), ld = std::max<int64_t>(K, 1);
    const at::Tensor ws = scratch(n, dev, "mpgemm_run_gated_backward");
    check(mpgemm_run_gated_backward(handle_of(a[9], dev), M, N, K, type, act, dH.data_ptr(), lddh, pointer(X), ldx, pointer(Wg), ldwg,
                                    pointer(Wu), ldwu, G.data_ptr(), ldg, U.data_ptr(), ldu, pointer(dX), ld, pointer(dWg), ld,
                                    pointer(dWu), ld, pointer(ws), n, stream_of(dev)), "mpgemm_run_gated_backward");
    return tuple({dX, dWg, dWu});
}

// (Aq, As, Wgq, Wgs, Wuq, Wus, act, dtype, out, handle) -> H
PyObject *gated_w8a8(PyObject *const *a) {
    const at::ScalarType dt = dtype_of(a[7], a[8]);
    const int type = type_of(dt, "dtype"), act = act_of(a[6]);
    const at::Device dev = tensor(a[0], "A").device();
    const I8Held A = i8_held(a[0], a[1], "A", dev), G = i8_held(a[2], a[3], "Wg", dev), U = i8_held(a[4], a[5], "Wu", dev);
    same_k(A.k, G.k, "A and Wg");
    same_k(A.k, U.k, "A and Wu");
    if (G.rows != U.rows)
        fail(PyExc_ValueError, "Wg and Wu disagree on N");
    int64_t ldh;
    at::Tensor H = result(a[8], A.rows, G.rows, dt, dev, ldh);
    const bool al = rows_aligned(A.q, A.ld, A.rows, 1) && rows_aligned(G.q, G.ld, G.rows, 1) && rows_aligned(U.q, U.ld, U.rows, 1);
    const int64_t n = mpgemm_run_gated_w8a8_workspace(A.rows, G.rows, A.k, al, cu_count(dev));
    const at::Tensor ws = scratch(n, dev, "mpgemm_run_gated_w8a8");
    check(mpgemm_run_gated_w8a8(handle_of(a[9], dev), A.rows, G.rows, A.k, act, A.q, A.ld, A.s, G.q, G.ld, G.s, U.q, U.ld, U.s, type,
                                H.data_ptr(), ldh, pointer(ws), n, stream_of(dev)), "mpgemm_run_gated_w8a8");
    return wrap(H);
}

// (X, Wgq, Wgs, Wuq, Wus, act, out, handle) -> H
PyObject *gated_w8a8_dyn(PyObject *const *a) {
    const at::Tensor &X = tensor(a[0], "X");
    no_gradient(X, "X");
    const at::ScalarType dt = X.scalar_type();
    const int type = type_of(dt, "X"), act = act_of(a[5]);
    const int64_t ldx = rows_of(X, dt, "X"), M = X.size(0), K = X.size(1);
    const at::Device dev = X.device();
    const I8Held G = i8_held(a[1], a[2], "Wg", dev), U = i8_held(a[3], a[4], "Wu", dev);
    same_k(K, G.k, "X and Wg");
    same_k(K, U.k, "X and Wu");
    if (G.rows != U.rows)
        fail(PyExc_ValueError, "Wg and Wu disagree on N");
    int64_t ldh;
    at::Tensor H = result(a[6], M, G.rows, dt, dev, ldh);
    const bool al = rows_aligned(G.q, G.ld, G.rows, 1) && rows_aligned(U.q, U.ld, U.rows, 1);
    const int64_t n = mpgemm_run_gated_w8a8_dyn_workspace(M, G.rows, K, al, cu_count(dev));
    const at::Tensor ws = scratch(n, dev, "mpgemm_run_gated_w8a8_dyn");
    check(mpgemm_run_gated_w8a8_dyn(handle_of(a[7], dev), M, G.rows, K, type, act, X.data_ptr(), ldx, G.q, G.ld, G.s, U.q, U.ld, U.s,
                                    H.data_ptr(), ldh, pointer(ws), n, stream_of(dev)), "mpgemm_run_gated_w8a8_dyn");
    return wrap(H);
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        // (outputs and scratch take no part in autograd)
        at::AutoDispatchBelowADInplaceOrView guard;
        return F(args);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define MPG_CALL(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<name, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {MPG_CALL(quantize, 3), MPG_CALL(dequantize, 6), MPG_CALL(gemm, 9),      MPG_CALL(dyn, 6),
                         MPG_CALL(backward, 8), MPG_CALL(newton_schulz, 6),
                         MPG_CALL(quantize_i8, 2), MPG_CALL(dequantize_i8, 5), MPG_CALL(gemm_w8a8, 8), MPG_CALL(w8a8_dyn, 6),
                         MPG_CALL(gated, 7), MPG_CALL(gated_backward, 10), MPG_CALL(gated_w8a8, 10), MPG_CALL(gated_w8a8_dyn, 8),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
