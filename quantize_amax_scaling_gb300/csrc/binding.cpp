// binding.cpp -- the 4-bit and residual-norm calls of the Python binding: torch
// tensors checked and marshalled into the C ABI of libfp8q (fp8q.h).
//
// A call of one token spends more time in Python's checks of a dozen tensors than
// on the GPU; here a tensor takes tens of nanoseconds.  fp8q.py passes every
// argument by position, in the order of its own signatures, and turns the status
// that comes back into an exception; what a tensor may not be is raised here, as
// ValueError.  The entry points' addresses come from bind(), so this module links
// no copy of the library.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp8q.h"

#include <cstdint>

namespace {

decltype(&fp8q_fp4_quantize_amax) g_quantize;
decltype(&fp8q_fp4_dequantize) g_dequantize;
decltype(&fp8q_fp4_matmul) g_matmul;
decltype(&fp8q_residual_norm_quantize_amax) g_norm;
decltype(&fp8q_residual_norm_backward) g_norm_backward;
decltype(&fp8q_residual_norm_backward_workspace) g_workspace;

struct Refused {};  // a Python exception has been set

enum Kind { kBf16, kByte, kF32, kGate };  // kByte: uint8 or a float8 type; kGate: binary32 or bf16

int64_t row_bytes(int64_t cols) { return (cols + 31) / 32 * 16; }
int64_t scale_bytes(int64_t rows, int64_t cols, int64_t fmt) {
    return (rows + 127) / 128 * (fmt == FP8Q_MXFP4 ? (cols + 127) / 128 : (cols + 63) / 64) * 512;
}

void matrix(const at::Tensor* t, const char* name, const char* shape) {
    if (t && t->dim() == 2) return;
    PyErr_Format(PyExc_ValueError, "%s must be %s", name, shape);
    throw Refused();
}

// One call's arguments, taken in turn.
class Args {
public:
    Args(const char* call, PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
        if (n == want) return;
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", call, want, n);
        throw Refused();
    }

    // The next tensor, or nullptr for None; with `shape`, one of two dimensions.
    const at::Tensor* tensor(Kind kind, const char* name, const char* shape = nullptr) {
        PyObject* o = a_[i_++];
        if (o == Py_None && !shape) return nullptr;
        if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
        const at::Tensor& t = THPVariable_Unpack(o);
        if (shape) matrix(&t, name, shape);
        if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
        const at::ScalarType s = t.scalar_type();
        const bool ok = kind == kBf16   ? s == at::kBFloat16
                        : kind == kF32  ? s == at::kFloat
                        : kind == kGate ? s == at::kFloat || s == at::kBFloat16
                                        : s == at::kByte || s == at::kFloat8_e4m3fn || s == at::kFloat8_e5m2;
        if (!ok) {
            PyErr_Format(PyExc_ValueError, "%s has dtype %s, expected %s", name, c10::toString(s),
                         kind == kBf16   ? "bfloat16"
                         : kind == kF32  ? "float32"
                         : kind == kGate ? "float32 or bfloat16"
                                         : "uint8 or a float8 type");
            throw Refused();
        }
        if (!t.is_contiguous()) refuse("%s must be contiguous", name);
        if (device_ < 0) device_ = c10::cuda::current_device();
        if (t.device().index() != device_) {
            PyErr_Format(PyExc_ValueError,
                         "%s is on cuda:%d but the current CUDA device is cuda:%d; the kernels launch on the current "
                         "device (wrap the call in torch.cuda.device)",
                         name, (int)t.device().index(), (int)device_);
            throw Refused();
        }
        return &t;
    }

    int64_t integer() {
        const long long v = PyLong_AsLongLong(a_[i_++]);
        if (v == -1 && PyErr_Occurred()) throw Refused();
        return v;
    }

    float real() {
        const double v = PyFloat_AsDouble(a_[i_++]);
        if (v == -1.0 && PyErr_Occurred()) throw Refused();
        return (float)v;
    }

    // The last argument: a stream's handle, an object with one, or None for the current stream.
    void* stream() {
        PyObject* o = a_[i_++];
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device_ < 0 ? c10::cuda::current_device() : device_).stream();
        if (!PyLong_Check(o)) {
            PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
            if (!h) throw Refused();
            void* s = PyLong_AsVoidPtr(h);
            Py_DECREF(h);
            if (PyErr_Occurred()) throw Refused();
            return s;
        }
        void* s = PyLong_AsVoidPtr(o);
        if (PyErr_Occurred()) throw Refused();
        return s;
    }

    [[noreturn]] static void refuse(const char* what, const char* name) {
        PyErr_Format(PyExc_ValueError, what, name);
        throw Refused();
    }

private:
    PyObject* const* a_;
    Py_ssize_t i_ = 0;
    c10::DeviceIndex device_ = -1;  // the current one, once a tensor has asked
};

void* ptr(const at::Tensor* t) { return t ? t->mutable_data_ptr() : nullptr; }
float* floats(const at::Tensor* t) { return static_cast<float*>(ptr(t)); }
uint8_t* bytes(const at::Tensor* t) { return static_cast<uint8_t*>(ptr(t)); }

void size(const at::Tensor* t, int64_t n, const char* name, const char* what) {
    if (!t || t->numel() == n) return;
    PyErr_Format(PyExc_ValueError, "%s must have %s=%lld elements", name, what, (long long)n);
    throw Refused();
}

void one(const at::Tensor* t, const char* name) {
    if (t && t->numel() != 1) Args::refuse("%s must have one element", name);
}

void packed(const at::Tensor* q, const at::Tensor* sf, int64_t rows, int64_t cols, int64_t fmt, const char* name) {
    if (q && sf && q->numel() == rows * row_bytes(cols) && sf->numel() == scale_bytes(rows, cols, fmt)) return;
    PyErr_Format(PyExc_ValueError, "%s is not a packed operand of [%lld, %lld]: see fp4_empty", name, (long long)rows, (long long)cols);
    throw Refused();
}

void gate_rows(const at::Tensor* gate, int64_t rows, int64_t hidden, int64_t per) {
    if (!gate) return;
    if (per < 1) Args::refuse("%s must be at least 1", "rows_per_gate");
    const int64_t groups = rows > 0 ? (rows - 1) / per + 1 : 0;
    if (gate->numel() == groups * hidden) return;
    PyErr_Format(PyExc_ValueError, "gate must be [%lld, %lld]", (long long)groups, (long long)hidden);
    throw Refused();
}

// The call of an entry point.  A launch waits where its stream's queue is full, and other Python threads go on meanwhile:
// every argument has been read by then, and the caller's references keep the tensors.
template <typename F, typename... A>
int64_t launch(F f, A... args) {
    PyThreadState* const state = PyEval_SaveThread();
    const int64_t status = f(args...);
    PyEval_RestoreThread(state);
    return status;
}

bool four_bits(int64_t fmt) { return fmt == FP8Q_MXFP4 || fmt == FP8Q_NVFP4; }

// (x, q, sf, fmt, scale, amax, qt, sft, stream)
int64_t quantize(PyObject* const* v, Py_ssize_t n) {
    Args a("fp4_quantize_amax", v, n, 9);
    const at::Tensor* x = a.tensor(kBf16, "x", "[rows, cols]");
    const at::Tensor *q = a.tensor(kByte, "q"), *sf = a.tensor(kByte, "sf");
    const int64_t fmt = a.integer(), rows = x->size(0), cols = x->size(1);
    const at::Tensor *scale = a.tensor(kF32, "scale"), *amax = a.tensor(kF32, "amax"), *qt = a.tensor(kByte, "qt"),
                     *sft = a.tensor(kByte, "sft");
    if (q) packed(q, sf, rows, cols, fmt, "(q, sf)");
    if (qt) packed(qt, sft, cols, rows, fmt, "(qt, sft)");
    one(scale, "scale");
    one(amax, "amax");
    return launch(g_quantize, ptr(x), rows, cols, bytes(q), bytes(sf), bytes(qt), bytes(sft), (fp8q_format)fmt, floats(scale), floats(amax),
                  a.stream());
}

// (q, sf, y, fmt, scale, stream)
int64_t dequantize(PyObject* const* v, Py_ssize_t n) {
    Args a("fp4_dequantize", v, n, 6);
    const at::Tensor *q = a.tensor(kByte, "q"), *sf = a.tensor(kByte, "sf"), *y = a.tensor(kBf16, "y", "[rows, cols]");
    const int64_t fmt = a.integer(), rows = y->size(0), cols = y->size(1);
    const at::Tensor* scale = a.tensor(kF32, "scale");
    packed(q, sf, rows, cols, fmt, "(q, sf)");
    one(scale, "scale");
    return launch(g_dequantize, bytes(q), bytes(sf), ptr(y), rows, cols, (fp8q_format)fmt, floats(scale), a.stream());
}

// (a, a_sf, b, b_sf, d, k, fmt, a_scale, b_scale, stream)
int64_t matmul(PyObject* const* v, Py_ssize_t n) {
    Args a("fp4_matmul", v, n, 10);
    const at::Tensor *p = a.tensor(kByte, "a"), *psf = a.tensor(kByte, "a_sf"), *q = a.tensor(kByte, "b"), *qsf = a.tensor(kByte, "b_sf"),
                     *d = a.tensor(kGate, "d", "[m, n]");
    const int64_t k = a.integer(), fmt = a.integer(), rows = d->size(0), cols = d->size(1);
    const at::Tensor *sa = a.tensor(kF32, "a_scale"), *sb = a.tensor(kF32, "b_scale");
    packed(p, psf, rows, k, fmt, "(a, a_sf)");
    packed(q, qsf, cols, k, fmt, "(b, b_sf)");
    one(sa, "a_scale");
    one(sb, "b_scale");
    return launch(g_matmul, bytes(p), bytes(psf), bytes(q), bytes(qsf), ptr(d), rows, cols, k, (fp8q_format)fmt,
                  d->scalar_type() == at::kFloat ? FP8Q_OUT_F32 : FP8Q_OUT_BF16, floats(sa), floats(sb), a.stream());
}

// (residual, residual_out, block, post_weight, gate, rows_per_gate, alpha, pre_weight, h, q, sf, fmt, scale, amax, rstd_post,
//  rstd_pre, eps, stream)
int64_t norm(PyObject* const* v, Py_ssize_t n) {
    Args a("residual_norm_quantize_amax", v, n, 18);
    const at::Tensor* residual = a.tensor(kBf16, "residual", "[rows, hidden]");
    const at::Tensor *out = a.tensor(kBf16, "residual_out"), *block = a.tensor(kBf16, "block"), *post = a.tensor(kF32, "post_weight"),
                     *gate = a.tensor(kGate, "gate");
    const int64_t per = a.integer();
    const float alpha = a.real();
    const at::Tensor *pre = a.tensor(kF32, "pre_weight"), *h = a.tensor(kBf16, "h"), *q = a.tensor(kByte, "q"), *sf = a.tensor(kByte, "sf");
    const int64_t fmt = a.integer(), rows = residual->size(0), hidden = residual->size(1);
    const at::Tensor *scale = a.tensor(kF32, "scale"), *amax = a.tensor(kF32, "amax"), *rpost = a.tensor(kF32, "rstd_post"),
                     *rpre = a.tensor(kF32, "rstd_pre");
    size(out, rows * hidden, "residual_out", "rows * hidden");
    size(block, rows * hidden, "block", "rows * hidden");
    size(h, rows * hidden, "h", "rows * hidden");
    size(post, hidden, "post_weight", "hidden");
    size(pre, hidden, "pre_weight", "hidden");
    size(rpost, rows, "rstd_post", "rows");
    size(rpre, rows, "rstd_pre", "rows");
    gate_rows(gate, rows, hidden, per);
    if (q && four_bits(fmt))
        packed(q, sf, rows, hidden, fmt, "(q, sf)");
    else
        size(q, rows * hidden, "q", "rows * hidden");
    one(scale, "scale");
    one(amax, "amax");
    fp8q_residual_norm g = {};
    g.rows = rows;
    g.hidden = (int32_t)(hidden > INT32_MAX ? INT32_MAX : hidden);
    g.fmt = (fp8q_format)fmt;
    g.residual = ptr(residual);
    g.block = ptr(block);
    g.post_weight = floats(post);
    g.gate = ptr(gate);
    g.rows_per_gate = per;
    g.gate_is_bf16 = gate && gate->scalar_type() == at::kBFloat16;
    g.alpha = alpha;
    g.eps = a.real();
    g.pre_weight = floats(pre);
    g.residual_out = ptr(out);
    g.h = ptr(h);
    g.q = bytes(q);
    g.sf = bytes(sf);
    g.scale = floats(scale);
    g.amax = floats(amax);
    g.rstd_post = floats(rpost);
    g.rstd_pre = floats(rpre);
    return launch(g_norm, &g, a.stream());
}

// (d_residual_out, d_h, residual_out, rstd_pre, pre_weight, d_residual, d_pre_weight, block, rstd_post, post_weight, gate,
//  rows_per_gate, alpha, d_block, d_post_weight, d_gate, workspace, stream)
int64_t norm_backward(PyObject* const* v, Py_ssize_t n) {
    Args a("residual_norm_backward", v, n, 18);
    const at::Tensor *dro = a.tensor(kBf16, "d_residual_out"), *dh = a.tensor(kBf16, "d_h"), *d = dro ? dro : dh;
    matrix(d, "d_residual_out or d_h", "[rows, hidden]");
    const int64_t rows = d->size(0), hidden = d->size(1);
    const at::Tensor *ro = a.tensor(kBf16, "residual_out"), *rpre = a.tensor(kF32, "rstd_pre"), *pre = a.tensor(kF32, "pre_weight"),
                     *dr = a.tensor(kBf16, "d_residual"), *dpre = a.tensor(kF32, "d_pre_weight"), *block = a.tensor(kBf16, "block"),
                     *rpost = a.tensor(kF32, "rstd_post"), *post = a.tensor(kF32, "post_weight"), *gate = a.tensor(kGate, "gate");
    const int64_t per = a.integer();
    const float alpha = a.real();
    const at::Tensor *db = a.tensor(kBf16, "d_block"), *dpost = a.tensor(kF32, "d_post_weight"), *dgate = a.tensor(kGate, "d_gate"),
                     *space = a.tensor(kByte, "workspace");
    const struct {
        const at::Tensor* t;
        const char* name;
    } whole[] = {{dro, "d_residual_out"}, {dh, "d_h"}, {ro, "residual_out"}, {block, "block"}, {dr, "d_residual"}, {db, "d_block"}},
      columns[] = {{pre, "pre_weight"}, {post, "post_weight"}, {dpre, "d_pre_weight"}, {dpost, "d_post_weight"}};
    for (const auto& w : whole) size(w.t, rows * hidden, w.name, "rows * hidden");
    for (const auto& w : columns) size(w.t, hidden, w.name, "hidden");
    size(rpre, rows, "rstd_pre", "rows");
    size(rpost, rows, "rstd_post", "rows");
    gate_rows(gate, rows, hidden, per);
    if (gate && dgate && (dgate->numel() != gate->numel() || dgate->scalar_type() != gate->scalar_type()))
        Args::refuse("%s must have gate's shape and type", "d_gate");
    fp8q_residual_norm_grad g = {};
    g.rows = rows;
    g.hidden = (int32_t)(hidden > INT32_MAX ? INT32_MAX : hidden);
    g.gate_is_bf16 = gate && gate->scalar_type() == at::kBFloat16;
    g.d_residual_out = ptr(dro);
    g.d_h = ptr(dh);
    g.residual_out = ptr(ro);
    g.rstd_pre = floats(rpre);
    g.pre_weight = floats(pre);
    g.block = ptr(block);
    g.rstd_post = floats(rpost);
    g.post_weight = floats(post);
    g.gate = ptr(gate);
    g.rows_per_gate = per;
    g.alpha = alpha;
    g.d_residual = ptr(dr);
    g.d_block = ptr(db);
    g.d_pre_weight = floats(dpre);
    g.d_post_weight = floats(dpost);
    g.d_gate = ptr(dgate);
    g.workspace = ptr(space);
    g.workspace_bytes = space ? space->numel() : 0;
    return launch(g_norm_backward, &g, a.stream());
}

template <int64_t (*F)(PyObject* const*, Py_ssize_t)>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        return PyLong_FromLongLong(F(a, n));
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {  // torch's own
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// (rows, hidden, rows_per_gate)
int64_t workspace(PyObject* const* v, Py_ssize_t n) {
    Args a("residual_norm_backward_workspace", v, n, 3);
    const int64_t rows = a.integer(), hidden = a.integer(), per = a.integer();
    return g_workspace(rows, (int32_t)(hidden > INT32_MAX ? INT32_MAX : hidden < 0 ? 0 : hidden), per);
}

// (rows, cols, fmt): room for a packed operand on the current CUDA device
PyObject* empty(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        int64_t v[3];
        for (int i = 0; i < 3; ++i) {
            v[i] = n == 3 ? PyLong_AsLongLong(a[i]) : -1;
            if (v[i] == -1 && PyErr_Occurred()) return nullptr;
        }
        // beyond what the calls take, the bytes of both arrays could pass 64 bits and come out as few
        constexpr int64_t kMax = 0x7FFFFC00;
        if (n != 3 || v[0] < 0 || v[1] < 0 || v[0] > kMax || v[1] > kMax || !four_bits(v[2])) {
            PyErr_SetString(PyExc_ValueError, "fp4_empty takes rows and cols from 0 to 2^31 - 1024 and MXFP4 or NVFP4");
            return nullptr;
        }
        const auto o = at::TensorOptions().dtype(at::kByte).device(at::kCUDA, c10::cuda::current_device());
        // one allocation for both, the scales behind the codes (a multiple of 16 bytes)
        const int64_t codes = v[0] * row_bytes(v[1]), scales = scale_bytes(v[0], v[1], v[2]);
        const at::Tensor all = at::empty({codes + scales}, o);
        const auto part = [&](at::IntArrayRef sizes, int64_t from) {
            at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
            t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
            t.unsafeGetTensorImpl()->set_storage_offset(from);
            return t;
        };
        PyObject* q = THPVariable_Wrap(part({v[0], row_bytes(v[1])}, 0));
        PyObject* sf = q ? THPVariable_Wrap(part({scales}, codes)) : nullptr;
        PyObject* both = sf ? PyTuple_Pack(2, q, sf) : nullptr;
        Py_XDECREF(q);
        Py_XDECREF(sf);
        return both;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// Addresses of the entry points, in the order of the calls below.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[6] = {};
    for (Py_ssize_t i = 0; i < 6; ++i) {
        if (i < n) p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind takes six addresses");
            return nullptr;
        }
    }
    g_quantize = reinterpret_cast<decltype(g_quantize)>(p[0]);
    g_dequantize = reinterpret_cast<decltype(g_dequantize)>(p[1]);
    g_matmul = reinterpret_cast<decltype(g_matmul)>(p[2]);
    g_norm = reinterpret_cast<decltype(g_norm)>(p[3]);
    g_norm_backward = reinterpret_cast<decltype(g_norm_backward)>(p[4]);
    g_workspace = reinterpret_cast<decltype(g_workspace)>(p[5]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f))
PyMethodDef g_methods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                           {"fp4_empty", FAST(empty), METH_FASTCALL, nullptr},
                           {"fp4_quantize_amax", FAST(call<quantize>), METH_FASTCALL, nullptr},
                           {"fp4_dequantize", FAST(call<dequantize>), METH_FASTCALL, nullptr},
                           {"fp4_matmul", FAST(call<matmul>), METH_FASTCALL, nullptr},
                           {"residual_norm_quantize_amax", FAST(call<norm>), METH_FASTCALL, nullptr},
                           {"residual_norm_backward", FAST(call<norm_backward>), METH_FASTCALL, nullptr},
                           {"residual_norm_backward_workspace", FAST(call<workspace>), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
