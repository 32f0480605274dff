// binding.cpp -- the calls of the Python binding from the 4-bit ones on: torch
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
decltype(&fp8q_matmul) g_product;
decltype(&fp8q_grouped_matmul) g_grouped;
decltype(&fp8q_grouped_weight_gradient) g_grouped_gradient;
decltype(&fp8q_checkpoint_quantize) g_checkpoint;
decltype(&fp8q_checkpoint_dequantize) g_checkpoint_back;
decltype(&fp8q_gelu_backward_quantize_amax) g_gelu_backward;
decltype(&fp8q_gelu_backward_workspace) g_gelu_workspace;

struct Refused {};  // a Python exception has been set

enum Kind { kBf16, kByte, kF32, kGate, kI32 };  // kByte: uint8 or a float8 type; kGate: binary32 or bf16

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
    // whole: contiguous; otherwise the caller looks at the strides.
    const at::Tensor* tensor(Kind kind, const char* name, const char* shape = nullptr, bool whole = true) {
        PyObject* o = a_[i_++];
        if (o == Py_None && !shape) return nullptr;
        if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
        const at::Tensor& t = THPVariable_Unpack(o);
        if (shape && whole) matrix(&t, name, shape);
        if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
        const at::ScalarType s = t.scalar_type();
        const bool ok = kind == kBf16   ? s == at::kBFloat16
                        : kind == kF32  ? s == at::kFloat
                        : kind == kGate ? s == at::kFloat || s == at::kBFloat16
                        : kind == kI32  ? s == at::kInt
                                        : s == at::kByte || s == at::kFloat8_e4m3fn || s == at::kFloat8_e5m2;
        if (!ok) {
            PyErr_Format(PyExc_ValueError, "%s has dtype %s, expected %s", name, c10::toString(s),
                         kind == kBf16   ? "bfloat16"
                         : kind == kF32  ? "float32"
                         : kind == kGate ? "float32 or bfloat16"
                         : kind == kI32  ? "int32"
                                         : "uint8 or a float8 type");
            throw Refused();
        }
        if (whole && !t.is_contiguous()) refuse("%s must be contiguous", name);
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

    // A matrix of FP8 codes, or with `groups` a stack of them: elements of a row side by side, rows a multiple of 16 bytes
    // apart (or one row), the matrices one behind the other.  Its row length in bytes as `ld`.
    const at::Tensor* codes(const char* name, bool groups, int64_t* ld) {
        const at::Tensor* t = tensor(kByte, name, groups ? "[groups, rows, cols]" : "[rows, cols]", false);
        const int64_t dims = groups ? 3 : 2;
        if (t->dim() != dims) {
            PyErr_Format(PyExc_ValueError, "%s must be %s", name, groups ? "[groups, rows, cols]" : "[rows, cols]");
            throw Refused();
        }
        const int64_t rows = t->size(dims - 2), cols = t->size(dims - 1);
        *ld = rows > 1 && cols > 0 ? t->stride(dims - 2) : (cols + 15) / 16 * 16;
        if (cols > 1 && t->stride(dims - 1) != 1) refuse("%s must have the elements of a row side by side", name);
        if (t->numel() > 0 && rows > 1 && (*ld < cols || *ld % 16)) refuse("%s must have rows a multiple of 16 bytes apart", name);
        if (groups && t->numel() > 0 && t->size(0) > 1) {
            if (rows == 1) *ld = t->stride(0);
            if (t->stride(0) != rows * *ld || *ld < cols || *ld % 16) refuse("%s must have its matrices one behind the other, rows a multiple of 16 bytes apart", name);
        }
        return t;
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

// Codes in a tensor whose type names another format than the call's argument does.
void format(const at::Tensor* t, int64_t fmt, const char* name, const char* arg) {
    if (!t) return;
    const at::ScalarType s = t->scalar_type();
    if (!(s == at::kFloat8_e4m3fn && fmt == FP8Q_E5M2) && !(s == at::kFloat8_e5m2 && fmt == FP8Q_E4M3FN)) return;
    PyErr_Format(PyExc_ValueError, "%s has dtype %s but %s is %s", name, c10::toString(s), arg, fmt == FP8Q_E5M2 ? "E5M2" : "E4M3FN");
    throw Refused();
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

// n elements in rows of `last`: their number alone would let a transposed result pass, to be filled in the wrong order.  Dimensions
// ahead of the last may be split or flattened together, and so may all.
void shaped(const at::Tensor* t, int64_t n, int64_t last, const char* name, const char* shape) {
    if (!t || (t->numel() == n && (n == 0 || t->dim() < 2 || t->size(-1) == last))) return;
    PyErr_Format(PyExc_ValueError, "%s must be %s (%lld elements in rows of %lld)", name, shape, (long long)n, (long long)last);
    throw Refused();
}

// (a, b, d, a_fmt, b_fmt, a_scale, b_scale, a_trans, b_trans, bias, act, residual, q, q_fmt, q_scale, amax, h, h_sf[, offsets], stream)
template <bool GROUPED>
int64_t product(PyObject* const* v, Py_ssize_t n) {
    Args a(GROUPED ? "grouped_matmul" : "matmul", v, n, GROUPED ? 20 : 19);
    fp8q_product p = {};
    const at::Tensor *x = a.codes("a", false, &p.lda), *w = a.codes("b", GROUPED, &p.ldb), *d = a.tensor(kGate, "d");
    p.a_fmt = (fp8q_format)a.integer();
    p.b_fmt = (fp8q_format)a.integer();
    const at::Tensor *sa = a.tensor(kF32, "a_scale"), *sb = a.tensor(kF32, "b_scale");
    p.a_trans = a.integer() != 0;
    p.b_trans = a.integer() != 0;
    const at::Tensor* bias = a.tensor(kGate, "bias");
    p.act = (fp8q_activation)a.integer();
    const at::Tensor *residual = a.tensor(kGate, "residual"), *q = a.tensor(kByte, "q");
    p.q_fmt = (fp8q_format)a.integer();
    const at::Tensor *qs = a.tensor(kF32, "q_scale"), *amax = a.tensor(kF32, "amax"), *h = a.tensor(kByte, "h"), *hs = a.tensor(kByte, "h_sf");
    const at::Tensor* offsets = GROUPED ? a.tensor(kI32, "offsets") : nullptr;
    const int64_t groups = GROUPED ? w->size(0) : 1, off = GROUPED ? 1 : 0;
    p.m = x->size(p.a_trans ? 1 : 0);
    p.k = x->size(p.a_trans ? 0 : 1);
    p.n = w->size(off + (p.b_trans ? 1 : 0));
    if (w->size(off + (p.b_trans ? 0 : 1)) != p.k) {
        PyErr_Format(PyExc_ValueError, "a and b must have the same k, not %lld and %lld", (long long)p.k,
                     (long long)w->size(off + (p.b_trans ? 0 : 1)));
        throw Refused();
    }
    if (GROUPED && (!offsets || offsets->numel() != groups + 1)) Args::refuse("%s must have one element more than b has matrices", "offsets");
    shaped(d, p.m * p.n, p.n, "d", "[m, n]");
    shaped(residual, p.m * p.n, p.n, "residual", "[m, n]");
    shaped(q, p.m * p.n, p.n, "q", "[m, n]");
    shaped(h, p.m * p.n, p.n, "h", "[m, n]");
    shaped(hs, p.m * ((p.n + 31) / 32), (p.n + 31) / 32, "h_sf", "[m, ceil(n / 32)]");
    shaped(bias, groups * p.n, p.n, "bias", GROUPED ? "[groups, n]" : "[n]");
    one(sa, "a_scale");
    one(sb, "b_scale");
    one(qs, "q_scale");
    one(amax, "amax");
    if (residual && residual->scalar_type() != (d ? d->scalar_type() : at::kBFloat16)) Args::refuse("%s must have d's type", "residual");
    format(x, p.a_fmt, "a", "a_fmt");
    format(w, p.b_fmt, "b", "b_fmt");
    format(q, p.q_fmt, "q", "q_fmt");
    format(h, FP8Q_E4M3FN, "h", "a checkpoint");
    p.a = bytes(x);
    p.b = bytes(w);
    p.a_scale = floats(sa);
    p.b_scale = floats(sb);
    p.bias = ptr(bias);
    p.bias_is_bf16 = bias && bias->scalar_type() == at::kBFloat16;
    p.residual = ptr(residual);
    p.d = ptr(d);
    p.out = d && d->scalar_type() == at::kFloat ? FP8Q_OUT_F32 : FP8Q_OUT_BF16;
    p.q = bytes(q);
    p.q_scale = floats(qs);
    p.amax = floats(amax);
    p.h = bytes(h);
    p.h_sf = bytes(hs);
    if (!GROUPED) return launch(g_product, &p, a.stream());
    return launch(g_grouped, &p, static_cast<int32_t*>(ptr(offsets)), (int32_t)(groups > INT32_MAX ? INT32_MAX : groups), a.stream());
}

// (a, b, offsets, d, a_fmt, b_fmt, a_scale, b_scale, residual, stream)
int64_t grouped_gradient(PyObject* const* v, Py_ssize_t n) {
    Args a("grouped_weight_gradient", v, n, 10);
    fp8q_product p = {};
    const at::Tensor *x = a.codes("a", false, &p.lda), *w = a.codes("b", false, &p.ldb), *offsets = a.tensor(kI32, "offsets"),
                     *d = a.tensor(kGate, "d");
    if (!d || d->dim() != 3) Args::refuse("%s must be [groups, m, n]", "d");
    p.a_fmt = (fp8q_format)a.integer();
    p.b_fmt = (fp8q_format)a.integer();
    const at::Tensor *sa = a.tensor(kF32, "a_scale"), *sb = a.tensor(kF32, "b_scale"), *residual = a.tensor(kGate, "residual");
    const int64_t groups = d->size(0);
    p.k = x->size(0);
    p.m = x->size(1);
    p.n = w->size(1);
    if (w->size(0) != p.k) Args::refuse("%s must have as many rows as a", "b");
    if (d->size(1) != p.m || d->size(2) != p.n) Args::refuse("%s must be [groups, m, n]", "d");
    if (!offsets || offsets->numel() != groups + 1) Args::refuse("%s must have one element more than d has matrices", "offsets");
    shaped(residual, groups * p.m * p.n, p.n, "residual", "[groups, m, n]");
    if (residual && residual->dim() == 3 && residual->sizes() != d->sizes()) Args::refuse("%s must be [groups, m, n]", "residual");
    if (residual && residual->scalar_type() != d->scalar_type()) Args::refuse("%s must have d's type", "residual");
    one(sa, "a_scale");
    one(sb, "b_scale");
    format(x, p.a_fmt, "a", "a_fmt");
    format(w, p.b_fmt, "b", "b_fmt");
    p.a = bytes(x);
    p.b = bytes(w);
    p.a_trans = p.b_trans = 1;
    p.a_scale = floats(sa);
    p.b_scale = floats(sb);
    p.residual = ptr(residual);
    p.d = ptr(d);
    p.out = d->scalar_type() == at::kFloat ? FP8Q_OUT_F32 : FP8Q_OUT_BF16;
    return launch(g_grouped_gradient, &p, static_cast<int32_t*>(ptr(offsets)), (int32_t)(groups > INT32_MAX ? INT32_MAX : groups), a.stream());
}

// (x, q, sf, stream) and (q, sf, y, stream)
template <bool BACK>
int64_t checkpoint(PyObject* const* v, Py_ssize_t n) {
    Args a(BACK ? "checkpoint_dequantize" : "checkpoint_quantize", v, n, 4);
    const at::Tensor* x = BACK ? nullptr : a.tensor(kBf16, "x", "[rows, cols]");
    const at::Tensor *q = a.tensor(kByte, "q"), *sf = a.tensor(kByte, "sf");
    if (BACK) x = a.tensor(kBf16, "y", "[rows, cols]");
    const int64_t rows = x->size(0), cols = x->size(1);
    if (!q || !sf) Args::refuse("%s must be a checkpoint: see checkpoint_empty", "(q, sf)");
    shaped(q, rows * cols, cols, "q", "[rows, cols]");
    shaped(sf, rows * ((cols + 31) / 32), (cols + 31) / 32, "sf", "[rows, ceil(cols / 32)]");
    format(q, FP8Q_E4M3FN, "q", "a checkpoint");
    return BACK ? launch(g_checkpoint_back, bytes(q), bytes(sf), ptr(x), rows, cols, a.stream())
                : launch(g_checkpoint, ptr(x), bytes(q), bytes(sf), rows, cols, a.stream());
}

// (d_y, h, h_sf, q, fmt, scale, amax, d_x, d_bias, workspace, stream)
int64_t gelu_backward(PyObject* const* v, Py_ssize_t n) {
    Args a("gelu_backward_quantize_amax", v, n, 11);
    fp8q_gelu_grad g = {};
    const at::Tensor *dy = a.tensor(kBf16, "d_y", "[rows, cols]"), *h = a.tensor(kByte, "h"), *hs = a.tensor(kByte, "h_sf"), *q = a.tensor(kByte, "q");
    g.fmt = (fp8q_format)a.integer();
    const at::Tensor *scale = a.tensor(kF32, "scale"), *amax = a.tensor(kF32, "amax"), *dx = a.tensor(kBf16, "d_x"),
                     *db = a.tensor(kF32, "d_bias"), *space = a.tensor(kByte, "workspace");
    g.rows = dy->size(0);
    g.cols = dy->size(1);
    shaped(h, g.rows * g.cols, g.cols, "h", "[rows, cols]");
    shaped(hs, g.rows * ((g.cols + 31) / 32), (g.cols + 31) / 32, "h_sf", "[rows, ceil(cols / 32)]");
    shaped(q, g.rows * g.cols, g.cols, "q", "[rows, cols]");
    shaped(dx, g.rows * g.cols, g.cols, "d_x", "[rows, cols]");
    shaped(db, g.cols, g.cols, "d_bias", "[cols]");
    one(scale, "scale");
    one(amax, "amax");
    format(h, FP8Q_E4M3FN, "h", "a checkpoint");
    format(q, g.fmt, "q", "fmt");
    g.d_y = ptr(dy);
    g.h = bytes(h);
    g.h_sf = bytes(hs);
    g.d_x = ptr(dx);
    g.q = bytes(q);
    g.scale = floats(scale);
    g.amax = floats(amax);
    g.d_bias = floats(db);
    g.workspace = ptr(space);
    g.workspace_bytes = space ? space->numel() : 0;
    return launch(g_gelu_backward, &g, a.stream());
}

// (rows, cols)
int64_t gelu_workspace(PyObject* const* v, Py_ssize_t n) {
    Args a("gelu_backward_workspace", v, n, 2);
    const int64_t rows = a.integer(), cols = a.integer();
    return g_gelu_workspace(rows, cols);
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

// Two contiguous byte tensors on the current CUDA device, in one allocation, the second behind the first (16-byte aligned).
PyObject* pair_of(at::IntArrayRef first, at::IntArrayRef second) {
    const auto o = at::TensorOptions().dtype(at::kByte).device(at::kCUDA, c10::cuda::current_device());
    const int64_t from = (c10::multiply_integers(first) + 15) / 16 * 16;
    const at::Tensor all = at::empty({from + c10::multiply_integers(second)}, o);
    const auto part = [&](at::IntArrayRef sizes, int64_t at) {
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
        t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
        t.unsafeGetTensorImpl()->set_storage_offset(at);
        return t;
    };
    PyObject* q = THPVariable_Wrap(part(first, 0));
    PyObject* sf = q ? THPVariable_Wrap(part(second, from)) : nullptr;
    PyObject* both = sf ? PyTuple_Pack(2, q, sf) : nullptr;
    Py_XDECREF(q);
    Py_XDECREF(sf);
    return both;
}

// (rows, cols, fmt): room for a packed operand; without fmt, for a checkpoint
template <bool CHECKPOINT>
PyObject* empty(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        constexpr Py_ssize_t kWant = CHECKPOINT ? 2 : 3;
        int64_t v[3] = {};
        for (Py_ssize_t i = 0; i < kWant; ++i) {
            v[i] = n == kWant ? PyLong_AsLongLong(a[i]) : -1;
            if (v[i] == -1 && PyErr_Occurred()) return nullptr;
        }
        // beyond what the calls take, the bytes of both arrays could pass 64 bits and come out as few
        constexpr int64_t kMax = 0x7FFFFC00;
        if (n != kWant || v[0] < 0 || v[1] < 0 || v[0] > kMax || v[1] > kMax || (!CHECKPOINT && !four_bits(v[2]))) {
            PyErr_SetString(PyExc_ValueError, CHECKPOINT ? "checkpoint_empty takes rows and cols from 0 to 2^31 - 1024"
                                                         : "fp4_empty takes rows and cols from 0 to 2^31 - 1024 and MXFP4 or NVFP4");
            return nullptr;
        }
        if (CHECKPOINT) return pair_of({v[0], v[1]}, {v[0], (v[1] + 31) / 32});
        return pair_of({v[0], row_bytes(v[1])}, {scale_bytes(v[0], v[1], v[2])});
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// Addresses of entry points, in the order of the calls below.
template <size_t N>
bool addresses(PyObject* const* a, Py_ssize_t n, void* (&p)[N]) {
    for (size_t i = 0; i < N; ++i) {
        p[i] = (Py_ssize_t)i < n ? PyLong_AsVoidPtr(a[i]) : nullptr;
        if (p[i]) continue;
        if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "bind takes %zu addresses", N);
        return false;
    }
    return true;
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[6];
    if (!addresses(a, n, p)) return nullptr;
    g_quantize = reinterpret_cast<decltype(g_quantize)>(p[0]);
    g_dequantize = reinterpret_cast<decltype(g_dequantize)>(p[1]);
    g_matmul = reinterpret_cast<decltype(g_matmul)>(p[2]);
    g_norm = reinterpret_cast<decltype(g_norm)>(p[3]);
    g_norm_backward = reinterpret_cast<decltype(g_norm_backward)>(p[4]);
    g_workspace = reinterpret_cast<decltype(g_workspace)>(p[5]);
    Py_RETURN_NONE;
}

PyObject* bind_products(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* p[7];
    if (!addresses(a, n, p)) return nullptr;
    g_product = reinterpret_cast<decltype(g_product)>(p[0]);
    g_grouped = reinterpret_cast<decltype(g_grouped)>(p[1]);
    g_grouped_gradient = reinterpret_cast<decltype(g_grouped_gradient)>(p[2]);
    g_checkpoint = reinterpret_cast<decltype(g_checkpoint)>(p[3]);
    g_checkpoint_back = reinterpret_cast<decltype(g_checkpoint_back)>(p[4]);
    g_gelu_backward = reinterpret_cast<decltype(g_gelu_backward)>(p[5]);
    g_gelu_workspace = reinterpret_cast<decltype(g_gelu_workspace)>(p[6]);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f))
PyMethodDef g_methods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                           {"bind_products", FAST(bind_products), METH_FASTCALL, nullptr},
                           {"fp4_empty", FAST(empty<false>), METH_FASTCALL, nullptr},
                           {"checkpoint_empty", FAST(empty<true>), METH_FASTCALL, nullptr},
                           {"fp4_quantize_amax", FAST(call<quantize>), METH_FASTCALL, nullptr},
                           {"fp4_dequantize", FAST(call<dequantize>), METH_FASTCALL, nullptr},
                           {"fp4_matmul", FAST(call<matmul>), METH_FASTCALL, nullptr},
                           {"residual_norm_quantize_amax", FAST(call<norm>), METH_FASTCALL, nullptr},
                           {"residual_norm_backward", FAST(call<norm_backward>), METH_FASTCALL, nullptr},
                           {"residual_norm_backward_workspace", FAST(call<workspace>), METH_FASTCALL, nullptr},
                           {"matmul", FAST(call<product<false>>), METH_FASTCALL, nullptr},
                           {"grouped_matmul", FAST(call<product<true>>), METH_FASTCALL, nullptr},
                           {"grouped_weight_gradient", FAST(call<grouped_gradient>), METH_FASTCALL, nullptr},
                           {"checkpoint_quantize", FAST(call<checkpoint<false>>), METH_FASTCALL, nullptr},
                           {"checkpoint_dequantize", FAST(call<checkpoint<true>>), METH_FASTCALL, nullptr},
                           {"gelu_backward_quantize_amax", FAST(call<gelu_backward>), METH_FASTCALL, nullptr},
                           {"gelu_backward_workspace", FAST(call<gelu_workspace>), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
