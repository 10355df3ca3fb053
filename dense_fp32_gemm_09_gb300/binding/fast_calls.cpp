// The usual form of the calls around the product, from Python to the C ABI in one step: CUDA
// tensors of the current device with ordinary strides on the current stream.  Each function
// returns None for anything else, and the Python code (mx4.py, norms.py, act8.py, layer_norms.py,
// gated.py), which states the checks and their messages, takes the call.  Nothing is computed here: outputs are
// allocated and sgemm_* functions called.  (A call of the Python code costs 7 to 24
// microseconds on the host where the kernels take 1 to 5.)
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>

#include "sgemm.h"

namespace {

decltype(&sgemm_mx4_quantize) f_quantize;
decltype(&sgemm_mx4_dequantize) f_dequantize;
decltype(&sgemm_mx4_matmul) f_matmul;
decltype(&sgemm_norm_forward) f_forward;
decltype(&sgemm_norm_backward_ws) f_backward;
decltype(&sgemm_norm_backward_workspace) f_backward_workspace;
decltype(&sgemm_act8_quantize) f_act8_quantize;
decltype(&sgemm_act8_dequantize) f_act8_dequantize;
decltype(&sgemm_layer_norm_forward) f_layer_norm;
decltype(&sgemm_layer_norm_backward) f_layer_norm_backward;
decltype(&sgemm_layer_norm_backward_workspace) f_layer_norm_workspace;
decltype(&sgemm_gated_ff_forward) f_gated_ff;
decltype(&sgemm_gated_ff_backward) f_gated_ff_backward;
decltype(&sgemm_gated_ff_workspace) f_gated_ff_workspace;

template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const std::exception&) {     // as torch raises it: torch.OutOfMemoryError, for one
        torch::translate_exception_to_python(std::current_exception());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}
PyObject* not_here() { Py_RETURN_NONE; }

int dtype_code(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return SGEMM_F32;
        case at::kBFloat16: return SGEMM_BF16;
        case at::kHalf: return SGEMM_F16;
        default: return -1;
    }
}
at::ScalarType dtype_of(int code) {
    return code == SGEMM_F32 ? at::kFloat : code == SGEMM_BF16 ? at::kBFloat16 : at::kHalf;
}
bool here(const at::Tensor& t) {
    return t.is_cuda() && t.device().index() == c10::cuda::current_device();
}
sgemm_stream_t stream() {
    return reinterpret_cast<sgemm_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
}
// Without Python's lock, as torch's own calls and those through ctypes: a launch waits where the
// queue is full, possibly for something that another thread of the program is to do.
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename... P, typename... A>
int unlocked(int (*f)(P...), A... a) {
    const Unlocked u;
    return f(a...);
}
at::Tensor empty(at::IntArrayRef size, at::ScalarType type) {
    const Unlocked u;
    return at::detail::empty_cuda(
        size, type, c10::Device(c10::DeviceType::CUDA, c10::cuda::current_device()), std::nullopt);
}
PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
// An optional tensor argument: false if it is neither None nor a tensor.
bool tensor(PyObject* o, at::Tensor* t) {
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) return false;
    *t = THPVariable_Unpack(o);
    return true;
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

struct Shape {
    long long rows, cols;
    at::ScalarType type;
};
// A matrix of this shape and type with unit column stride: its leading dimension, or -1.
int matrix(const at::Tensor& t, const Shape& s) {
    if (!t.defined()) return 0;
    if (t.dim() != 2 || t.size(0) != s.rows || t.size(1) != s.cols || t.scalar_type() != s.type ||
        !here(t))
        return -1;
    if (s.cols > 1 && t.stride(1) != 1) return -1;
    const long long ld = s.rows > 1 ? t.stride(0) : std::max(s.cols, 1LL);
    return ld < s.cols || ld > INT_MAX || s.rows > INT_MAX ? -1 : static_cast<int>(ld);
}
bool vector(const at::Tensor& t, long long n, at::ScalarType type) {
    return !t.defined() || (t.dim() == 1 && t.size(0) == n && t.scalar_type() == type && here(t) &&
                            (n <= 1 || t.stride(0) == 1));
}
bool one_float(const at::Tensor& t, int format) {
    return !t.defined() || (t.numel() == 1 && t.scalar_type() == at::kFloat && here(t) &&
                            format == SGEMM_NVFP4);
}
// Type code of the weights given, -1 where they do not agree.
int weights(const at::Tensor& a, const at::Tensor& b, const Shape& s) {
    const at::Tensor& any = a.defined() ? a : b;
    if (!any.defined()) return SGEMM_F32;
    const at::ScalarType type = any.scalar_type();
    if ((type != at::kFloat && type != s.type) || !vector(a, s.cols, type) ||
        !vector(b, s.cols, type))
        return -1;
    return dtype_code(any);
}
// Leading dimension of a gate: 0 for one row shared by all (or none), -1 if it fits neither.
int gate_ld(const at::Tensor& g, const Shape& s) {
    if (!g.defined()) return 0;
    if (g.dim() == 1) return vector(g, s.cols, s.type) ? 0 : -1;
    return matrix(g, s);
}
long long code_bytes(long long rows, long long cols) {
    return (rows + 127) / 128 * ((cols + 127) / 128) * 8192;
}
long long stored_bytes(long long rows, long long cols, int format) {
    const long long codes = code_bytes(rows, cols);
    return codes + codes / (format == SGEMM_NVFP4 ? 8 : 16);
}
at::Tensor stored(long long rows, long long cols, int format) {
    return empty({stored_bytes(rows, cols, format)}, at::kByte);
}
PyObject* status(int st) { return PyLong_FromLong(st); }

// mx4_quantize(x, format, tensor_scale) -> buffer
PyObject* mx4_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        at::Tensor x, ts;
        if (n != 3 || !tensor(a[0], &x) || !x.defined() || !tensor(a[2], &ts)) return not_here();
        const int format = static_cast<int>(PyLong_AsLong(a[1])), dt = dtype_code(x);
        if (dt < 0 || x.dim() != 2 || !here(x) || !one_float(ts, format)) return not_here();
        const long long rows = x.size(0), cols = x.size(1);
        if (rows < 1 || cols < 2 || rows > INT_MAX || cols > INT_MAX) return not_here();
        const int trans = x.stride(1) == 1 ? 0 : 1;
        if (trans && x.stride(0) != 1) return not_here();
        const long long lines = trans ? cols : rows, width = trans ? rows : cols;
        const long long ld = lines > 1 ? x.stride(trans) : width;
        if (ld < width || ld > INT_MAX) return not_here();
        at::Tensor q = stored(rows, cols, format);
        uint8_t* p = static_cast<uint8_t*>(q.data_ptr());
        const int st = unlocked(
            f_quantize, trans, rows, cols, dt, x.data_ptr(), ld, format,
                                  static_cast<const float*>(ptr(ts)), p, p + code_bytes(rows, cols),
                                  stream());
        return st ? status(st) : wrap(q);
    });
}

// Whether these buffers hold a rows x cols matrix: codes and scales, or both in one (no scales).
bool holds(const at::Tensor& codes, const at::Tensor& scales, const at::Tensor& ts, long long rows,
           long long cols, int format) {
    if (!codes.defined() || rows < 0 || cols < 0 || codes.scalar_type() != at::kByte ||
        !codes.is_contiguous() || !here(codes) || !one_float(ts, format))
        return false;
    if (!scales.defined()) return codes.dim() == 1 && codes.size(0) == stored_bytes(rows, cols, format);
    const long long rb = (rows + 127) / 128, cb = (cols + 127) / 128;
    const long long groups = cb * (format == SGEMM_NVFP4 ? 2 : 1);
    return codes.dim() == 4 && codes.size(0) == rb && codes.size(1) == 4 * cb &&
           codes.size(2) == 128 && codes.size(3) == 16 && scales.scalar_type() == at::kByte &&
           scales.dim() == 5 && scales.size(0) == rb && scales.size(1) == groups &&
           scales.size(2) == 32 && scales.size(3) == 4 && scales.size(4) == 4 &&
           scales.is_contiguous() && here(scales);
}
// Addresses of a matrix given as (codes, scales, tensor_scale), looked up in each call: a
// tensor's memory may be another one by the next.
bool stored_at(PyObject* t, long long rows, long long cols, int format, const void* (&p)[3]) {
    at::Tensor codes, scales, ts;
    if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 3 || !tensor(PyTuple_GET_ITEM(t, 0), &codes) ||
        !tensor(PyTuple_GET_ITEM(t, 1), &scales) || !tensor(PyTuple_GET_ITEM(t, 2), &ts) ||
        !holds(codes, scales, ts, rows, cols, format))
        return false;
    p[0] = codes.data_ptr();
    p[1] = scales.defined() ? scales.data_ptr()
                            : static_cast<uint8_t*>(codes.data_ptr()) + code_bytes(rows, cols);
    p[2] = ptr(ts);
    return true;
}

// mx4_holds((codes, scales, tensor_scale), rows, cols, format) -> True or None
PyObject* mx4_holds(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 4) return not_here();
        const long long rows = PyLong_AsLongLong(a[1]), cols = PyLong_AsLongLong(a[2]);
        const int format = static_cast<int>(PyLong_AsLong(a[3]));
        if (PyErr_Occurred()) return nullptr;
        const void* p[3];
        if (!stored_at(a[0], rows, cols, format, p)) return not_here();
        Py_RETURN_TRUE;
    });
}

// mx4_dequantize(stored, rows, cols, format, dtype code) -> tensor
PyObject* mx4_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 5) return not_here();
        const long rows = PyLong_AsLong(a[1]), cols = PyLong_AsLong(a[2]);
        const int format = static_cast<int>(PyLong_AsLong(a[3]));
        const int dt = static_cast<int>(PyLong_AsLong(a[4]));
        if (PyErr_Occurred()) return nullptr;
        const void* p[3];
        if (!stored_at(a[0], rows, cols, format, p)) return not_here();
        at::Tensor y = empty({rows, cols}, dtype_of(dt));
        const int st = unlocked(
            f_dequantize, rows, cols, format, p[0], p[1], static_cast<const float*>(p[2]),
                                    dt, y.data_ptr(), std::max(cols, 1L), stream());
        return st ? status(st) : wrap(y);
    });
}

// mx4_matmul(stored a, stored b, M, N, K, format, alpha, dtype code) -> tensor
PyObject* mx4_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 8) return not_here();
        const long M = PyLong_AsLong(a[2]), N = PyLong_AsLong(a[3]), K = PyLong_AsLong(a[4]);
        const int format = static_cast<int>(PyLong_AsLong(a[5]));
        const float alpha = static_cast<float>(PyFloat_AsDouble(a[6]));
        const int dt = static_cast<int>(PyLong_AsLong(a[7]));
        if (PyErr_Occurred()) return nullptr;
        const void *p[3], *q[3];
        if (!stored_at(a[0], M, K, format, p) || !stored_at(a[1], N, K, format, q))
            return not_here();
        at::Tensor c = empty({M, N}, dtype_of(dt));
        const int st = unlocked(
            f_matmul, M, N, K, format, alpha, p[0], p[1],
                                static_cast<const float*>(p[2]), q[0], q[1],
                                static_cast<const float*>(q[2]), 0.0f, dt, c.data_ptr(),
                                std::max(N, 1L), stream());
        return st ? status(st) : wrap(c);
    });
}

PyObject* tuple(std::initializer_list<at::Tensor> ts) {
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o = wrap(t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// norm_forward(residual, block, weight, gate, scale, eps, next, next_weight, format,
// tensor_scale) -> (y, rstd, h or the quantised buffer, next_rstd)
PyObject* norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        at::Tensor x, block, weight, gate, next_weight, ts;
        if (n != 10 || !tensor(a[0], &x) || !x.defined() || !tensor(a[1], &block) ||
            !tensor(a[2], &weight) || !tensor(a[3], &gate) || !tensor(a[7], &next_weight) ||
            !tensor(a[9], &ts) || x.dim() != 2)
            return not_here();
        const float scale = static_cast<float>(PyFloat_AsDouble(a[4]));
        const float eps = static_cast<float>(PyFloat_AsDouble(a[5]));
        const int next = PyObject_IsTrue(a[6]), format = static_cast<int>(PyLong_AsLong(a[8]));
        if (PyErr_Occurred()) return nullptr;
        const Shape s{x.size(0), x.size(1), x.scalar_type()};
        const int dt = dtype_code(x), ldr = matrix(x, s), ldb = matrix(block, s);
        const int wt = weights(weight, next_weight, s), ldg = gate_ld(gate, s);
        if (dt < 0 || s.cols < 1 || s.cols > INT_MAX || ldr < 0 || ldb < 0 || wt < 0 || ldg < 0 ||
            !one_float(ts, format))
            return not_here();
        at::Tensor y, rstd, h, next_rstd;
        if (block.defined()) {
            y = empty({s.rows, s.cols}, s.type);
            rstd = empty({s.rows}, at::kFloat);
        }
        uint8_t* codes = nullptr;
        if (next) {
            next_rstd = empty({s.rows}, at::kFloat);
            h = format < 0 ? empty({s.rows, s.cols}, s.type) : stored(s.rows, s.cols, format);
            if (format >= 0) codes = static_cast<uint8_t*>(h.data_ptr());
        }
        const int st = unlocked(
            f_forward, s.rows, s.cols, dt, ptr(block), ldb, x.data_ptr(), ldr, ptr(weight), ptr(next_weight),
            wt, ptr(gate), ldg, scale, eps, ptr(y), s.cols, static_cast<float*>(ptr(rstd)), next,
            codes ? nullptr : ptr(h), s.cols, static_cast<float*>(ptr(next_rstd)), format,
            static_cast<const float*>(ptr(ts)), codes,
            codes ? codes + code_bytes(s.rows, s.cols) : nullptr, stream());
        return st ? status(st) : tuple({y, rstd, h, next_rstd});
    });
}

// norm_backward(ref, dy, dh, y, next_rstd, next_weight, block, rstd, weight, gate, scale) ->
// (dx, dblock, dweight, dgate, dnext_weight)
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        at::Tensor ref, dy, dh, y, next_rstd, next_weight, block, rstd, weight, gate;
        at::Tensor* to[] = {&ref, &dy, &dh, &y, &next_rstd, &next_weight, &block, &rstd, &weight,
                            &gate};
        if (n != 11) return not_here();
        for (int i = 0; i < 10; ++i)
            if (!tensor(a[i], to[i])) return not_here();
        const float scale = static_cast<float>(PyFloat_AsDouble(a[10]));
        if (PyErr_Occurred()) return nullptr;
        if (!ref.defined() || ref.dim() != 2) return not_here();
        const Shape s{ref.size(0), ref.size(1), ref.scalar_type()};
        const int dt = dtype_code(ref), lddy = matrix(dy, s), lddh = matrix(dh, s);
        const int ldy = matrix(y, s), ldb = matrix(block, s), ldg = gate_ld(gate, s);
        const int wt = weights(weight, next_weight, s);
        if (dt < 0 || s.cols < 1 || s.cols > INT_MAX || lddy < 0 || lddh < 0 || ldy < 0 ||
            ldb < 0 || ldg < 0 || wt < 0 || !vector(rstd, s.rows, at::kFloat) ||
            !vector(next_rstd, s.rows, at::kFloat))
            return not_here();
        at::Tensor dx, dblock, dweight, dgate, dnext;
        if (dh.defined()) {
            dx = empty({s.rows, s.cols}, s.type);
            if (next_weight.defined()) dnext = empty({s.cols}, at::kFloat);
        }
        if (block.defined()) {
            dblock = empty({s.rows, s.cols}, s.type);
            if (weight.defined()) dweight = empty({s.cols}, at::kFloat);
            if (gate.defined())
                dgate = ldg ? empty({s.rows, s.cols}, s.type) : empty({s.cols}, at::kFloat);
        }
        // From torch's allocator, so that a captured graph owns what it uses.
        at::Tensor ws;
        size_t ws_bytes = 0;
        if (dweight.defined() || dnext.defined() || (dgate.defined() && ldg == 0)) {
            if (const int st = f_backward_workspace(s.rows, s.cols, &ws_bytes)) return status(st);
            ws = empty({static_cast<int64_t>(ws_bytes)}, at::kByte);
        }
        const int st = unlocked(
            f_backward, s.rows, s.cols, dt, ptr(dy), lddy, ptr(dh), lddh, ptr(y), ldy,
            static_cast<const float*>(ptr(next_rstd)), ptr(next_weight), ptr(block), ldb,
            static_cast<const float*>(ptr(rstd)), ptr(weight), wt, ptr(gate), ldg, scale, ptr(dx),
            s.cols, ptr(dblock), s.cols, ptr(dgate), s.cols, static_cast<float*>(ptr(dweight)),
            static_cast<float*>(ptr(dnext)), ptr(ws), ws_bytes, stream());
        return st ? status(st) : tuple({dx, dblock, dweight, dgate, dnext});
    });
}

// ----------------------------------------------------------------------------
// 8-bit checkpoints, layer norm, the gated feed-forward block
// ----------------------------------------------------------------------------
long long act8_blocks(long long cols) { return (cols + 63) / 64; }
// An unwritten checkpoint's buffers.
struct Kept {
    at::Tensor codes, scales;
    static Kept make(long long rows, long long cols) {
        return {empty({rows, 64 * act8_blocks(cols)}, at::kChar),
                empty({rows, act8_blocks(cols)}, at::kFloat)};
    }
    // Whether these hold a rows x cols matrix.
    bool holds(long long rows, long long cols) const {
        return codes.defined() && scales.defined() && codes.scalar_type() == at::kChar &&
               scales.scalar_type() == at::kFloat && codes.dim() == 2 && scales.dim() == 2 &&
               codes.size(0) == rows && scales.size(0) == rows &&
               codes.size(1) == 64 * act8_blocks(cols) && scales.size(1) == act8_blocks(cols) &&
               codes.is_contiguous() && scales.is_contiguous() && here(codes) && here(scales);
    }
};
float* floats(const at::Tensor& t) { return static_cast<float*>(ptr(t)); }
// Shape, type and leading dimension of a matrix that a call goes by; false if it is not usual.
bool leading(const at::Tensor& t, Shape* s, int* dt, int* ld) {
    if (!t.defined() || t.dim() != 2) return false;
    *s = Shape{t.size(0), t.size(1), t.scalar_type()};
    *dt = dtype_code(t);
    if (*dt < 0 || s->cols < 1 || s->cols > INT_MAX) return false;
    *ld = matrix(t, *s);
    return *ld >= 0;
}

// act8_quantize(x) -> (codes, scales)
PyObject* act8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        at::Tensor x;
        Shape s;
        int dt, ld;
        if (n != 1 || !tensor(a[0], &x) || !leading(x, &s, &dt, &ld)) return not_here();
        const Kept q = Kept::make(s.rows, s.cols);
        const int st = unlocked(f_act8_quantize, s.rows, s.cols, dt, x.data_ptr(), ld, ptr(q.codes),
                                floats(q.scales), stream());
        return st ? status(st) : tuple({q.codes, q.scales});
    });
}

// act8_dequantize(codes, scales, rows, cols, dtype code) -> tensor
PyObject* act8_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Kept q;
        if (n != 5 || !tensor(a[0], &q.codes) || !tensor(a[1], &q.scales)) return not_here();
        const long rows = PyLong_AsLong(a[2]), cols = PyLong_AsLong(a[3]);
        const int dt = static_cast<int>(PyLong_AsLong(a[4]));
        if (PyErr_Occurred()) return nullptr;
        if (!q.holds(rows, cols)) return not_here();
        at::Tensor y = empty({rows, cols}, dtype_of(dt));
        const int st = unlocked(f_act8_dequantize, rows, cols, ptr(q.codes), floats(q.scales), dt,
                                y.data_ptr(), std::max(cols, 1L), stream());
        return st ? status(st) : wrap(y);
    });
}

// layer_norm(x, weight, bias, eps, keep) -> (y, mean, rstd, codes, scales)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        at::Tensor x, weight, bias;
        Shape s;
        int dt, ld;
        if (n != 5 || !tensor(a[0], &x) || !tensor(a[1], &weight) || !tensor(a[2], &bias) ||
            !leading(x, &s, &dt, &ld))
            return not_here();
        const float eps = static_cast<float>(PyFloat_AsDouble(a[3]));
        const int keep = PyObject_IsTrue(a[4]);
        if (PyErr_Occurred()) return nullptr;
        const int wt = weights(weight, bias, s);
        if (wt < 0) return not_here();
        at::Tensor y = empty({s.rows, s.cols}, s.type), mean = empty({s.rows}, at::kFloat),
                   rstd = empty({s.rows}, at::kFloat);
        Kept q;
        if (keep) q = Kept::make(s.rows, s.cols);
        const int st = unlocked(f_layer_norm, s.rows, s.cols, dt, x.data_ptr(), ld, ptr(weight),
                                ptr(bias), wt, eps, y.data_ptr(), s.cols, floats(mean), floats(rstd),
                                ptr(q.codes), floats(q.scales), stream());
        return st ? status(st) : tuple({y, mean, rstd, q.codes, q.scales});
    });
}

// layer_norm_backward(dh, x, codes, scales, mean, rstd, weight, dy) -> (dx, dweight, dbias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        at::Tensor dh, x, mean, rstd, weight, dy;
        Kept q;
        at::Tensor* to[] = {&dh, &x, &q.codes, &q.scales, &mean, &rstd, &weight, &dy};
        if (n != 8) return not_here();
        for (int i = 0; i < 8; ++i)
            if (!tensor(a[i], to[i])) return not_here();
        Shape s;
        int dt, lddh;
        if (!leading(dh, &s, &dt, &lddh)) return not_here();
        const int ldx = matrix(x, s), lddy = matrix(dy, s), wt = weights(weight, at::Tensor(), s);
        if (ldx < 0 || lddy < 0 || wt < 0 || x.defined() == q.codes.defined() || !mean.defined() ||
            !rstd.defined() || !vector(mean, s.rows, at::kFloat) ||
            !vector(rstd, s.rows, at::kFloat) || (!x.defined() && !q.holds(s.rows, s.cols)))
            return not_here();
        at::Tensor dx = empty({s.rows, s.cols}, s.type), dweight, dbias = empty({s.cols}, at::kFloat);
        if (weight.defined()) dweight = empty({s.cols}, at::kFloat);
        // From torch's allocator, so that a captured graph owns what it uses.
        size_t ws_bytes = 0;
        if (const int st = f_layer_norm_workspace(s.rows, s.cols, &ws_bytes)) return status(st);
        at::Tensor ws = empty({static_cast<int64_t>(ws_bytes)}, at::kByte);
        const int st = unlocked(f_layer_norm_backward, s.rows, s.cols, dt, dh.data_ptr(), lddh, ptr(dy),
                                lddy, ptr(x), x.defined() ? ldx : static_cast<int>(s.cols),
                                ptr(q.codes), floats(q.scales), floats(mean), floats(rstd),
                                ptr(weight), wt, dx.data_ptr(), s.cols, floats(dweight),
                                floats(dbias), ws.data_ptr(), ws_bytes, stream());
        return st ? status(st) : tuple({dx, dweight, dbias});
    });
}

// Whether a block reads a copy of these rows (include/sgemm.h).
int packed(int bit, const at::Tensor& t, int ld) {
    return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 && (t.size(0) <= 1 || ld % 8 == 0) ? 0
                                                                                                  : bit;
}
// The two weights of a block whose tokens are of type `type`.
struct Layer {
    long long N = 0, K = 0;
    int ldg = -1, ldu = -1;
    bool usual(const at::Tensor& wg, const at::Tensor& wu, at::ScalarType type) {
        if (!wg.defined() || !wu.defined() || wg.dim() != 2) return false;
        N = wg.size(0);
        K = wg.size(1);
        if (N < 1 || K < 1 || K > INT_MAX) return false;
        const Shape s{N, K, type};
        ldg = matrix(wg, s);
        ldu = matrix(wu, s);
        return ldg >= 0 && ldu >= 0;
    }
};
at::Tensor workspace(size_t bytes) {
    return bytes ? empty({static_cast<int64_t>(bytes)}, at::kByte) : at::Tensor();
}

// gated_ff(x, w_gate, w_up, activation, keep) -> (h, gate, up, gate_scales, up_scales)
PyObject* gated_ff(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        at::Tensor x, wg, wu;
        Shape s;
        int dt, ldx;
        Layer w;
        if (n != 5 || !tensor(a[0], &x) || !tensor(a[1], &wg) || !tensor(a[2], &wu) ||
            !leading(x, &s, &dt, &ldx) || dt == SGEMM_F32 || !w.usual(wg, wu, s.type) || w.K != s.cols)
            return not_here();
        const int act = static_cast<int>(PyLong_AsLong(a[3]));
        const int keep = static_cast<int>(PyLong_AsLong(a[4]));
        if (PyErr_Occurred()) return nullptr;
        const long long M = s.rows;
        at::Tensor h = empty({M, w.N}, s.type);
        Kept gate, up;
        const long long ldk = keep == SGEMM_KEEP_FULL ? (w.N + 7) / 8 * 8 : w.N;
        if (keep == SGEMM_KEEP_FULL) {
            for (at::Tensor* t : {&gate.codes, &up.codes}) {
                *t = empty({M, ldk}, s.type);
                if (ldk != w.N) *t = t->narrow(1, 0, w.N);
            }
        } else if (keep == SGEMM_KEEP_8BIT) {
            gate = Kept::make(M, w.N);
            up = Kept::make(M, w.N);
        }
        size_t bytes = 0;
        const bool in_place = M <= 16 && keep != SGEMM_KEEP_8BIT;       // (include/sgemm.h)
        const int pack =
            in_place ? 0 : packed(1, x, ldx) | packed(2, wg, w.ldg) | packed(4, wu, w.ldu);
        if (pack)
            if (const int st = f_gated_ff_workspace(M, w.N, w.K, 0, pack, &bytes)) return status(st);
        const at::Tensor ws = workspace(bytes);
        const int st = unlocked(f_gated_ff, M, w.N, w.K, dt, act, x.data_ptr(), ldx, wg.data_ptr(),
                                w.ldg, wu.data_ptr(), w.ldu, h.data_ptr(), w.N, keep, ptr(gate.codes),
                                ptr(up.codes), ldk, floats(gate.scales), floats(up.scales), ptr(ws),
                                bytes, stream());
        return st ? status(st) : tuple({h, gate.codes, up.codes, gate.scales, up.scales});
    });
}

// gated_ff_backward(dh, x, x_codes, x_scales, w_gate, w_up, gate, up, gate_scales, up_scales,
// activation, return_h) -> (dx, dw_gate, dw_up, h)
PyObject* gated_ff_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        at::Tensor dh, x, wg, wu;
        Kept kx, gate, up;
        at::Tensor* to[] = {&dh, &x, &kx.codes, &kx.scales, &wg, &wu,
                            &gate.codes, &up.codes, &gate.scales, &up.scales};
        if (n != 12) return not_here();
        for (int i = 0; i < 10; ++i)
            if (!tensor(a[i], to[i])) return not_here();
        const int act = static_cast<int>(PyLong_AsLong(a[10])), again = PyObject_IsTrue(a[11]);
        if (PyErr_Occurred()) return nullptr;
        Shape s;
        int dt, lddh;
        Layer w;
        if (!leading(dh, &s, &dt, &lddh) || dt == SGEMM_F32 || !w.usual(wg, wu, s.type) || w.N != s.cols)
            return not_here();
        const long long M = s.rows;
        const int ldx = matrix(x, Shape{M, w.K, s.type});
        if (ldx < 0 || x.defined() == kx.codes.defined() || (!x.defined() && !kx.holds(M, w.K)) ||
            !gate.codes.defined() || !up.codes.defined())
            return not_here();
        int keep = SGEMM_KEEP_8BIT, ldk = static_cast<int>(w.N);
        if (!gate.scales.defined() && !up.scales.defined()) {
            keep = SGEMM_KEEP_FULL;
            ldk = matrix(gate.codes, s);
            if (ldk < 0 || matrix(up.codes, s) != ldk) return not_here();
        } else if (!gate.holds(M, w.N) || !up.holds(M, w.N)) {
            return not_here();
        }
        at::Tensor dx = empty({M, w.K}, s.type), dwg = empty({w.N, w.K}, s.type),
                   dwu = empty({w.N, w.K}, s.type), h;
        if (again) h = empty({M, w.N}, s.type);
        const int pack = (x.defined() ? packed(1, x, ldx) : 1) | packed(2, wg, w.ldg) |
                         packed(4, wu, w.ldu) | (dt == SGEMM_F16 ? 8 : 0);
        size_t bytes = 0;
        if (const int st = f_gated_ff_workspace(M, w.N, w.K, 1, pack, &bytes)) return status(st);
        const at::Tensor ws = workspace(bytes);
        const int st = unlocked(
            f_gated_ff_backward, M, w.N, w.K, dt, act, dh.data_ptr(), lddh, ptr(x),
            x.defined() ? ldx : static_cast<int>(w.K), ptr(kx.codes), floats(kx.scales), wg.data_ptr(),
            w.ldg, wu.data_ptr(), w.ldu, keep, ptr(gate.codes), ptr(up.codes), ldk,
            floats(gate.scales), floats(up.scales), dx.data_ptr(), w.K, dwg.data_ptr(), w.K,
            dwu.data_ptr(), w.K, ptr(h), w.N, ptr(ws), bytes, stream());
        return st ? status(st) : tuple({dx, dwg, dwu, h});
    });
}

// The C functions' addresses, in the order given.
template <size_t COUNT>
PyObject* take(PyObject* const* a, Py_ssize_t n, const char* name, void** const (&to)[COUNT]) {
    if (n != static_cast<Py_ssize_t>(COUNT)) {
        PyErr_Format(PyExc_TypeError, "%s takes %zu addresses", name, COUNT);
        return nullptr;
    }
    void* p[COUNT];
    for (size_t i = 0; i < COUNT; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
    for (size_t i = 0; i < COUNT; ++i) *to[i] = p[i];
    Py_RETURN_NONE;
}
template <typename F>
void** slot(F& f) { return reinterpret_cast<void**>(&f); }
// bind(those of the 4-bit operands and the norms)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void** const to[] = {slot(f_quantize), slot(f_dequantize), slot(f_matmul),
                         slot(f_forward), slot(f_backward), slot(f_backward_workspace)};
    return take(a, n, "bind", to);
}
// bind_train(those of the checkpoints, layer norm and the feed-forward block)
PyObject* bind_train(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void** const to[] = {slot(f_act8_quantize), slot(f_act8_dequantize), slot(f_layer_norm),
                         slot(f_layer_norm_backward), slot(f_layer_norm_workspace),
                         slot(f_gated_ff), slot(f_gated_ff_backward), slot(f_gated_ff_workspace)};
    return take(a, n, "bind_train", to);
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {METHOD(bind), METHOD(bind_train), METHOD(mx4_holds), METHOD(mx4_quantize), METHOD(mx4_dequantize),
                          METHOD(mx4_matmul), METHOD(norm_forward), METHOD(norm_backward),
                          METHOD(act8_quantize), METHOD(act8_dequantize), METHOD(layer_norm),
                          METHOD(layer_norm_backward), METHOD(gated_ff), METHOD(gated_ff_backward),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fast_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast_calls() { return PyModule_Create(&kModule); }
