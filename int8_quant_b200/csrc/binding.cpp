// binding.cpp — the Python binding of the layer operators (ssd_add_rmsnorm_i8, ssd_gated_rmsnorm_i8,
// ssd_matmul_i8, ssd_conv_fwd_bf16, ssd_conv_step_bf16): checks the tensors, takes the stream and calls the
// C ABI.  In C++ because a one-token step is a handful of microseconds on the GPU: checking and marshalling
// its tensors in Python (through ctypes) takes 10 to 14 us a call, here under one.
//
// Every function returns None, or (status, detail) for the caller to raise.  The kernels launch on the
// tensors' device, whatever the current one is; a stream of None is that device's current stream.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/SmallVector.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/ssd.h"

namespace {

using Sizes = c10::SmallVector<int64_t, 5>;                        // on the stack

// A refusal: status SSD_ERR_INVALID_ARG with its reason.
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

std::string text(c10::IntArrayRef v) {
    std::string s = "[";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused(std::string(name) + " has to be a tensor");
    return THPVariable_Unpack(o);
}

struct Call {
    int dev = -1;

    // the device of the call is that of its first tensor
    const at::Tensor& first(PyObject* o, const char* name) {
        const at::Tensor& t = tensor(o, name);
        if (!t.is_cuda()) throw Refused("the tensors have to be on a CUDA device, not on " + t.device().str());
        dev = t.get_device();
        return t;
    }
    [[noreturn]] void bad(const at::Tensor& t, const char* name, at::ScalarType type, c10::IntArrayRef shape,
                          const char* form) const {
        throw Refused(std::string(name) + " has to be a " + form + c10::toString(type) + " tensor " + text(shape) +
                      " on cuda:" + std::to_string(dev) + "; it is " + c10::toString(t.scalar_type()) + ' ' +
                      text(t.sizes()) + ", strides " + text(t.strides()) + ", on " + t.device().str());
    }
    bool fits(const at::Tensor& t, at::ScalarType type, c10::IntArrayRef shape) const {
        return t.scalar_type() == type && t.sizes() == shape && t.is_cuda() && t.get_device() == dev;
    }
    template <typename T>
    T* dense(PyObject* o, const char* name, at::ScalarType type, c10::IntArrayRef shape) const {
        const at::Tensor& t = tensor(o, name);
        if (!fits(t, type, shape) || !t.is_contiguous()) bad(t, name, type, shape, "contiguous ");
        return static_cast<T*>(t.data_ptr());
    }
    template <typename T>
    T* optional(PyObject* o, const char* name, at::ScalarType type, c10::IntArrayRef shape) const {
        return o == Py_None ? nullptr : dense<T>(o, name, type, shape);
    }
    // A tensor whose rows (its last axis) are evenly spaced: dense, or a slice of wider rows.  *ld receives the
    // elements from row to row, or 0 where there are fewer than two rows.
    uint16_t* rows(PyObject* o, const char* name, c10::IntArrayRef shape, int64_t* ld) const {
        const at::Tensor& t = tensor(o, name);
        if (!fits(t, at::kBFloat16, shape)) bad(t, name, at::kBFloat16, shape, "");
        const auto st = t.strides();
        const size_t n = shape.size() - 1;
        *ld = 0;
        int64_t count = 1;
        if (t.numel() > 0) {
            if (shape[n] > 1 && st[n] != 1) bad(t, name, at::kBFloat16, shape, "row-contiguous ");
            for (size_t i = n; i-- > 0;) {
                if (shape[i] == 1) continue;                      // an axis of one element has no stride of its own
                if (count == 1) *ld = st[i];
                else if (st[i] != *ld * count) bad(t, name, at::kBFloat16, shape, "row-contiguous, evenly spaced ");
                count *= shape[i];
            }
            if (count > 1 && *ld <= 0) bad(t, name, at::kBFloat16, shape, "row-contiguous, not expanded ");
        }
        return static_cast<uint16_t*>(t.data_ptr());
    }
    template <typename F>
    PyObject* launch(PyObject* stream, F f) const {
        cudaStream_t st;
        if (stream == Py_None) {
            st = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        } else {
            st = static_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
            if (PyErr_Occurred()) {
                PyErr_Clear();
                throw Refused("stream has to be None, a stream or its handle");
            }
        }
        ssd_status s;
        {
            std::optional<c10::cuda::CUDAGuard> guard;
            if (c10::cuda::current_device() != dev) guard.emplace((c10::DeviceIndex)dev);
            Py_BEGIN_ALLOW_THREADS
            s = f(st);
            Py_END_ALLOW_THREADS
        }
        if (s == SSD_OK) Py_RETURN_NONE;
        return Py_BuildValue("(is)", (int)s, "");
    }
};

int as_int(int64_t v, const char* what) {
    if (v > 0x7fffffff) throw Refused(std::string(what) + " has 2^31 elements or more along an axis");
    return (int)v;
}

template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F f) {
    if (have != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, have);
        return nullptr;
    }
    try {
        return f();
    } catch (const std::exception& e) {                           // Refused, or torch's own (a tensor without memory)
        return Py_BuildValue("(is)", (int)SSD_ERR_INVALID_ARG, e.what());
    }
}

double as_double(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused(std::string(name) + " has to be a number");
    }
    return v;
}

// (x, residual, weight, eps, residual_out, q, scale, values, stream)
PyObject* add_rmsnorm_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        Call c;
        const at::Tensor& x = c.first(a[0], "x");
        if (x.dim() != 2) throw Refused("x has to be [tokens, d], not " + text(x.sizes()));
        const auto shape = x.sizes();
        const int T = as_int(shape[0], "x"), d = as_int(shape[1], "x");
        const bool res = a[1] != Py_None;
        // the residual stream's type: the residual's, or without one that of residual_out
        PyObject* stream_of = res ? a[1] : a[4];
        const bool fp32 = stream_of != Py_None && tensor(stream_of, "residual").scalar_type() == at::kFloat;
        const at::ScalarType kept = fp32 ? at::kFloat : at::kBFloat16;
        const uint16_t* xp = c.dense<uint16_t>(a[0], "x", at::kBFloat16, shape);
        const void* rp = c.optional<void>(a[1], "residual", kept, shape);
        const float* w = c.optional<float>(a[2], "weight", at::kFloat, {shape[1]});
        const float eps = (float)as_double(a[3], "eps");
        void* ro = c.optional<void>(a[4], "residual_out", kept, shape);
        int8_t* q = c.dense<int8_t>(a[5], "q", at::kChar, shape);
        float* s = c.dense<float>(a[6], "scale", at::kFloat, {shape[0]});
        uint16_t* val = c.optional<uint16_t>(a[7], "values", at::kBFloat16, shape);
        return c.launch(a[8], [&](cudaStream_t st) {
            return ssd_add_rmsnorm_i8(T, d, xp, rp, fp32, w, eps, ro, q, s, val, st);
        });
    });
}

// (y, z, weight, eps, q, scale, values, stream)
PyObject* gated_rmsnorm_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        Call c;
        const at::Tensor& y = c.first(a[0], "y");
        if (y.dim() != 2) throw Refused("y has to be [tokens, d], not " + text(y.sizes()));
        const auto shape = y.sizes();
        const int T = as_int(shape[0], "y"), d = as_int(shape[1], "y");
        const uint16_t* yp = c.dense<uint16_t>(a[0], "y", at::kBFloat16, shape);
        int64_t ld;
        const uint16_t* zp = c.rows(a[1], "z", shape, &ld);
        const float* w = c.optional<float>(a[2], "weight", at::kFloat, {shape[1]});
        const float eps = (float)as_double(a[3], "eps");
        int8_t* q = c.dense<int8_t>(a[4], "q", at::kChar, shape);
        float* s = c.dense<float>(a[5], "scale", at::kFloat, {shape[0]});
        uint16_t* val = c.optional<uint16_t>(a[6], "values", at::kBFloat16, shape);
        return c.launch(a[7], [&](cudaStream_t st) {
            return ssd_gated_rmsnorm_i8(T, d, yp, zp, ld ? ld : d, w, eps, q, s, val, st);
        });
    });
}

// (q, s_t, Wq, s_w, bias, out, status, stream)
PyObject* matmul_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        Call c;
        const at::Tensor& q = c.first(a[0], "q");
        const at::Tensor& w = tensor(a[2], "Wq");
        if (q.dim() != 2 || w.dim() != 2) throw Refused("q has to be [tokens, k] and Wq [n, k]");
        const int64_t T = q.size(0), K = q.size(1), N = w.size(0);
        const int Ti = as_int(T, "q"), Ki = as_int(K, "q"), Ni = as_int(N, "Wq");
        const int8_t* qp = c.dense<int8_t>(a[0], "q", at::kChar, {T, K});
        const float* st_ = c.dense<float>(a[1], "s_t", at::kFloat, {T});
        const int8_t* wp = c.dense<int8_t>(a[2], "Wq", at::kChar, {N, K});
        const float* sw = c.dense<float>(a[3], "s_w", at::kFloat, {N});
        const float* b = c.optional<float>(a[4], "bias", at::kFloat, {N});
        uint16_t* out = c.dense<uint16_t>(a[5], "out", at::kBFloat16, {T, N});
        int* status = c.dense<int>(a[6], "status", at::kInt, {1});
        return c.launch(a[7], [&](cudaStream_t st) {
            return ssd_matmul_i8(Ti, Ki, Ni, qp, st_, wp, sw, b, out, status, st);
        });
    });
}

struct Conv {
    Call c;
    ssd_shape shape{};
    int64_t width = 0, ch = 0, ld = 0;
    const uint16_t* xbc;
    const uint16_t* dt_raw = nullptr;
    const float *weight, *bias, *dt_bias;
    uint16_t *x, *B, *C;
    float* dt;

    // lead: the axes in front of [H, P], {b, L} or {b}
    Conv(size_t lead_n, PyObject* xbc_o, PyObject* dt_raw_o, PyObject* w_o, PyObject* bias_o, PyObject* dt_bias_o,
         PyObject* x_o, PyObject* dt_o, PyObject* B_o, PyObject* C_o) {
        const at::Tensor& xt = c.first(x_o, "x");
        const at::Tensor& bt = tensor(B_o, "B");
        const at::Tensor& wt = tensor(w_o, "weight");
        if ((size_t)xt.dim() != lead_n + 2 || (size_t)bt.dim() != lead_n + 2 || wt.dim() != 2)
            throw Refused(lead_n == 2 ? "x has to be [batch, seqlen, H, P], B [batch, seqlen, G, N], weight [width, channels]"
                                      : "x has to be [batch, H, P], B [batch, G, N] and weight [width, channels]");
        const int64_t H = xt.size(lead_n), P = xt.size(lead_n + 1), G = bt.size(lead_n), N = bt.size(lead_n + 1);
        shape = ssd_shape{as_int(xt.size(0), "x"), lead_n == 2 ? as_int(xt.size(1), "x") : 1, as_int(H, "x"),
                          as_int(P, "x"), as_int(G, "B"), as_int(N, "B"), 256};
        ch = H * P + 2 * G * N;
        width = wt.size(0);
        Sizes s(xt.sizes().begin(), xt.sizes().begin() + lead_n);
        const auto with = [&](std::initializer_list<int64_t> tail) {
            Sizes v = s;
            v.append(tail.begin(), tail.end());
            return v;
        };
        xbc = c.rows(xbc_o, "xbc", with({ch}), &ld);
        if (dt_raw_o != Py_None) {
            int64_t ld_dt;
            dt_raw = c.rows(dt_raw_o, "dt_raw", with({H}), &ld_dt);
            if (ld_dt != ld)
                throw Refused("the rows of xbc and dt_raw have to be equally far apart, not " + std::to_string(ld) +
                              " and " + std::to_string(ld_dt) + " elements");
        }
        if (ld == 0) ld = (ch + 7) / 8 * 8;                        // a single row
        weight = c.dense<float>(w_o, "weight", at::kFloat, {width, ch});
        bias = c.optional<float>(bias_o, "bias", at::kFloat, {ch});
        dt_bias = c.optional<float>(dt_bias_o, "dt_bias", at::kFloat, {H});
        x = c.dense<uint16_t>(x_o, "x", at::kBFloat16, with({H, P}));
        dt = c.optional<float>(dt_o, "dt", at::kFloat, with({H}));
        B = c.dense<uint16_t>(B_o, "B", at::kBFloat16, with({G, N}));
        C = c.dense<uint16_t>(C_o, "C", at::kBFloat16, with({G, N}));
    }
};

// (xbc, dt_raw, weight, bias, dt_bias, lengths, initial_state, x, dt, B, C, final_state, stream)
PyObject* conv_fwd_bf16(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const Conv v(2, a[0], a[1], a[2], a[3], a[4], a[7], a[8], a[9], a[10]);
        const Sizes state{v.shape.batch, v.width - 1, v.ch};
        const int* lengths = v.c.optional<int>(a[5], "lengths", at::kInt, {v.shape.batch});
        const uint16_t* init = v.c.optional<uint16_t>(a[6], "initial_state", at::kBFloat16, state);
        uint16_t* fin = v.c.optional<uint16_t>(a[11], "final_state", at::kBFloat16, state);
        return v.c.launch(a[12], [&](cudaStream_t st) {
            return ssd_conv_fwd_bf16(&v.shape, (int)v.width, v.xbc, v.dt_raw, v.ld, v.weight, v.bias, v.dt_bias,
                                     lengths, init, v.x, v.dt, v.B, v.C, fin, st);
        });
    });
}

// (xbc, dt_raw, weight, bias, dt_bias, state, x, dt, B, C, stream)
PyObject* conv_step_bf16(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const Conv v(1, a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8], a[9]);
        const Sizes shape{v.shape.batch, v.width - 1, v.ch};
        uint16_t* state = v.c.dense<uint16_t>(a[5], "state", at::kBFloat16, shape);
        return v.c.launch(a[10], [&](cudaStream_t st) {
            return ssd_conv_step_bf16(&v.shape, (int)v.width, v.xbc, v.dt_raw, v.ld, v.weight, v.bias, v.dt_bias,
                                      state, v.x, v.dt, v.B, v.C, st);
        });
    });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr

PyMethodDef methods[] = {{"add_rmsnorm_i8", FAST(add_rmsnorm_i8)},   {"gated_rmsnorm_i8", FAST(gated_rmsnorm_i8)},
                         {"matmul_i8", FAST(matmul_i8)},             {"conv_fwd_bf16", FAST(conv_fwd_bf16)},
                         {"conv_step_bf16", FAST(conv_step_bf16)},   {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
    PyObject* m = PyModule_Create(&module);
    // its calls read torch's objects directly, so it serves the torch that it was built for alone
    if (m && PyModule_AddStringConstant(m, "torch_version", SSD_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
