// m3_call.cpp -- native argument handling of the binding's calls that a decode
// loop makes for every token and layer (CPython extension _m3_call).
//
// A small call takes the GPU 2 to 4 us, and checking its tensors one method call
// at a time in Python took 7 to 9 us.  A function here reads the dims, checks
// every tensor (a CUDA tensor of the expected type, size and device,
// contiguous) and calls the C entry point on the device's current stream: 3 us.
// Whatever is not as expected (another device than the current one, a stream
// given by the caller, a wrong tensor) gives None: the caller's Python code
// then handles the call or raises the error that names the argument.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "m3.h"

namespace {

decltype(&m3_delta_step) p_delta_step;
decltype(&m3_delta_fwd) p_delta_fwd;
decltype(&m3_delta_bwd) p_delta_bwd;
decltype(&m3_rms_norm_fwd) p_norm_fwd;
decltype(&m3_rms_norm_bwd) p_norm_bwd;

constexpr int kFields = 9;
static_assert(sizeof(m3_dims) == kFields * sizeof(int), "m3_dims is nine ints");
const char* const kFieldNames[kFields] = {"batch", "seqlen", "nheads", "ngroups", "headdim",
                                          "dstate", "rank", "chunk", "io_dtype"};
PyObject* field_name[kFields];

struct Refuse {};                        // not as expected: the Python code takes over

m3_dims dims_of(PyObject* o) {
    m3_dims d;
    int* out = reinterpret_cast<int*>(&d);
    for (int i = 0; i < kFields; ++i) {
        PyObject* v = PyObject_GetAttr(o, field_name[i]);
        if (!v) throw Refuse();
        const long long x = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if ((x == -1 && PyErr_Occurred()) || x < INT_MIN || x > INT_MAX) throw Refuse();
        out[i] = (int)x;
    }
    return d;
}

const at::Tensor& tensor_of(PyObject* o) {
    if (!THPVariable_Check(o)) throw Refuse();
    return THPVariable_Unpack(o);
}

// the device of a call's tensors (the current one), its stream, and what a call's tensors have to be
struct Call {
    int dev;
    void* stream;
    at::ScalarType io;

    Call(const at::Tensor& t, at::ScalarType io_type) : io(io_type) {
        if (!t.is_cuda()) throw Refuse();
        dev = t.get_device();
        if (dev != (int)c10::cuda::current_device()) throw Refuse();
        stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    }
    void* ptr(PyObject* o, at::ScalarType type, int64_t numel) const {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor_of(o);
        if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.numel() != numel || !t.is_contiguous())
            throw Refuse();
        return t.data_ptr();
    }
    void* arg(PyObject* o, int64_t numel) const { return ptr(o, io, numel); }
    float* f32(PyObject* o, int64_t numel) const { return static_cast<float*>(ptr(o, at::kFloat, numel)); }
    void* workspace(PyObject* o, size_t* bytes) const {
        const at::Tensor& t = tensor_of(o);
        *bytes = (size_t)t.numel() * t.element_size();
        return ptr(o, t.scalar_type(), t.numel());
    }
};

float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refuse();
    return (float)v;
}

at::ScalarType io_of(const m3_dims& d) { return d.io_dtype == M3_BF16 ? at::kBFloat16 : at::kFloat; }
at::ScalarType io_of(const at::Tensor& t) {
    const at::ScalarType s = t.scalar_type();
    if (s != at::kBFloat16 && s != at::kFloat) throw Refuse();
    return s;
}

// runs `body(args)` for `want` arguments: its status, or None
template <typename F>
PyObject* guarded(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, F body) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)body(a));
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}
template <typename F>
m3_status unlocked(F f) {                // the C entry points throw nothing
    m3_status s;
    Py_BEGIN_ALLOW_THREADS
    s = f();
    Py_END_ALLOW_THREADS
    return s;
}

struct Sizes {
    int64_t k, v, g, h;                  // q and k; v and y; g and beta; a state
    Sizes(const m3_dims& d, int64_t tokens)
        : k(tokens * d.ngroups * d.dstate), v(tokens * d.nheads * d.headdim), g(tokens * d.nheads),
          h((int64_t)d.batch * d.nheads * d.headdim * d.dstate) {}
};

// dims, h, h_out, q, k, v, g, beta, scale, y
PyObject* delta_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, 10, [](PyObject* const* a) {
        const m3_dims d = dims_of(a[0]);
        const Call c(tensor_of(a[3]), io_of(d));
        const Sizes z(d, d.batch);
        const float *hi = c.f32(a[1], z.h), *g = c.f32(a[6], z.g), *beta = c.f32(a[7], z.g);
        float* ho = c.f32(a[2], z.h);
        const void *q = c.arg(a[3], z.k), *k = c.arg(a[4], z.k), *v = c.arg(a[5], z.v);
        const float scale = real(a[8]);
        void* y = c.arg(a[9], z.v);
        return unlocked([&] { return p_delta_step(&d, hi, ho, q, k, v, g, beta, scale, y, c.stream); });
    });
}

// dims, q, k, v, g, beta, scale, lengths, init_h, y, final_h, workspace
PyObject* delta_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, 12, [](PyObject* const* a) {
        const m3_dims d = dims_of(a[0]);
        const Call c(tensor_of(a[1]), io_of(d));
        const Sizes z(d, (int64_t)d.batch * d.seqlen);
        const void *q = c.arg(a[1], z.k), *k = c.arg(a[2], z.k), *v = c.arg(a[3], z.v);
        const float *g = c.f32(a[4], z.g), *beta = c.f32(a[5], z.g), *h0 = c.f32(a[8], z.h);
        const float scale = real(a[6]);
        const int* len = static_cast<const int*>(c.ptr(a[7], at::kInt, d.batch));
        void* y = c.arg(a[9], z.v);
        float* h1 = c.f32(a[10], z.h);
        size_t bytes;
        void* ws = c.workspace(a[11], &bytes);
        return unlocked([&] { return p_delta_fwd(&d, q, k, v, g, beta, scale, len, h0, y, h1, ws, bytes, c.stream); });
    });
}

// dims, q, k, v, g, beta, scale, lengths, init_h, dy, d_final_h, dq, dk, dv, dg, dbeta, d_init_h, workspace
PyObject* delta_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, 18, [](PyObject* const* a) {
        const m3_dims d = dims_of(a[0]);
        const Call c(tensor_of(a[1]), io_of(d));
        const Sizes z(d, (int64_t)d.batch * d.seqlen);
        const void *q = c.arg(a[1], z.k), *k = c.arg(a[2], z.k), *v = c.arg(a[3], z.v), *dy = c.arg(a[9], z.v);
        const float *g = c.f32(a[4], z.g), *beta = c.f32(a[5], z.g), *h0 = c.f32(a[8], z.h), *dh = c.f32(a[10], z.h);
        const float scale = real(a[6]);
        const int* len = static_cast<const int*>(c.ptr(a[7], at::kInt, d.batch));
        void *dq = c.arg(a[11], z.k), *dk = c.arg(a[12], z.k), *dv = c.arg(a[13], z.v);
        void *dg = c.arg(a[14], z.g), *dbeta = c.arg(a[15], z.g);
        float* dh0 = c.f32(a[16], z.h);
        size_t bytes;
        void* ws = c.workspace(a[17], &bytes);
        return unlocked([&] {
            return p_delta_bwd(&d, q, k, v, g, beta, scale, len, h0, dy, dh, dq, dk, dv, dg, dbeta, dh0, ws, bytes, c.stream);
        });
    });
}

// x, eps, residual, weight, sum, y, y8, scale, scale_block
PyObject* rms_norm_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, 9, [](PyObject* const* a) {
        const at::Tensor& x = tensor_of(a[0]);
        const Call c(x, io_of(x));
        const int64_t cells = x.numel(), width = x.dim() ? x.size(-1) : 0;
        const long block = PyLong_AsLong(a[8]);
        if (width < 1 || width > INT_MAX || block < 0 || block > INT_MAX) throw Refuse();
        const int64_t rows = cells / width, blocks = block ? (width + block - 1) / block : 1;
        const float eps = real(a[1]);
        const void *px = c.arg(a[0], cells), *r = c.arg(a[2], cells);
        const float* w = c.f32(a[3], width);
        void *sum = c.arg(a[4], cells), *y = c.arg(a[5], cells), *y8 = c.ptr(a[6], at::kFloat8_e4m3fn, cells);
        float* scale = c.f32(a[7], rows * blocks);
        const int io = c.io == at::kBFloat16 ? M3_BF16 : M3_F32;
        return unlocked([&] { return p_norm_fwd(rows, (int)width, io, px, r, w, eps, sum, y, y8, scale, (int)block, c.stream); });
    });
}

// s, dy, eps, dx, workspace, weight, d_sum, dweight
PyObject* rms_norm_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded(args, n, 8, [](PyObject* const* a) {
        const at::Tensor& s = tensor_of(a[0]);
        const Call c(s, io_of(s));
        const int64_t cells = s.numel(), width = s.dim() ? s.size(-1) : 0;
        if (width < 1 || width > INT_MAX) throw Refuse();
        const void *ps = c.arg(a[0], cells), *dy = c.arg(a[1], cells), *ds = c.arg(a[6], cells);
        const float eps = real(a[2]);
        void* dx = c.arg(a[3], cells);
        size_t bytes;
        void* ws = c.workspace(a[4], &bytes);
        const float* w = c.f32(a[5], width);
        float* dw = c.f32(a[7], width);
        const int io = c.io == at::kBFloat16 ? M3_BF16 : M3_F32;
        return unlocked([&] { return p_norm_bwd(cells / width, (int)width, io, ps, w, eps, dy, ds, dx, dw, ws, bytes, c.stream); });
    });
}

// the addresses of the C entry points in the library that the package loaded
PyObject* bind(PyObject*, PyObject* args) {
    unsigned long long p[5];
    if (!PyArg_ParseTuple(args, "KKKKK", &p[0], &p[1], &p[2], &p[3], &p[4])) return nullptr;
    p_delta_step = reinterpret_cast<decltype(p_delta_step)>(p[0]);
    p_delta_fwd = reinterpret_cast<decltype(p_delta_fwd)>(p[1]);
    p_delta_bwd = reinterpret_cast<decltype(p_delta_bwd)>(p[2]);
    p_norm_fwd = reinterpret_cast<decltype(p_norm_fwd)>(p[3]);
    p_norm_bwd = reinterpret_cast<decltype(p_norm_bwd)>(p[4]);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"delta_step", fast(delta_step), METH_FASTCALL, nullptr},
                         {"delta_fwd", fast(delta_fwd), METH_FASTCALL, nullptr},
                         {"delta_bwd", fast(delta_bwd), METH_FASTCALL, nullptr},
                         {"rms_norm_fwd", fast(rms_norm_fwd), METH_FASTCALL, nullptr},
                         {"rms_norm_bwd", fast(rms_norm_bwd), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_m3_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__m3_call() {
    for (int i = 0; i < kFields; ++i)
        if (!(field_name[i] = PyUnicode_InternFromString(kFieldNames[i]))) return nullptr;
    return PyModule_Create(&module);
}
