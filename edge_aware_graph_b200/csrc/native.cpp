// Python entry of the operators around the block (_native): checks each call's
// tensors and passes their addresses and the stream on to libeaga.so.
//
// The same checks in Python took 10 us a call, more than the small operators
// run on the GPU; here a call costs its launch.  Each function takes the dims
// (a ctypes structure), the call's tensors in the C entry's order and the stream
// (None: the current one, a torch stream, or its handle as a number), and
// returns the C entry's status.  The structures have to be eaga.py's classes of
// them; what a tensor has to be is read from the dims:
// a contiguous CUDA tensor on the current device, of the dtype and the number of
// elements that the kernels will go by.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <climits>
#include <stdexcept>
#include <string>
#include "eaga.h"

namespace {

// A Python exception has been set.
struct Raised {};

[[noreturn]] void refuse(const std::string &what) {
    PyErr_SetString(PyExc_ValueError, what.c_str());
    throw Raised{};
}
std::string dtype_name(at::ScalarType t) { return std::string("torch.") + torch::getTHPDtype(t)->name; }

// The ctypes classes of the library's structures (eaga.py's, given once by bind()).
template <typename T>
struct Structure {
    static PyObject *type;
    static const char *const name;
};
template <typename T> PyObject *Structure<T>::type = nullptr;
template <> const char *const Structure<eaga_linear_dims>::name = "LinearDims";
template <> const char *const Structure<eaga_residual_norm_dims>::name = "ResidualNormDims";
template <> const char *const Structure<eaga_adamw_config>::name = "AdamwConfig";
template <> const char *const Structure<eaga_adamw_tensor>::name = "AdamwTensor";

// Whether `o` is one of `type` or a ctypes array of them.
bool is_structure(PyObject *o, PyObject *type) {
    if (!type) return false;
    if (PyObject_TypeCheck(o, reinterpret_cast<PyTypeObject *>(type))) return true;
    PyObject *of = PyObject_GetAttrString(reinterpret_cast<PyObject *>(Py_TYPE(o)), "_type_");
    PyErr_Clear();
    Py_XDECREF(of);
    return of == type;
}

struct Call {
    PyObject *const *args;
    Py_ssize_t n;
    Py_ssize_t at = 0;
    int dev = -2;
    at::ScalarType storage = at::kFloat;

    PyObject *next() {
        if (at >= n) throw std::runtime_error("too few arguments");
        return args[at++];
    }
    // The ctypes structure `T`, or an array of at least `count` of them.
    template <typename T>
    const T *structure(Py_ssize_t count = 1) {
        PyObject *o = next();
        if (!is_structure(o, Structure<T>::type)) refuse(std::string("a ") + Structure<T>::name + " is required (got " + Py_TYPE(o)->tp_name + ")");
        Py_buffer b;
        if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Raised{};
        const void *p = b.buf;
        const Py_ssize_t len = b.len;
        PyBuffer_Release(&b);                        // the argument keeps the memory
        // (a table of more entries than the library takes is refused there, unread)
        if (count > (1 << 20)) count = 1;
        if (len < (Py_ssize_t)sizeof(T) * count) refuse(std::string("a table of ") + std::to_string(count) + " " + Structure<T>::name + " is required");
        return static_cast<const T *>(p);
    }
    // The address of a tensor of `numel` elements (-1: any number); null for None where `optional`.
    void *tensor(const char *name, at::ScalarType dtype, long long numel, bool optional = false, size_t *bytes = nullptr) {
        PyObject *o = next();
        if (bytes) *bytes = 0;
        if (o == Py_None) {
            if (optional) return nullptr;
            refuse(std::string(name) + ": a tensor is required");
        }
        if (!THPVariable_Check(o)) refuse(std::string(name) + ": a tensor is required");
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) refuse(std::string(name) + ": a CUDA tensor is required (got " + t.device().str() + ")");
        if (dev == -2) dev = c10::cuda::current_device();
        if (t.device().index() != dev)
            refuse(std::string(name) + ": on " + t.device().str() + ", but the current device is cuda:" + std::to_string(dev));
        if (t.scalar_type() != dtype) refuse(std::string(name) + ": dtype " + dtype_name(t.scalar_type()) + ", expected " + dtype_name(dtype));
        if (numel >= 0 && t.numel() != numel)
            refuse(std::string(name) + ": " + std::to_string(t.numel()) + " elements, expected " + std::to_string(numel));
        if (!t.is_contiguous()) refuse(std::string(name) + ": must be contiguous");
        if (bytes) *bytes = t.nbytes();
        return t.data_ptr();
    }
    void *stored(const char *name, long long numel, bool optional = false) { return tensor(name, storage, numel, optional); }
    float *f32(const char *name, long long numel) { return static_cast<float *>(tensor(name, at::kFloat, numel, true)); }
    // A whole number that the library takes as an int.
    int number(const char *name) {
        const long long v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) throw Raised{};
        if (v < INT_MIN || v > INT_MAX) refuse(std::string(name) + ": " + std::to_string(v) + " is out of range");
        return (int)v;
    }
    void *stream() {
        PyObject *o = next();
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev >= 0 ? dev : c10::cuda::current_device()).stream();
        if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
        PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
        if (!h) throw Raised{};
        void *p = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (PyErr_Occurred()) throw Raised{};
        return p;
    }
};

template <typename F>
PyObject *guarded(PyObject *const *args, Py_ssize_t n, F &&f) {
    try {
        Call c{args, n};
        return PyLong_FromLong((long)f(c));
    } catch (const Raised &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

at::ScalarType storage_of(int dtype) { return dtype == EAGA_BF16 ? at::kBFloat16 : at::kFloat; }

PyObject *linear_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [](Call &c) {
        const auto *d = c.structure<eaga_linear_dims>();
        c.storage = storage_of(d->dtype);
        const long long in = d->in, out = d->out;
        size_t bytes;
        const void *X = c.stored("X", d->rows * in), *W = c.stored("W", in * out), *b = c.stored("b", out, true);
        const void *R = c.stored("R", d->rows * out, true);
        void *Y = c.stored("Y", d->rows * out), *Z = c.stored("Z", d->rows * out, true);
        void *ws = c.tensor("workspace", at::kByte, -1, false, &bytes);
        return eaga_linear_forward(d, X, W, b, R, Y, Z, ws, bytes, c.stream());
    });
}

PyObject *linear_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [](Call &c) {
        const auto *d = c.structure<eaga_linear_dims>();
        c.storage = storage_of(d->dtype);
        const long long ni = d->rows * (long long)d->in, no = d->rows * (long long)d->out, nw = (long long)d->in * d->out;
        size_t bytes;
        const void *X = c.stored("X", ni, true), *W = c.stored("W", nw, true), *Z = c.stored("Z", no, true), *dY = c.stored("dY", no);
        const int act_in = c.number("act_in");
        const void *Zin = c.stored("Zin", ni, true), *dR = c.stored("dR", ni, true);
        void *dX = c.stored("dX", ni, true);
        float *dW = c.f32("dW", nw), *db = c.f32("db", d->out);
        void *ws = c.tensor("workspace", at::kByte, -1, false, &bytes);
        return eaga_linear_backward(d, X, W, Z, dY, act_in, Zin, dR, dX, dW, db, ws, bytes, c.stream());
    });
}

PyObject *residual_norm_forward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [](Call &c) {
        const auto *d = c.structure<eaga_residual_norm_dims>();
        c.storage = storage_of(d->dtype);
        const long long w = d->w, nx = d->rows * w, ng = d->rows_per_group > 0 ? d->rows / d->rows_per_group * w : 0;
        const void *x = c.stored("x", nx, true), *u = c.stored("u", nx);
        const void *M = c.tensor("M", at::kByte, d->rows, true), *gate = c.stored("gate", ng, true);
        const void *post_g = c.stored("post_g", w, true), *post_s = c.stored("post_s", w, true);
        const void *pre_g = c.stored("pre_g", w, true), *pre_s = c.stored("pre_s", w, true);
        void *r = c.stored("r", nx, true), *h = c.stored("h", nx, true);
        return eaga_residual_norm_forward(d, x, u, static_cast<const uint8_t *>(M), gate, post_g, post_s, pre_g, pre_s, r, h, c.stream());
    });
}

PyObject *residual_norm_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [](Call &c) {
        const auto *d = c.structure<eaga_residual_norm_dims>();
        c.storage = storage_of(d->dtype);
        const long long w = d->w, nx = d->rows * w, ng = d->rows_per_group > 0 ? d->rows / d->rows_per_group * w : 0;
        size_t bytes;
        const void *r = c.stored("r", nx, true), *u = c.stored("u", nx, true);
        const void *M = c.tensor("M", at::kByte, d->rows, true), *gate = c.stored("gate", ng, true);
        const void *post_g = c.stored("post_g", w, true), *post_s = c.stored("post_s", w, true), *pre_g = c.stored("pre_g", w, true);
        const void *dr = c.stored("dr", nx, true), *dh = c.stored("dh", nx, true);
        void *dx = c.stored("dx", nx, true), *du = c.stored("du", nx, true), *dgate = c.stored("dgate", ng, true);
        float *dpost_g = c.f32("dpost_g", w), *dpost_s = c.f32("dpost_s", w), *dpre_g = c.f32("dpre_g", w), *dpre_s = c.f32("dpre_s", w);
        void *ws = c.tensor("workspace", at::kByte, -1, false, &bytes);
        return eaga_residual_norm_backward(d, r, u, static_cast<const uint8_t *>(M), gate, post_g, post_s, pre_g, dr, dh, dx, du, dgate,
                                           dpost_g, dpost_s, dpre_g, dpre_s, ws, bytes, c.stream());
    });
}

// config, table, count, state, lr, stream
PyObject *adamw_step(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [&](Call &c) {
        const auto *config = c.structure<eaga_adamw_config>();
        Call peek{args, n, 2};
        const int count = peek.number("count");
        const auto *table = c.structure<eaga_adamw_tensor>(count);
        c.number("count");
        void *state = c.tensor("state", at::kLong, 2);
        const float *lr = c.f32("lr", 1);
        return eaga_adamw_step(config, table, count, state, lr, c.stream());
    });
}

// table, count, stream
PyObject *adamw_unpack(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [&](Call &c) {
        Call peek{args, n, 1};
        const int count = peek.number("count");
        const auto *table = c.structure<eaga_adamw_tensor>(count);
        c.number("count");
        return eaga_adamw_unpack(table, count, c.stream());
    });
}

// LinearDims, ResidualNormDims, AdamwConfig, AdamwTensor
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    PyObject **const to[4] = {&Structure<eaga_linear_dims>::type, &Structure<eaga_residual_norm_dims>::type, &Structure<eaga_adamw_config>::type,
                              &Structure<eaga_adamw_tensor>::type};
    for (Py_ssize_t k = 0; k < 4; ++k) {
        if (n != 4 || !PyType_Check(args[k])) {
            PyErr_SetString(PyExc_TypeError, "four ctypes classes are required");
            return nullptr;
        }
    }
    for (int k = 0; k < 4; ++k) Py_XSETREF(*to[k], Py_NewRef(args[k]));
    Py_RETURN_NONE;
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(linear_forward), ENTRY(linear_backward), ENTRY(residual_norm_forward), ENTRY(residual_norm_backward),
                         ENTRY(adamw_step), ENTRY(adamw_unpack), ENTRY(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
