// Argument marshalling of the operators in mosaic_ops.h for Python: reads tensors through
// PyTorch's C++ interface, checks them, and calls the library. A decode step's kernels take 2
// to 10 us, and the same checks and copies written in Python with ctypes cost a call 6 to 12
// us of host time; here a whole call takes 3.5 to 5, launches included.
//
// The library's functions are bound by address (bind), so this module links to nothing of it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdio>
#include <stdexcept>
#include <string>

#include "mosaic_ops.h"

namespace {

struct Lib {
    decltype(&mq_gemv) gemv;
    decltype(&mq_qk_norm_rope) qk_norm_rope;
    decltype(&mq_kv_append) kv_append;
    decltype(&mq_qkv_append) qkv_append;
    decltype(&mq_kv_read) kv_read;
    decltype(&mq_kv_attention) kv_attention;
    decltype(&mq_status_string) status_string;
    decltype(&mq_gemv_workspace_bytes) gemv_workspace_bytes;
} lib;
PyObject* mosaic_error = nullptr;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

std::string shape_of(const at::Tensor& t) {
    std::string s = "shape (";
    for (int64_t v : t.sizes()) s += std::to_string(v) + ", ";
    s += "), strides (";
    for (int64_t v : t.strides()) s += std::to_string(v) + ", ";
    return s + "), " + c10::toString(t.scalar_type()) + " on " + t.device().str();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw Refused(std::string(what) + ": a tensor is wanted");
    return THPVariable_Unpack(o);
}

// What one call's operands share.
struct Common {
    at::ScalarType type;
    mq_dtype code;
    c10::DeviceIndex dev;
    explicit Common(const at::Tensor& t) : type(t.scalar_type()), dev(t.device().index()) {
        if (type != at::kBFloat16 && type != at::kHalf)
            throw Refused(std::string("bf16 or fp16 tensors are taken, not ") + c10::toString(type));
        if (!t.is_cuda()) throw Refused("libmosaic takes CUDA tensors only");
        code = type == at::kHalf ? MQ_F16 : MQ_BF16;
    }
};

bool on(const at::Tensor& t, c10::DeviceIndex dev) { return t.is_cuda() && t.device().index() == dev; }

// [T][heads][D] with adjacent elements; None: null.
struct Heads {
    mq_heads h;
    mq_heads* p = nullptr;
    Heads(PyObject* o, const char* what, const Common& c, int64_t T, int64_t D) {
        if (o == Py_None) return;
        const at::Tensor& t = tensor(o, what);
        if (t.dim() != 3 || t.size(0) != T || t.size(2) != D || (t.stride(2) != 1 && D > 1) || t.scalar_type() != c.type || !on(t, c.dev))
            throw Refused(std::string(what) + ": [" + std::to_string(T) + "][heads][" + std::to_string(D) + "] of " +
                          c10::toString(c.type) + " on cuda:" + std::to_string((int)c.dev) + " with adjacent elements is wanted, got " +
                          shape_of(t));
        h = mq_heads{t.data_ptr(), t.size(1), t.stride(0), t.stride(1)};
        p = &h;
    }
};

// A contiguous array of at least n elements; None: null.
template <typename P>
P* array(PyObject* o, const char* what, at::ScalarType type, int64_t n, c10::DeviceIndex dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, what);
    if (t.scalar_type() != type || !on(t, dev) || t.numel() < n || !t.is_contiguous())
        throw Refused(std::string(what) + ": " + std::to_string(n) + " contiguous " + c10::toString(type) + " values on cuda:" +
                      std::to_string((int)dev) + " are wanted, got " + shape_of(t));
    return static_cast<P*>(t.data_ptr());
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw std::bad_exception();
    return v;
}
// An integer that the library takes as int.
int integer32(PyObject* o) {
    const int64_t v = integer(o);
    if (v != (int)v) throw Refused("an integer argument is out of range");
    return (int)v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw std::bad_exception();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw std::bad_exception();
    return v != 0;
}
template <typename P>
P* pointer(PyObject* o) {
    return o == Py_None ? nullptr : reinterpret_cast<P*>(integer(o));
}
int extent(int64_t v) {
    if (v != (int)v) throw Refused("a tensor's extent is out of range");
    return (int)v;
}

// The call's stream (None: dev's current one), with dev current while it lives: a launch on
// another device's stream fails.
struct OnDevice {
    c10::DeviceIndex before;
    bool moved;
    void* stream;
    OnDevice(c10::DeviceIndex dev, PyObject* s) : before(c10::cuda::current_device()), moved(before != dev) {
        if (moved) c10::cuda::set_device(dev);
        stream = s == Py_None ? c10::cuda::getCurrentCUDAStream(dev).stream() : reinterpret_cast<void*>(integer(s));
    }
    ~OnDevice() {
        if (moved) c10::cuda::set_device(before);
    }
};

PyObject* done(mq_status st, const char* what) {
    if (st == MQ_OK) Py_RETURN_NONE;
    PyErr_Format(mosaic_error, "%s: %s (status %d)", what, lib.status_string(st), (int)st);
    return nullptr;
}

// No C++ exception leaves a call: it becomes a Python one.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
    try {
        if (n != want) throw Refused("wrong number of arguments");
        if (!lib.gemv) throw Refused("the library is not bound");
        return f();
    } catch (const Refused& e) {
        PyErr_SetString(mosaic_error ? mosaic_error : PyExc_RuntimeError, e.what());
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (X, Y, N, K, device, weight, residual, flags, stream, workspace)
PyObject* py_gemv(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor &X = tensor(a[0], "X"), &Y = tensor(a[1], "Y");
        const Common c(X);
        const int64_t N = integer(a[2]), K = integer(a[3]), dev = integer(a[4]);
        if (X.dim() != 2 || Y.dim() != 2 || X.size(1) != K || Y.size(1) != N || Y.size(0) != X.size(0) || X.stride(1) != 1 ||
            Y.stride(1) != 1 || Y.scalar_type() != c.type || !on(Y, c.dev) || dev != c.dev)
            throw Refused("X [M][" + std::to_string(K) + "] and Y [M][" + std::to_string(N) + "] of one 16-bit type on cuda:" +
                          std::to_string(dev) + " are wanted, got X " + shape_of(X) + ", Y " + shape_of(Y));
        OnDevice d(c.dev, a[8]);
        // no workspace given: one from the caching allocator, which hands it on in the stream's order
        at::Tensor ws;
        const size_t need = lib.gemv_workspace_bytes(extent(X.size(0)), (int)K);
        if (a[9] != Py_None) {
            array<void>(a[9], "ws", at::kByte, 0, c.dev);
            ws = tensor(a[9], "ws");
        } else if (need > 0) {
            c10::cuda::OptionalCUDAStreamGuard g;
            if (a[8] != Py_None) g.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(d.stream), c.dev));
            ws = at::empty({(int64_t)need}, X.options().dtype(at::kByte));
        }
        return done(lib.gemv(X.data_ptr(), c.code, X.stride(0), pointer<mq_nvfp4_mat>(a[5]), pointer<mq_residual_packed>(a[6]),
                             Y.data_ptr(), Y.stride(0), extent(X.size(0)), (int)N, (int)K, (unsigned)integer32(a[7]),
                             ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (size_t)ws.numel() : 0, d.stream),
                    "mq_gemv");
    });
}

struct Turn {
    const int64_t* pos = nullptr;
    const double* freq = nullptr;
    int rot = 0;
    Turn(PyObject* po, PyObject* fo, int64_t T, c10::DeviceIndex dev) {
        if (fo == Py_None) return;
        freq = array<double>(fo, "freq", at::kDouble, 1, dev);
        rot = extent(2 * tensor(fo, "freq").numel());
        pos = array<int64_t>(po, "pos", at::kLong, T, dev);
    }
};

// (q, k, q_out, k_out, pos, freq, q_weight, k_weight, eps, interleaved, stream)
PyObject* py_qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const at::Tensor& x = tensor(a[0] != Py_None ? a[0] : a[1], "q or k");
        const Common c(x);
        if (x.dim() != 3) throw Refused("[T][heads][D] is wanted, got " + shape_of(x));
        const int64_t T = x.size(0), D = x.size(2);
        Heads q(a[0], "q", c, T, D), k(a[1], "k", c, T, D), qo(a[2], "q_out", c, T, D), ko(a[3], "k_out", c, T, D);
        const Turn t(a[4], a[5], T, c.dev);
        const void *wq = array<void>(a[6], "q_weight", c.type, D, c.dev), *wk = array<void>(a[7], "k_weight", c.type, D, c.dev);
        OnDevice d(c.dev, a[10]);
        return done(lib.qk_norm_rope(q.p, k.p, qo.p, ko.p, extent(T), extent(D), c.code, wq, wk, (float)real(a[8]), t.pos, t.freq,
                                     t.rot, truth(a[9]), d.stream),
                    "mq_qk_norm_rope");
    });
}

// A KVCache's struct, its D and its device; they have to be the operands' too.
const mq_kv_cache* cache_of(PyObject* ptr, PyObject* dev, const Common& c) {
    if (integer(dev) != c.dev) throw Refused("the cache lies on another device than the operands");
    return pointer<mq_kv_cache>(ptr);
}

// (k, v, slots, cache, cache device, stream)
PyObject* py_kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor& x = tensor(a[0], "k");
        const Common c(x);
        const mq_kv_cache* kv = cache_of(a[3], a[4], c);
        const int64_t T = x.dim() == 3 ? x.size(0) : -1;
        Heads k(a[0], "k", c, T, kv->D), v(a[1], "v", c, T, kv->D);
        const int64_t* slots = array<int64_t>(a[2], "slots", at::kLong, T, c.dev);
        OnDevice d(c.dev, a[5]);
        return done(lib.kv_append(k.p, v.p, extent(T), c.code, slots, kv, d.stream), "mq_kv_append");
    });
}

// (q, k, v, q_out, k_out, pos, freq, q_weight, k_weight, eps, interleaved, slots, cache, cache device, stream)
PyObject* py_qkv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const at::Tensor& x = tensor(a[0], "q");
        const Common c(x);
        const mq_kv_cache* kv = cache_of(a[12], a[13], c);
        const int64_t T = x.dim() == 3 ? x.size(0) : -1, D = kv->D;
        Heads q(a[0], "q", c, T, D), k(a[1], "k", c, T, D), v(a[2], "v", c, T, D), qo(a[3], "q_out", c, T, D), ko(a[4], "k_out", c, T, D);
        const Turn t(a[5], a[6], T, c.dev);
        const void *wq = array<void>(a[7], "q_weight", c.type, D, c.dev), *wk = array<void>(a[8], "k_weight", c.type, D, c.dev);
        const int64_t* slots = array<int64_t>(a[11], "slots", at::kLong, T, c.dev);
        OnDevice d(c.dev, a[14]);
        return done(lib.qkv_append(q.p, k.p, v.p, qo.p, ko.p, extent(T), c.code, wq, wk, (float)real(a[9]), t.pos, t.freq, t.rot,
                                   truth(a[10]), slots, kv, d.stream),
                    "mq_qkv_append");
    });
}

// (cache, cache device, slots, k, v, stream)
PyObject* py_kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor& x = tensor(a[3], "k");
        const Common c(x);
        const mq_kv_cache* kv = cache_of(a[0], a[1], c);
        const int64_t T = x.dim() == 3 ? x.size(0) : -1;
        Heads k(a[3], "k", c, T, kv->D), v(a[4], "v", c, T, kv->D);
        const int64_t* slots = array<int64_t>(a[2], "slots", at::kLong, T, c.dev);
        OnDevice d(c.dev, a[5]);
        return done(lib.kv_read(kv, slots, extent(T), k.p, v.p, c.code, d.stream), "mq_kv_read");
    });
}

// (q, cache, cache device, block_table, kv_len, out, scale, cu_q, max_q, window, lse, ws, stream)
PyObject* py_kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        const at::Tensor &x = tensor(a[0], "q"), &table = tensor(a[3], "block_table"), &len = tensor(a[4], "kv_len");
        const Common c(x);
        const mq_kv_cache* kv = cache_of(a[1], a[2], c);
        const int64_t T = x.dim() == 3 ? x.size(0) : -1, B = len.numel();
        Heads q(a[0], "q", c, T, kv->D), o(a[5], "out", c, T, kv->D);
        const int32_t* kv_len = array<int32_t>(a[4], "kv_len", at::kInt, B, c.dev);
        if (table.dim() != 2 || table.scalar_type() != at::kInt || !on(table, c.dev) || table.size(0) < B ||
            (table.stride(1) != 1 && table.size(1) > 1))
            throw Refused("block_table: int32 [" + std::to_string(B) + "][pages] on cuda:" + std::to_string((int)c.dev) +
                          " is wanted, got " + shape_of(table));
        const int32_t* cu = array<int32_t>(a[7], "cu_q", at::kInt, B + 1, c.dev);
        float* lse = array<float>(a[10], "lse", at::kFloat, T * x.size(1), c.dev);
        void* ws = array<void>(a[11], "ws", at::kByte, 0, c.dev);
        const size_t ws_bytes = a[11] == Py_None ? 0 : (size_t)tensor(a[11], "ws").numel();
        OnDevice d(c.dev, a[12]);
        return done(lib.kv_attention(q.p, o.p, lse, extent(T), c.code, kv, static_cast<const int32_t*>(table.data_ptr()), table.stride(0),
                                     extent(table.size(1)), extent(B), cu, integer32(a[8]), kv_len, (float)real(a[6]), integer32(a[9]),
                                     ws, ws_bytes, d.stream),
                    "mq_kv_attention");
    });
}

// (error class, addresses of the eight functions in Lib's order)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 9) {
        PyErr_SetString(PyExc_TypeError, "bind: an error class and eight addresses");
        return nullptr;
    }
    void* at[8];
    for (int i = 0; i < 8; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (!at[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return nullptr;
        }
    }
    Py_INCREF(a[0]);
    Py_XDECREF(mosaic_error);
    mosaic_error = a[0];
    lib.gemv = reinterpret_cast<decltype(lib.gemv)>(at[0]);
    lib.qk_norm_rope = reinterpret_cast<decltype(lib.qk_norm_rope)>(at[1]);
    lib.kv_append = reinterpret_cast<decltype(lib.kv_append)>(at[2]);
    lib.qkv_append = reinterpret_cast<decltype(lib.qkv_append)>(at[3]);
    lib.kv_read = reinterpret_cast<decltype(lib.kv_read)>(at[4]);
    lib.kv_attention = reinterpret_cast<decltype(lib.kv_attention)>(at[5]);
    lib.status_string = reinterpret_cast<decltype(lib.status_string)>(at[6]);
    lib.gemv_workspace_bytes = reinterpret_cast<decltype(lib.gemv_workspace_bytes)>(at[7]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<py_bind>("bind"),           method<py_gemv>("gemv"),
                         method<py_qk_norm_rope>("qk_norm_rope"), method<py_kv_append>("kv_append"),
                         method<py_qkv_append>("qkv_append"),     method<py_kv_read>("kv_read"),
                         method<py_kv_attention>("kv_attention"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Operand checks and calls of libmosaic's operators.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
