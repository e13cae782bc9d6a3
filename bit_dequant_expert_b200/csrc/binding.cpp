// Python binding of the attention operators' C ABI: reads the tensors' fields
// directly, so that a call costs a few microseconds less on the host than the
// kernel of a decode step runs.  Argument marshalling only; the functions
// carry the C ABI's names and argument order and return its status.
//
// A pointer argument is a tensor, a raw integer address or None (NULL).  A
// tensor must be on the current CUDA device, of the type the call reads,
// contiguous (where the call takes a row stride: contiguous within each index
// of its first dimension) and hold all that the call may touch.  The stream is
// an integer, an object with a cuda_stream attribute, or None: torch's current
// stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>

#include "attn_b200.h"

namespace {

struct Fail {};   // a Python exception is set

struct Args {
    PyObject* const* a;
    Py_ssize_t n, i = 0;
    int device = -1;   // the current one, once a tensor is to be compared with it

    Args(PyObject* const* args, Py_ssize_t given, Py_ssize_t want) : a(args), n(given) {
        if (given != want) {
            PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", given, want);
            throw Fail{};
        }
    }
    PyObject* next() { return a[i++]; }

    int64_t i64() {
        const long long v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) throw Fail{};
        return v;
    }
    int32_t i32() {
        const int64_t v = i64();
        if (v < INT32_MIN || v > INT32_MAX) {
            PyErr_Format(PyExc_OverflowError, "%lld does not fit 32 bits", (long long)v);
            throw Fail{};
        }
        return (int32_t)v;
    }
    float f32() {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) throw Fail{};
        return (float)v;
    }
    const attn_config_t* config(attn_config_t& c) {
        Py_buffer view;
        if (PyObject_GetBuffer(next(), &view, PyBUF_SIMPLE)) throw Fail{};
        const bool ok = view.len == (Py_ssize_t)sizeof(c);
        if (ok) c = *static_cast<const attn_config_t*>(view.buf);
        PyBuffer_Release(&view);
        if (!ok) {
            PyErr_SetString(PyExc_TypeError, "cfg must be an attn_config_t");
            throw Fail{};
        }
        return &c;
    }
    // `need`: elements from the first on that the call may touch.
    template <typename T>
    T* ptr(const char* name, at::ScalarType kind, int64_t need, bool rows = false,
           at::ScalarType or_kind = at::ScalarType::Undefined) {
        return of<T>(next(), name, kind, need, rows, or_kind);
    }
    template <typename T>
    T* of(PyObject* o, const char* name, at::ScalarType kind, int64_t need, bool rows = false,
          at::ScalarType or_kind = at::ScalarType::Undefined) {
        if (o == Py_None) return nullptr;
        if (PyLong_CheckExact(o)) {
            void* p = PyLong_AsVoidPtr(o);
            if (!p && PyErr_Occurred()) throw Fail{};
            return static_cast<T*>(p);
        }
        if (!THPVariable_Check(o)) {
            PyErr_Format(PyExc_TypeError, "%s must be a tensor, an address or None", name);
            throw Fail{};
        }
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) {
            PyErr_Format(PyExc_ValueError, "%s is on %s, not on a GPU", name, t.device().str().c_str());
            throw Fail{};
        }
        if (device < 0) device = c10::cuda::current_device();
        if (t.device().index() != device) {
            PyErr_Format(PyExc_ValueError, "%s is on %s, not on the current device", name, t.device().str().c_str());
            throw Fail{};
        }
        if (t.scalar_type() != kind && t.scalar_type() != or_kind) {
            PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(kind), c10::toString(t.scalar_type()));
            throw Fail{};
        }
        if (!t.is_contiguous() && !(rows && rows_contiguous(t))) {
            PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
            throw Fail{};
        }
        const int64_t held = t.is_contiguous() || t.numel() == 0 ? t.numel() : (t.size(0) - 1) * t.stride(0) + t.numel() / t.size(0);
        if (held < need) {
            PyErr_Format(PyExc_ValueError, "%s holds %lld elements of the %lld that the call may touch", name, (long long)held,
                         (long long)need);
            throw Fail{};
        }
        return static_cast<T*>(t.data_ptr());
    }
    static bool rows_contiguous(const at::Tensor& t) {
        int64_t step = 1;
        for (int64_t d = t.dim() - 1; d > 0; --d) {
            if (t.size(d) != 1 && t.stride(d) != step) return false;
            step *= t.size(d);
        }
        return t.dim() > 0;
    }
    void* stream() {
        PyObject* o = next();
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
        PyObject* v = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        if (!v) throw Fail{};
        void* p = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        if (!p && PyErr_Occurred()) throw Fail{};
        return p;
    }
};

// Elements from the first to the last of n rows, `stride` apart.
int64_t span(int64_t n, int64_t stride, int64_t row) { return n > 0 ? (n - 1) * stride + row : 0; }

constexpr auto kBf16 = at::ScalarType::BFloat16;
constexpr auto kF32 = at::ScalarType::Float;
constexpr auto kI32 = at::ScalarType::Int;
constexpr auto kU8 = at::ScalarType::Byte;
constexpr auto kE4m3 = at::ScalarType::Float8_e4m3fn;

struct Cache {
    void *k, *v;
    float *ks, *vs;
    Cache(Args& a, const attn_config_t& c, int32_t pages, bool used = true) {
        const bool codes = c.cache_type == ATTN_CACHE_E4M3;   // codes may come as bytes
        const int64_t rows = used ? (int64_t)std::max(0, pages) * c.kv_heads * c.page_size : 0;
        k = a.ptr<void>("k_cache", codes ? kE4m3 : kBf16, rows * c.head_dim, false, codes ? kU8 : kBf16);
        v = a.ptr<void>("v_cache", codes ? kE4m3 : kBf16, rows * c.head_dim, false, codes ? kU8 : kBf16);
        ks = a.ptr<float>("k_scale", kF32, codes ? rows : 0);
        vs = a.ptr<float>("v_scale", kF32, codes ? rows : 0);
    }
};

// The call's status as a Python integer; nothing thrown leaves.
template <typename Call>
PyObject* guarded(Call call) {
    try {
        return PyLong_FromLongLong((long long)call());
    } catch (const Fail&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject* qkv_prepare(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a(args, n, 22);
        attn_config_t c;
        a.config(c);
        const int32_t T = a.i32();
        PyObject* qkv_arg = a.next();
        const int64_t stride = a.i64(), q_row = (int64_t)c.q_heads * c.head_dim, k_row = (int64_t)c.kv_heads * c.head_dim;
        const uint16_t* qkv = a.of<uint16_t>(qkv_arg, "qkv", kBf16, span(T, stride, q_row + 2 * k_row), true);
        const uint16_t* qw = a.ptr<uint16_t>("q_weight", kBf16, c.head_dim);
        const uint16_t* kw = a.ptr<uint16_t>("k_weight", kBf16, c.head_dim);
        const float eps = a.f32();
        PyObject* inv_arg = a.next();
        const int32_t rot = a.i32(), layout = a.i32();
        const float* inv = a.of<float>(inv_arg, "inv_freq", kF32, rot / 2);
        const float scale = a.f32();
        const int32_t* pos = a.ptr<int32_t>("positions", kI32, rot ? T : 0);
        const int32_t* slots = a.ptr<int32_t>("slots", kI32, T);
        const int32_t pages = a.i32();
        const Cache k(a, c, pages, slots != nullptr);
        uint16_t* q_out = a.ptr<uint16_t>("q_out", kBf16, T * q_row);
        uint16_t* k_out = a.ptr<uint16_t>("k_out", kBf16, T * k_row);
        int32_t* err = a.ptr<int32_t>("err", kI32, 1);
        void* stream = a.stream();
        return attn_qkv_prepare(&c, T, qkv, stride, qw, kw, eps, inv, rot, layout, scale, pos, slots, pages, k.k, k.v, k.ks,
                                k.vs, q_out, k_out, err, stream);
    });
}

PyObject* kv_read(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a(args, n, 15);
        attn_config_t c;
        a.config(c);
        const int32_t B = a.i32(), total = a.i32();
        PyObject* table_arg = a.next();
        const int64_t stride = a.i64(), row = (int64_t)c.kv_heads * c.head_dim;
        const int32_t* table = a.of<int32_t>(table_arg, "page_table", kI32, total > 0 ? B * stride : 0, true);
        const int32_t* cu = a.ptr<int32_t>("cu_lens", kI32, total > 0 ? (int64_t)B + 1 : 0);
        const int32_t pages = a.i32();
        const Cache k(a, c, pages, total > 0);
        uint16_t* k_out = a.ptr<uint16_t>("k_out", kBf16, total * row);
        uint16_t* v_out = a.ptr<uint16_t>("v_out", kBf16, total * row);
        int32_t* err = a.ptr<int32_t>("err", kI32, 1);
        void* stream = a.stream();
        return attn_kv_read(&c, B, total, table, stride, cu, pages, k.k, k.v, k.ks, k.vs, k_out, v_out, err, stream);
    });
}

PyObject* prefill(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a(args, n, 18);
        attn_config_t c;
        a.config(c);
        const int32_t B = a.i32(), total_q = a.i32(), total_k = a.i32();
        const int32_t* cu_q = a.ptr<int32_t>("cu_q", kI32, (int64_t)B + 1);
        const int32_t* cu_k = a.ptr<int32_t>("cu_k", kI32, (int64_t)B + 1);
        const int64_t q_row = (int64_t)c.q_heads * c.head_dim, k_row = (int64_t)c.kv_heads * c.head_dim;
        PyObject* q_arg = a.next();
        const int64_t qs = a.i64();
        PyObject* k_arg = a.next();
        const int64_t ks = a.i64();
        PyObject* v_arg = a.next();
        const int64_t vs = a.i64();
        const uint16_t* q = a.of<uint16_t>(q_arg, "q", kBf16, span(total_q, qs, q_row), true);
        const uint16_t* k = a.of<uint16_t>(k_arg, "k", kBf16, span(total_k, ks, k_row), true);
        const uint16_t* v = a.of<uint16_t>(v_arg, "v", kBf16, span(total_k, vs, k_row), true);
        const float scale = a.f32();
        const int32_t causal = a.i32();
        uint16_t* out = a.ptr<uint16_t>("out", kBf16, total_q * q_row);
        float* lse = a.ptr<float>("lse", kF32, (int64_t)total_q * c.q_heads);
        int32_t* err = a.ptr<int32_t>("err", kI32, 1);
        void* stream = a.stream();
        return attn_prefill(&c, B, total_q, total_k, cu_q, cu_k, q, qs, k, ks, v, vs, scale, causal, out, lse, err, stream);
    });
}

PyObject* decode_workspace_size(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a(args, n, 4);
        attn_config_t c;
        a.config(c);
        const int32_t B = a.i32(), nq = a.i32(), max_len = a.i32();
        return attn_decode_workspace_size(&c, B, nq, max_len);
    });
}

PyObject* decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&] {
        Args a(args, n, 21);
        attn_config_t c;
        a.config(c);
        const int32_t B = a.i32(), nq = a.i32(), max_len = a.i32();
        const int64_t rows = (int64_t)B * nq, q_row = (int64_t)c.q_heads * c.head_dim;
        PyObject* q_arg = a.next();
        const int64_t qs = a.i64();
        const uint16_t* q = a.of<uint16_t>(q_arg, "q", kBf16, span(rows, qs, q_row), true);
        PyObject* table_arg = a.next();
        const int64_t stride = a.i64(), need = c.page_size > 0 ? ((int64_t)max_len + c.page_size - 1) / c.page_size : 0;
        const int32_t* table = a.of<int32_t>(table_arg, "page_table", kI32, span(B, stride, need), true);
        const int32_t* lens = a.ptr<int32_t>("seq_lens", kI32, B);
        const int32_t pages = a.i32();
        const Cache k(a, c, pages);
        const float scale = a.f32();
        uint16_t* out = a.ptr<uint16_t>("out", kBf16, rows * q_row);
        float* lse = a.ptr<float>("lse", kF32, rows * c.q_heads);
        // the workspace's size comes with it unless it is given
        PyObject* w = a.a[a.i];
        void* ws = a.ptr<void>("ws", kU8, 0);
        PyObject* given = a.next();
        size_t bytes = 0;
        if (given != Py_None) {
            bytes = PyLong_AsSize_t(given);
            if (bytes == (size_t)-1 && PyErr_Occurred()) throw Fail{};
        } else if (THPVariable_Check(w)) {
            bytes = (size_t)THPVariable_Unpack(w).numel();
        }
        int32_t* err = a.ptr<int32_t>("err", kI32, 1);
        void* stream = a.stream();
        return attn_decode(&c, B, nq, max_len, q, qs, table, stride, lens, pages, k.k, k.v, k.ks, k.vs, scale, out, lse, ws,
                           bytes, err, stream);
    });
}

#define METHOD(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("attn_qkv_prepare", qkv_prepare),
                         METHOD("attn_kv_read", kv_read),
                         METHOD("attn_prefill", prefill),
                         METHOD("attn_decode_workspace_size", decode_workspace_size),
                         METHOD("attn_decode", decode),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_binding() { return PyModule_Create(&module); }
