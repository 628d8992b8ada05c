// The quick way from torch tensors to the latent-attention entry points: a
// CPython module whose functions take the arguments of the Python ones, check
// types, shapes, layouts and devices, and call the library.  A kernel of a few
// microseconds waits on its caller otherwise: a call of nine tensors spends
// about 5 us on the same checks in Python and 2 us in ctypes.
//
// A function returns the entry point's code, or 1 when anything does not fit,
// whereupon the Python function finds out what and says so.  Nothing else
// launches these kernels for Python: no call goes round these checks.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "coli_mla.h"

namespace {

struct Misfit {};

// The arguments of a call; every tensor has to be on the first one's device.
struct Args {
    PyObject *const *v;
    int64_t device = -1;

    bool none(int i) const { return v[i] == Py_None; }
    const at::Tensor &tensor(int i) {
        if (!THPVariable_Check(v[i])) throw Misfit();
        const at::Tensor &t = THPVariable_Unpack(v[i]);
        if (!t.is_cuda()) throw Misfit();
        if (device < 0) device = t.device().index();
        if (t.device().index() != device) throw Misfit();
        return t;
    }
    const at::Tensor &of(int i, at::ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor &t = tensor(i);
        if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape)) throw Misfit();
        return t;
    }
    void *dense(int i, at::ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor &t = of(i, type, shape);
        if (!t.is_contiguous()) throw Misfit();
        return t.data_ptr();
    }
    // the same, or null for None
    void *dense_or_none(int i, at::ScalarType type, std::initializer_list<int64_t> shape) {
        return none(i) ? nullptr : dense(i, type, shape);
    }
    struct View {
        void *at = nullptr;
        int64_t token = 0, head = 0;
    };
    View view(int i, at::ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor &t = of(i, type, shape);
        if (t.stride(2) != 1) throw Misfit();
        // the stride of a dimension of one element is never used
        return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
    }
    int64_t size(int i, int64_t dim, int64_t dims) {
        const at::Tensor &t = tensor(i);
        if (t.dim() != dims) throw Misfit();
        return t.size(dim);
    }
    int64_t number(int i) {
        const int64_t n = PyLong_AsLongLong(v[i]);
        if (n == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            throw Misfit();
        }
        if (n > INT32_MAX || n < INT32_MIN) throw Misfit();
        return n;
    }
    // a raw stream handle, or None for the device's current stream
    void *stream(int i) {
        if (!none(i)) {
            const size_t handle = PyLong_AsSize_t(v[i]);
            if (handle == (size_t)-1 && PyErr_Occurred()) throw Misfit();
            return reinterpret_cast<void *>(handle);
        }
        return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
    }
};

at::ScalarType type_of(const coli_mla_dims *d) { return d->dtype == COLI_BF16 ? at::kBFloat16 : at::kHalf; }

struct Cache {
    void *pages;
    float *scale;
    int64_t n;
};
Cache cache(Args &a, const coli_mla_dims *d, int pages, int scale) {
    const bool codes = d->kv_format == COLI_KV_E4M3;
    const int64_t n = a.size(pages, 0, 3);
    if (n > INT32_MAX) throw Misfit();
    return {a.dense(pages, codes ? at::kByte : type_of(d), {n, d->page_size, d->rank + (codes ? 2 : 1) * COLI_MLA_ROPE}),
            static_cast<float *>(a.dense_or_none(scale, at::kFloat, {n * d->page_size})), n};
}

// Runs f on the arguments (the first of them the address of the dims, except
// for project) with the tensors' device current.
template <int N, class F>
PyObject *call(PyObject *const *v, Py_ssize_t n, F f) {
    if (n != N) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    long rc = 1;
    try {
        Args a{v};
        rc = f(a, reinterpret_cast<const coli_mla_dims *>(N == 4 ? 0 : PyLong_AsSize_t(v[0])));
    } catch (const Misfit &) {
    } catch (const std::exception &) {
    }
    if (PyErr_Occurred()) PyErr_Clear();
    return PyLong_FromLong(rc);
}

// No two of `outer` x `inner` runs of 64 elements at these strides share an
// element, the inner ones lying between two outer ones.
bool apart(int64_t outer, int64_t outer_stride, int64_t inner, int64_t inner_stride) {
    return (inner == 1 || inner_stride >= COLI_MLA_ROPE) &&
           (outer == 1 || outer_stride >= (inner - 1) * inner_stride + COLI_MLA_ROPE);
}

at::Device device_of(const Args &a) { return at::Device(at::kCUDA, (c10::DeviceIndex)a.device); }

// dims, kv_a, norm_w, positions, slots, inv_freq, q_pe, q_pe_out, pages, kv_scale, ws, stream
PyObject *append(PyObject *, PyObject *const *v, Py_ssize_t n) {
    return call<12>(v, n, [](Args &a, const coli_mla_dims *d) -> long {
        const at::ScalarType t = type_of(d);
        const int64_t tokens = a.size(1, 0, 2);
        if (tokens > INT32_MAX) throw Misfit();
        void *kv_a = a.dense(1, t, {tokens, d->rank + COLI_MLA_ROPE}), *norm_w = a.dense_or_none(2, t, {d->rank});
        void *positions = a.dense(3, at::kInt, {tokens}), *slots = a.dense(4, at::kLong, {tokens});
        void *freq = a.dense(5, at::kDouble, {COLI_MLA_ROPE / 2});
        Args::View q, o;
        if (!a.none(6)) q = a.view(6, t, {tokens, d->n_heads, COLI_MLA_ROPE});
        if (!a.none(7)) {
            o = a.view(7, t, {tokens, d->n_heads, COLI_MLA_ROPE});
            if (tokens > 0 && !apart(tokens, o.token, d->n_heads, o.head) && !apart(d->n_heads, o.head, tokens, o.token))
                throw Misfit();
        }
        const Cache c = cache(a, d, 8, 9);
        const int64_t ws = a.size(10, 0, 1);
        void *w = a.dense(10, at::kByte, {ws});
        const c10::DeviceGuard guard(device_of(a));
        return coli_mla_append(d, (int32_t)tokens, kv_a, norm_w, static_cast<int32_t *>(positions), static_cast<int64_t *>(slots),
                               static_cast<double *>(freq), q.at, q.token, q.head, o.at, o.token, o.head, c.pages, c.scale,
                               (int32_t)c.n, w, (size_t)ws, a.stream(11));
    });
}

// x, w, out, stream
PyObject *project(PyObject *, PyObject *const *v, Py_ssize_t n) {
    return call<4>(v, n, [](Args &a, const coli_mla_dims *) -> long {
        const at::ScalarType t = a.tensor(0).scalar_type();
        if (t != at::kBFloat16 && t != at::kHalf) throw Misfit();
        const int64_t tokens = a.size(0, 0, 3), heads = a.size(0, 1, 3), n_in = a.size(0, 2, 3), n_out = a.size(1, 1, 3);
        if (tokens > INT32_MAX || heads > INT32_MAX || n_in > INT32_MAX || n_out > INT32_MAX) throw Misfit();
        const Args::View x = a.view(0, t, {tokens, heads, n_in});
        void *w = a.dense(1, t, {heads, n_out, n_in}), *out = a.dense(2, t, {tokens, heads, n_out});
        const c10::DeviceGuard guard(device_of(a));
        return coli_mla_project(t == at::kBFloat16 ? COLI_BF16 : COLI_FP16, (int32_t)tokens, (int32_t)heads, (int32_t)n_in,
                                (int32_t)n_out, x.at, x.token, x.head, w, out, a.stream(3));
    });
}

// dims, q_lat, q_pe, pages, kv_scale, table, kv_lens, max_kv, out, lse, ws, stream
PyObject *decode(PyObject *, PyObject *const *v, Py_ssize_t n) {
    return call<12>(v, n, [](Args &a, const coli_mla_dims *d) -> long {
        const at::ScalarType t = type_of(d);
        const int64_t rows = a.size(1, 0, 3), batch = a.size(6, 0, 1), width = a.size(5, 1, 2);
        if ((batch > 0 && (rows < 1 || rows % batch)) || rows > INT32_MAX || batch > INT32_MAX || width > INT32_MAX) throw Misfit();
        void *q_lat = a.dense(1, t, {rows, d->n_heads, d->rank}), *q_pe = a.dense(2, t, {rows, d->n_heads, COLI_MLA_ROPE});
        const Cache c = cache(a, d, 3, 4);
        void *table = a.dense(5, at::kInt, {batch, width}), *lens = a.dense(6, at::kInt, {batch});
        const int64_t max_kv = a.number(7);
        void *out = a.dense(8, t, {rows, d->n_heads, d->rank}), *lse = a.dense_or_none(9, at::kFloat, {rows, d->n_heads});
        const int64_t ws = a.size(10, 0, 1);
        void *w = a.dense(10, at::kByte, {ws});
        const c10::DeviceGuard guard(device_of(a));
        return coli_mla_decode(d, (int32_t)batch, batch ? (int32_t)(rows / batch) : 1, q_lat, q_pe, c.pages, c.scale, (int32_t)c.n,
                               static_cast<int32_t *>(table), (int32_t)width, static_cast<int32_t *>(lens), (int32_t)max_kv, out,
                               static_cast<float *>(lse), w, (size_t)ws, a.stream(11));
    });
}

// dims, pages, kv_scale, table, cu_k, w, kv, k_pe, ws, stream
PyObject *expand(PyObject *, PyObject *const *v, Py_ssize_t n) {
    return call<10>(v, n, [](Args &a, const coli_mla_dims *d) -> long {
        const at::ScalarType t = type_of(d);
        const int64_t rows = a.size(6, 0, 3), batch = a.size(4, 0, 1) - 1, width = a.size(3, 1, 2), wide = d->nope + d->v_dim;
        if (batch < 0 || batch > INT32_MAX || rows > INT32_MAX || width > INT32_MAX) throw Misfit();
        const Cache c = cache(a, d, 1, 2);
        void *table = a.dense(3, at::kInt, {batch, width}), *cu = a.dense(4, at::kInt, {batch + 1});
        void *w = a.dense(5, t, {d->n_heads, d->nope + d->v_dim, d->rank}), *kv = a.dense(6, t, {rows, d->n_heads, wide});
        void *k_pe = a.dense(7, t, {rows, COLI_MLA_ROPE});
        const int64_t ws = a.size(8, 0, 1);
        void *space = a.dense(8, at::kByte, {ws});
        const c10::DeviceGuard guard(device_of(a));
        return coli_mla_expand(d, (int32_t)batch, (int32_t)rows, c.pages, c.scale, (int32_t)c.n, static_cast<int32_t *>(table),
                               (int32_t)width, static_cast<int32_t *>(cu), w, kv, k_pe, space, (size_t)ws, a.stream(9));
    });
}

// dims, q, k_nope, k_pe, v, cu_q, cu_k, max_q, causal, out, lse, ws, stream
PyObject *prefill(PyObject *, PyObject *const *v, Py_ssize_t n) {
    return call<13>(v, n, [](Args &a, const coli_mla_dims *d) -> long {
        const at::ScalarType t = type_of(d);
        const int64_t rows = a.size(1, 0, 3), keys = a.size(2, 0, 3), batch = a.size(5, 0, 1) - 1;
        if (batch < 0 || batch > INT32_MAX || rows > INT32_MAX || keys > INT32_MAX) throw Misfit();
        const Args::View q = a.view(1, t, {rows, d->n_heads, d->nope + COLI_MLA_ROPE});
        const Args::View k = a.view(2, t, {keys, d->n_heads, d->nope});
        void *k_pe = a.dense(3, t, {keys, COLI_MLA_ROPE});
        const Args::View val = a.view(4, t, {keys, d->n_heads, d->v_dim});
        void *cu_q = a.dense(5, at::kInt, {batch + 1}), *cu_k = a.dense(6, at::kInt, {batch + 1});
        const int64_t max_q = a.number(7);
        const int causal = PyObject_IsTrue(a.v[8]);
        if (causal < 0) throw Misfit();
        void *out = a.dense(9, t, {rows, d->n_heads, d->v_dim}), *lse = a.dense_or_none(10, at::kFloat, {rows, d->n_heads});
        const int64_t ws = a.size(11, 0, 1);
        void *w = a.dense(11, at::kByte, {ws});
        const c10::DeviceGuard guard(device_of(a));
        return coli_mla_prefill(d, (int32_t)batch, (int32_t)rows, (int32_t)keys, q.at, q.token, q.head, k.at, k.token, k.head, k_pe,
                                val.at, val.token, val.head, static_cast<int32_t *>(cu_q), static_cast<int32_t *>(cu_k),
                                (int32_t)max_q, causal, out, static_cast<float *>(lse), w, (size_t)ws, a.stream(12));
    });
}

PyMethodDef methods[] = {{"append", (PyCFunction)(void (*)())append, METH_FASTCALL, nullptr},
                         {"project", (PyCFunction)(void (*)())project, METH_FASTCALL, nullptr},
                         {"decode", (PyCFunction)(void (*)())decode, METH_FASTCALL, nullptr},
                         {"expand", (PyCFunction)(void (*)())expand, METH_FASTCALL, nullptr},
                         {"prefill", (PyCFunction)(void (*)())prefill, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mla_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mla_bind(void) { return PyModule_Create(&module); }
