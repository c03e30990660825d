// Marshalling of the serving calls from torch tensors in C++ (module _host).
//
// A step of a server is a row of small calls, and reading a tensor's type, place, shape and strides from Python
// costs 0.06 us a look, so a call's checks (some forty looks) cost as much as its kernel.  These functions take
// the regular call: tensors of exactly the type, shape and strides that the kernels read, on the current
// device.  They launch it and return what the Python function returns; or the library's status, an int, if it
// refused; or None for a call that is not regular: nothing has been launched then, and the Python function copies what
// has to be dense or says what is wrong.  us of the host, launch included, here and in Python: an attention call over
// a tree of 13 nodes 3.7 and 8.3; rules on 8 rows of logits 3.9 and 8.2; two caches' append, move and read-out 23
// and 43; adapters added to 61 rows 6.6 and 10.5.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <vector>

#include "../../include/q4gsw.h"

namespace {

// The library's functions, from the handle that the binding has opened.
#define Q4GSW_CALLS(X)                                                                                      \
    X(kv_append) X(kv_read) X(kv_attention_ex) X(kv_attention_workspace_bytes) X(kv_tree_attention_ex)       \
    X(kv_tree_attention_workspace_bytes) X(kv_keep) X(logits_adjust) X(adapters_add) X(adapters_fwd)         \
    X(adapters_workspace_bytes)
struct Library {
#define Q4GSW_MEMBER(f) decltype(&q4gsw_##f) f = nullptr;
    Q4GSW_CALLS(Q4GSW_MEMBER)
#undef Q4GSW_MEMBER
} lib;
PyObject *get_device = nullptr, *get_stream = nullptr;

// A call that is not regular.
struct Irregular {};
void need(bool ok) {
    if (!ok) throw Irregular{};
}

int64_t integer(PyObject* o, int64_t lo, int64_t hi) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Irregular{};
    }
    need(v >= lo && v <= hi);
    return v;
}
int32_t int32(PyObject* o) { return (int32_t)integer(o, 0, 0x7fffffff); }

template <class S>
S* address(PyObject* o) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p) {
        PyErr_Clear();
        throw Irregular{};
    }
    return static_cast<S*>(p);
}

// A strided tensor on GPU `dev`, of plain torch.Tensor's own class.
const at::Tensor& tensor(PyObject* o, int dev) {
    need(THPVariable_CheckExact(o));
    const at::Tensor& t = THPVariable_Unpack(o);
    need(t.defined() && t.device().type() == at::kCUDA && t.device().index() == dev && t.layout() == at::kStrided);
    return t;
}
template <class T>
T* dense(PyObject* o, int dev, at::ScalarType type, int64_t n) {
    const at::Tensor& t = tensor(o, dev);
    need(t.scalar_type() == type && t.dim() == 1 && t.size(0) == n && t.is_contiguous());
    return static_cast<T*>(t.data_ptr());
}
template <class T>
T* dense_or_null(PyObject* o, int dev, at::ScalarType type, int64_t n) {
    return o == Py_None ? nullptr : dense<T>(o, dev, type, n);
}
// A [rows, columns] tensor of dense rows that do not overlap.
template <class T>
T* table(PyObject* o, int dev, at::ScalarType type, int64_t rows, int64_t* ld, int64_t* cols) {
    const at::Tensor& t = tensor(o, dev);
    need(t.scalar_type() == type && t.dim() == 2 && t.size(0) == rows);
    *cols = t.size(1);
    *ld = rows <= 1 ? *cols : t.stride(0);
    need((*cols <= 1 || t.stride(1) == 1) && *ld >= *cols);
    return static_cast<T*>(t.data_ptr());
}
int32_t dtype_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat: return Q4GSW_F32;
        case at::kHalf: return Q4GSW_F16;
        case at::kBFloat16: return Q4GSW_BF16;
        default: throw Irregular{};
    }
}
// Token rows [tokens, heads, dim] that the kernels take as they are.
const void* token_rows(const at::Tensor& t, int64_t heads, int64_t dim, int64_t* ld) {
    need(t.dim() == 3 && t.size(1) == heads && t.size(2) == dim);
    *ld = t.size(0) <= 1 ? heads * dim : t.stride(0);
    void* p = t.data_ptr();
    need(t.stride(2) == 1 && (heads == 1 || t.stride(1) == dim) && *ld >= heads * dim);
    need(((reinterpret_cast<uintptr_t>(p) | (uint64_t)*ld * t.element_size()) & 15u) == 0);
    return p;
}

// table, cu, lens of a call with `tokens` token rows; returns the batch.
int64_t sequences(PyObject* const* args, int dev, int64_t tokens, q4gsw_kv_seqs* s) {
    const at::Tensor& lens = tensor(args[2], dev);
    need(lens.dim() == 1 && lens.size(0) >= 1 && lens.size(0) <= 0x7fffffff);
    const int64_t n = lens.size(0);
    int64_t ld = 0, cols = 0;
    s->table = table<int32_t>(args[0], dev, at::kInt, n, &ld, &cols);
    need(cols <= 0x7fffffff);
    s->table_ld = ld;
    s->table_cols = (int32_t)cols;
    s->batch = (int32_t)n;
    s->cu = dense<int32_t>(args[1], dev, at::kInt, n + 1);
    s->lens = dense<int32_t>(args[2], dev, at::kInt, n);
    s->tokens = tokens;
    return n;
}

// The current stream of the current device, which has to be `dev`.
void* stream(int dev) {
    PyObject* d = PyObject_CallNoArgs(get_device);
    const bool here = d && PyLong_AsLong(d) == dev;
    PyObject* s = here ? PyObject_CallOneArg(get_stream, d) : nullptr;
    Py_XDECREF(d);
    void* p = s ? PyLong_AsVoidPtr(s) : nullptr;
    const bool ok = s && !PyErr_Occurred();
    Py_XDECREF(s);
    PyErr_Clear();
    need(ok);
    return p;
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
}
// The caller's workspace, or a new one.
at::Tensor bytes_of(PyObject* o, int dev, uint64_t bytes) {
    if (o == Py_None) return fresh({(int64_t)bytes}, at::kByte, dev);
    const at::Tensor& t = tensor(o, dev);
    need(t.scalar_type() == at::kByte && t.is_contiguous());
    return t;
}

template <class F>
int status_of(F&& f) {
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = (int)f();
    Py_END_ALLOW_THREADS;
    return st;
}
PyObject* result(int status, PyObject* (*wrap)(const at::Tensor&), const at::Tensor& t) {
    return status ? PyLong_FromLong(status) : wrap(t);
}
PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

template <class F>
PyObject* regular(Py_ssize_t n, Py_ssize_t want, F&& f) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Irregular&) {
        Py_RETURN_NONE;
    } catch (const std::exception&) {                         // an allocation that failed: before any launch
        if (PyErr_Occurred()) return nullptr;
        Py_RETURN_NONE;
    }
}

// (cache, device, q, parents or None, table, cu, lens, max_new, max_ctx, window, softcap, out or None, workspace or None)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return regular(n, 13, [&]() -> PyObject* {
        const q4gsw_kv_cache* c = address<const q4gsw_kv_cache>(a[0]);
        const int dev = int32(a[1]);
        const at::Tensor& q = tensor(a[2], dev);
        need(q.dim() == 3 && q.size(1) <= 0x7fffffff);
        const int32_t dt = dtype_of(q), hq = (int32_t)q.size(1);
        const int64_t tokens = q.size(0);
        int64_t ld = 0;
        const void* qp = token_rows(q, hq, c->dim, &ld);
        q4gsw_kv_seqs s{};
        const int64_t batch = sequences(a + 4, dev, tokens, &s);
        const bool tree = a[3] != Py_None;
        const int32_t* parents = tree ? dense<int32_t>(a[3], dev, at::kInt, tokens) : nullptr;
        const int32_t max_new = int32(a[7]), max_ctx = int32(a[8]), window = int32(a[9]);
        const double cap = PyFloat_AsDouble(a[10]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            throw Irregular{};
        }
        void* st = stream(dev);
        at::Tensor out = a[11] == Py_None ? fresh({tokens, hq, c->dim}, q.scalar_type(), dev) : tensor(a[11], dev);
        need(out.scalar_type() == q.scalar_type() && out.dim() == 3 && out.size(0) == tokens && out.size(1) == hq &&
             out.size(2) == c->dim && out.is_contiguous());
        uint64_t bytes = 0;
        if (a[12] == Py_None) {
            const int e = tree ? lib.kv_tree_attention_workspace_bytes(c, (int32_t)batch, tokens, hq, max_new, max_ctx, &bytes)
                               : lib.kv_attention_workspace_bytes(c, (int32_t)batch, tokens, hq, max_new, max_ctx, &bytes);
            need(e == Q4GSW_OK);
        }
        const at::Tensor ws = bytes_of(a[12], dev, bytes);
        void *op = out.data_ptr(), *wp = ws.data_ptr();
        const uint64_t wb = (uint64_t)ws.numel();
        const int e = status_of([&] {
            return tree ? lib.kv_tree_attention_ex(c, &s, parents, qp, ld, dt, hq, max_new, max_ctx, window, (float)cap, op, wp, wb, nullptr, st)
                        : lib.kv_attention_ex(c, &s, qp, ld, dt, hq, max_new, max_ctx, window, (float)cap, op, wp, wb, nullptr, st);
        });
        return result(e, wrap, out);
    });
}

// (cache, device, k, v, table, cu, lens): the status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return regular(n, 7, [&]() -> PyObject* {
        const q4gsw_kv_cache* c = address<const q4gsw_kv_cache>(a[0]);
        const int dev = int32(a[1]);
        const at::Tensor &k = tensor(a[2], dev), &v = tensor(a[3], dev);
        const int32_t dt = dtype_of(k);
        int64_t k_ld = 0, v_ld = 0;
        const void *kp = token_rows(k, c->heads, c->dim, &k_ld), *vp = token_rows(v, c->heads, c->dim, &v_ld);
        need(v.scalar_type() == k.scalar_type() && v.size(0) == k.size(0));
        q4gsw_kv_seqs s{};
        sequences(a + 4, dev, k.size(0), &s);
        void* st = stream(dev);
        return PyLong_FromLong(status_of([&] { return lib.kv_append(c, &s, kp, k_ld, vp, v_ld, dt, st); }));
    });
}

// (cache, device, table, cu, lens, tokens): (k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return regular(n, 6, [&]() -> PyObject* {
        const q4gsw_kv_cache* c = address<const q4gsw_kv_cache>(a[0]);
        const int dev = int32(a[1]);
        const int64_t tokens = int32(a[5]);
        q4gsw_kv_seqs s{};
        sequences(a + 2, dev, tokens, &s);
        void* st = stream(dev);
        const at::Tensor k = fresh({tokens, c->heads, c->dim}, at::kFloat, dev), v = fresh({tokens, c->heads, c->dim}, at::kFloat, dev);
        float *kp = k.data_ptr<float>(), *vp = v.data_ptr<float>();
        const int e = status_of([&] { return lib.kv_read(c, &s, kp, vp, st); });
        return e ? PyLong_FromLong(e) : Py_BuildValue("(NN)", wrap(k), wrap(v));
    });
}

// (addresses of the caches, device, parents, leaf, table, cu, lens, max_new, kept or None, path or None): (kept, path)
PyObject* keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return regular(n, 10, [&]() -> PyObject* {
        need(PyList_CheckExact(a[0]) && PyList_GET_SIZE(a[0]) >= 1 && PyList_GET_SIZE(a[0]) <= 128);
        const int32_t count = (int32_t)PyList_GET_SIZE(a[0]);
        q4gsw_kv_cache caches[128];
        for (int32_t i = 0; i < count; ++i) caches[i] = *address<const q4gsw_kv_cache>(PyList_GET_ITEM(a[0], i));
        const int dev = int32(a[1]);
        const at::Tensor& up = tensor(a[2], dev);
        need(up.dim() == 1);
        const int64_t tokens = up.size(0);
        const int32_t* parents = dense<int32_t>(a[2], dev, at::kInt, tokens);
        q4gsw_kv_seqs s{};
        const int64_t batch = sequences(a + 4, dev, tokens, &s);
        const int32_t *leaf = dense<int32_t>(a[3], dev, at::kInt, batch), max_new = int32(a[7]);
        need(max_new >= 1);
        void* st = stream(dev);
        const at::Tensor kept = a[8] == Py_None ? fresh({batch}, at::kInt, dev) : tensor(a[8], dev);
        const at::Tensor path = a[9] == Py_None ? fresh({batch, max_new}, at::kInt, dev) : tensor(a[9], dev);
        need(kept.scalar_type() == at::kInt && kept.dim() == 1 && kept.size(0) == batch && kept.is_contiguous());
        need(path.scalar_type() == at::kInt && path.dim() == 2 && path.size(0) == batch && path.size(1) == max_new && path.is_contiguous());
        int32_t *kp = kept.data_ptr<int32_t>(), *pp = path.data_ptr<int32_t>();
        const int e = status_of([&] { return lib.kv_keep(caches, count, &s, parents, leaf, max_new, kp, pp, st); });
        return e ? PyLong_FromLong(e) : Py_BuildValue("(NN)", wrap(kept), wrap(path));
    });
}

// (weight or None, set, device, x, slots, y or None, out or None, workspace or None): out
PyObject* adapters(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return regular(n, 8, [&]() -> PyObject* {
        const q4gsw_weight* w = a[0] == Py_None ? nullptr : address<const q4gsw_weight>(a[0]);
        const q4gsw_adapters* set = address<const q4gsw_adapters>(a[1]);
        const int dev = int32(a[2]);
        const at::Tensor& x = tensor(a[3], dev);
        const int32_t dt = dtype_of(x);
        need(x.dim() == 2 && x.size(1) == set->K && x.size(0) >= 1 && x.is_contiguous());
        const int64_t M = x.size(0);
        const int32_t* slots = dense<int32_t>(a[4], dev, at::kInt, M);
        auto rows = [&](const at::Tensor& t) {
            need(t.scalar_type() == at::kFloat && t.dim() == 2 && t.size(0) == M && t.size(1) == set->N && t.is_contiguous());
            return t.data_ptr<float>();
        };
        const float* y = w ? nullptr : rows(tensor(a[5], dev));
        uint64_t bytes = 0;
        need(lib.adapters_workspace_bytes(set, w, M, dt, &bytes) == Q4GSW_OK);
        void* st = stream(dev);
        const at::Tensor out = a[6] == Py_None ? fresh({M, set->N}, at::kFloat, dev) : tensor(a[6], dev);
        float* op = rows(out);
        const at::Tensor ws = bytes_of(a[7], dev, bytes);
        need((uint64_t)ws.numel() >= bytes);
        void *wp = ws.data_ptr(), *xp = x.data_ptr();
        const uint64_t wb = (uint64_t)ws.numel();
        const int e = status_of([&] {
            return w ? lib.adapters_fwd(w, set, xp, dt, M, slots, op, wp, wb, st)
                     : lib.adapters_add(set, xp, dt, M, slots, y, op, wp, wb, st);
        });
        return result(e, wrap, out);
    });
}

// (logits, cu, max_new, history, history_lens, prompt_lens, ids, parents, repetition, presence, frequency, bias_ids,
// bias, mask, out), each but the first and third or None: out
PyObject* logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return regular(n, 15, [&]() -> PyObject* {
        need(THPVariable_CheckExact(a[0]));
        const int dev = THPVariable_Unpack(a[0]).device().index();
        const at::Tensor& x = tensor(a[0], dev);
        const int32_t dt = dtype_of(x);
        need(x.dim() == 2);
        const int64_t rows = x.size(0), V = x.size(1);
        auto pitch = [&](const at::Tensor& t) {
            const int64_t ld = rows <= 1 ? V : t.stride(0);
            need((V <= 1 || t.stride(1) == 1) && ld >= V);
            return ld;
        };
        int64_t batch = rows;
        if (a[1] != Py_None) {
            const at::Tensor& cu = tensor(a[1], dev);
            need(cu.dim() == 1 && cu.size(0) >= 2);
            batch = cu.size(0) - 1;
        }
        need(batch <= 0x7fffffff);
        q4gsw_logits_rules r{};
        r.batch = (int32_t)batch;
        r.cu = dense_or_null<int32_t>(a[1], dev, at::kInt, batch + 1);
        r.max_new = int32(a[2]);
        int64_t cols = 0, other = 0, other_ld = 0;
        if (a[3] != Py_None) {
            r.history = table<int32_t>(a[3], dev, at::kInt, batch, &r.history_ld, &cols);
            need(a[4] != Py_None && cols <= 0x7fffffff);
            r.history_cols = (int32_t)cols;
        }
        r.history_len = dense_or_null<int32_t>(a[4], dev, at::kInt, batch);
        r.prompt_len = dense_or_null<int32_t>(a[5], dev, at::kInt, batch);
        r.ids = dense_or_null<int32_t>(a[6], dev, at::kInt, rows);
        r.parents = dense_or_null<int32_t>(a[7], dev, at::kInt, rows);
        need(!r.parents || (a[1] != Py_None && a[6] != Py_None));
        r.repetition = dense_or_null<float>(a[8], dev, at::kFloat, batch);
        r.presence = dense_or_null<float>(a[9], dev, at::kFloat, batch);
        r.frequency = dense_or_null<float>(a[10], dev, at::kFloat, batch);
        need((a[11] == Py_None) == (a[12] == Py_None));
        if (a[11] != Py_None) {
            r.bias_ids = table<int32_t>(a[11], dev, at::kInt, batch, &r.bias_ld, &cols);
            r.bias = table<float>(a[12], dev, at::kFloat, batch, &other_ld, &other);
            need(other == cols && other_ld == r.bias_ld && cols <= 0x7fffffff);
            r.bias_cols = (int32_t)cols;
        }
        if (a[13] != Py_None) {
            r.mask = reinterpret_cast<const uint32_t*>(table<int32_t>(a[13], dev, at::kInt, rows, &r.mask_ld, &cols));
            need(cols >= (V + 31) / 32);
        }
        void* st = stream(dev);
        const at::Tensor out = a[14] == Py_None ? fresh({rows, V}, x.scalar_type(), dev) : tensor(a[14], dev);
        need(out.scalar_type() == x.scalar_type() && out.dim() == 2 && out.size(0) == rows && out.size(1) == V);
        const int64_t ld = pitch(x), out_ld = pitch(out);
        void *xp = x.data_ptr(), *op = out.data_ptr();
        const int e = status_of([&] { return lib.logits_adjust(xp, dt, rows, V, ld, &r, op, out_ld, st); });
        return result(e, wrap, out);
    });
}

// (handle of the library, torch's current device, its raw stream of a device)
PyObject* open(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    void* h = PyLong_AsVoidPtr(a[0]);
    if (PyErr_Occurred()) return nullptr;
#define Q4GSW_FIND(f)                                                                        \
    if (!(lib.f = reinterpret_cast<decltype(lib.f)>(dlsym(h, "q4gsw_" #f)))) {              \
        PyErr_SetString(PyExc_ImportError, "the library has no q4gsw_" #f);                 \
        return nullptr;                                                                     \
    }
    Q4GSW_CALLS(Q4GSW_FIND)
#undef Q4GSW_FIND
    Py_INCREF(a[1]);
    Py_INCREF(a[2]);
    get_device = a[1];
    get_stream = a[2];
    Py_RETURN_NONE;
}

#define Q4GSW_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {Q4GSW_METHOD(open), Q4GSW_METHOD(attention), Q4GSW_METHOD(append), Q4GSW_METHOD(read),
                         Q4GSW_METHOD(keep), Q4GSW_METHOD(adapters), Q4GSW_METHOD(logits), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) Py_CLEAR(m);      // whose tensors it reads
    return m;
}
