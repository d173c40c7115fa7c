// The ordinary case of the binding's calls that a model makes once per layer and token, natively.
//
// Each function takes what the Python function of the same entry point takes (agent_kv_cache_lse_b200/kvc.py), and if every
// tensor is as that function requires (type, shape, contiguity, all on the current CUDA device), packs the C arguments,
// makes the call and returns its status.  Otherwise it does nothing and returns -1, and the Python function goes on:
// it says what is wrong, or handles what is rare (another device than the current one, tokens inside a wider array).
// Attribute reads, shape tuples and ctypes conversions took 9 to 17 us a call in Python; the launches take 2 to 5.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <string>

#include "../../include/kvc.h"

namespace {

decltype(&kvc_reserve_slots) f_reserve;
decltype(&kvc_norm_rope_write) f_write;
decltype(&kvc_block_bounds) f_bounds;
decltype(&kvc_select_blocks) f_select;
decltype(&kvc_block_attention) f_attend;

PyObject *s_k_pool, *s_v_pool, *s_table, *s_len, *s_pos, *s_label, *s_seqs, *s_layers, *s_heads, *s_stream;

using Shape = std::initializer_list<int64_t>;

// A call's tensors: anything that is not as required clears `ok` for good.
struct Call {
    bool ok = true;
    kvc_cache cache{};
    int64_t rows = 0, pages = 0, P = 0, D = 0, S = 0, L = 0, H = 0;  // pages: of a row at most
    c10::ScalarType type{};
    int dev = -1;
    PyObject *held[10] = {};  // attributes read from the cache object

    ~Call() {
        for (PyObject *o : held) Py_XDECREF(o);
    }

    bool fits(const at::Tensor &t, c10::ScalarType st, Shape shape) {
        const auto have = t.sizes();
        if (t.scalar_type() != st || have.size() != shape.size() || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
            return false;
        size_t i = 0;
        for (int64_t n : shape)
            if (have[i++] != n) return false;
        return true;
    }
    const at::Tensor *tensor(PyObject *o) {
        if (!o || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    void *arg(PyObject *o, c10::ScalarType st, Shape shape) {
        if (!ok) return nullptr;
        const at::Tensor *t = tensor(o);
        if (!t || !fits(*t, st, shape)) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    void *opt(PyObject *o, c10::ScalarType st, Shape shape) { return o == Py_None ? nullptr : arg(o, st, shape); }
    int64_t size(PyObject *o, int dims, int dim) {
        const at::Tensor *t = ok ? tensor(o) : nullptr;
        if (!t || t->dim() != dims) {
            ok = false;
            return 0;
        }
        return t->size(dim);
    }
    PyObject *attr(PyObject *o, PyObject *name, int i) {
        held[i] = PyObject_GetAttr(o, name);
        if (!held[i]) {
            PyErr_Clear();
            ok = false;
        }
        return held[i];
    }
    int64_t number(PyObject *o, int64_t lo, int64_t hi) {
        if (!ok || !o || !PyLong_Check(o)) {
            ok = false;
            return 0;
        }
        int over = 0;
        const long long v = PyLong_AsLongLongAndOverflow(o, &over);
        if (over || v < lo || v > hi) ok = false;
        return v;
    }

    // The cache object's fields; `tables`: its tables are read and must have their shapes
    explicit Call(PyObject *c, bool tables) {
        PyObject *kp = attr(c, s_k_pool, 0), *vp = attr(c, s_v_pool, 1), *bt = attr(c, s_table, 2), *len = attr(c, s_len, 3),
                 *pos = attr(c, s_pos, 4), *label = attr(c, s_label, 5);
        S = number(attr(c, s_seqs, 6), 1, INT32_MAX);
        L = number(attr(c, s_layers, 7), 1, INT32_MAX);
        H = number(attr(c, s_heads, 8), 1, INT32_MAX);
        if (!ok) return;
        const at::Tensor *k = tensor(kp), *b = tensor(bt);
        if (!ok || !k->is_cuda() || k->dim() != 3 || b->dim() != 2 || S * L > INT32_MAX) {
            ok = false;
            return;
        }
        dev = (int)k->get_device();
        type = k->scalar_type();
        if (dev != c10::cuda::current_device() || (type != c10::kBFloat16 && type != c10::kFloat)) {
            ok = false;
            return;
        }
        rows = S * L * H;
        pages = b->size(1);
        P = k->size(1);
        D = k->size(2);
        const int64_t n = k->size(0);
        cache.k_pool = arg(kp, type, {n, P, D});
        cache.v_pool = arg(vp, type, {n, P, D});
        cache.num_pages = n;
        if (P > INT32_MAX || D > INT32_MAX || pages > INT32_MAX) ok = false;
        cache.page_size = (int32_t)P;
        cache.head_dim = (int32_t)D;
        cache.dtype = type == c10::kBFloat16 ? KVC_BF16 : KVC_F32;
        cache.max_pages_per_row = (int32_t)pages;
        cache.num_seqs = (int32_t)S;
        cache.num_layers = (int32_t)L;
        cache.num_kv_heads = (int32_t)H;
        if (tables) {
            cache.block_table = (int32_t *)arg(bt, c10::kInt, {rows, pages});
            cache.row_len = (int32_t *)arg(len, c10::kInt, {rows});
            cache.slot_pos = (int32_t *)arg(pos, c10::kInt, {rows, pages * P});
            cache.slot_label = (uint8_t *)opt(label, c10::kByte, {rows, pages * P});
        } else if (ok) {  // only passed on
            const at::Tensor *l = tensor(len), *p = tensor(pos);
            if (!ok) return;
            cache.block_table = (int32_t *)b->data_ptr();
            cache.row_len = (int32_t *)l->data_ptr();
            cache.slot_pos = (int32_t *)p->data_ptr();
        }
    }
    // a workspace of any type: address and bytes
    void *work(PyObject *o, size_t &bytes) {
        const at::Tensor *t = ok ? tensor(o) : nullptr;
        if (!t || !t->is_cuda() || t->get_device() != dev || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        bytes = t->nbytes();
        return t->data_ptr();
    }
    int32_t *status(PyObject *o) { return (int32_t *)opt(o, c10::kInt, {2}); }
    kvc_stream_t stream(PyObject *o) {
        if (!ok) return nullptr;
        if (o == Py_None) return (kvc_stream_t)c10::cuda::getCurrentCUDAStream(dev).stream();
        PyObject *h = PyLong_Check(o) ? o : attr(o, s_stream, 9);
        if (!h || !PyLong_Check(h)) {
            ok = false;
            return nullptr;
        }
        const unsigned long long s = PyLong_AsUnsignedLongLong(h);
        if (s == ~0ull && PyErr_Occurred()) ok = false;  // negative, or past 64 bits
        return (kvc_stream_t)(uintptr_t)s;
    }
};

PyObject *unhandled() {
    PyErr_Clear();
    return PyLong_FromLong(-1);
}

// (cache, new_count, next_pos, label, crf, free_pages, free_count, row_len_out, free_count_out, token_start, token_pos,
//  slot_map, workspace, d_status, stream)
PyObject *reserve(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 15 || !f_reserve) return unhandled();
    Call c(a[0], true);
    const int64_t T = c.size(a[10], 1, 0), free = c.size(a[5], 1, 0);
    auto cnt = (const int32_t *)c.arg(a[1], c10::kInt, {c.S}), next = (const int32_t *)c.arg(a[2], c10::kInt, {c.S});
    const int64_t label = c.number(a[3], 0, 255);
    auto crf = (float *)c.opt(a[4], c10::kFloat, {c.rows, c.pages * c.P});
    auto fp = (const int32_t *)c.arg(a[5], c10::kInt, {free});
    auto fc = (const int64_t *)c.arg(a[6], c10::kLong, {1});
    auto len = (int32_t *)c.arg(a[7], c10::kInt, {c.rows});
    auto fo = (int64_t *)c.arg(a[8], c10::kLong, {1});
    auto start = (int32_t *)c.arg(a[9], c10::kInt, {c.S + 1}), pos = (int32_t *)c.arg(a[10], c10::kInt, {T});
    auto map = (int64_t *)c.arg(a[11], c10::kLong, {T, c.L, c.H});
    size_t bytes = 0;
    void *ws = c.work(a[12], bytes);
    int32_t *st = c.status(a[13]);
    kvc_stream_t stream = c.stream(a[14]);
    if (!c.ok || T > INT32_MAX) return unhandled();
    return PyLong_FromLong(f_reserve(&c.cache, cnt, next, (uint8_t)label, crf, fp, free, fc, (int32_t)T, len, fo, start, pos, map, ws,
                                     bytes, st, stream));
}

// (cache, qkv, token_pos, slot_map, q_out, q_weight, k_weight, eps, inv_freq, interleaved, token_count, d_status, stream)
PyObject *write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13 || !f_write) return unhandled();
    Call c(a[0], false);
    const int64_t T = c.size(a[1], 4, 0), heads = c.size(a[1], 4, 2), Hq = heads - 2 * c.H;
    auto qkv = c.arg(a[1], c.type, {T, c.L, heads, c.D});
    auto pos = (const int32_t *)c.arg(a[2], c10::kInt, {T});
    auto map = (const int64_t *)c.arg(a[3], c10::kLong, {T, c.L, c.H});
    auto out = c.arg(a[4], c.type, {T, c.L, Hq, c.D});
    auto qw = c.opt(a[5], c.type, {c.L, c.D}), kw = c.opt(a[6], c.type, {c.L, c.D});
    const double eps = PyFloat_AsDouble(a[7]);
    if (eps == -1.0 && PyErr_Occurred()) return unhandled();
    const int64_t half = a[8] == Py_None ? 0 : c.size(a[8], 1, 0);
    auto inv = (const float *)c.opt(a[8], c10::kFloat, {half});
    const int inter = PyObject_IsTrue(a[9]);
    auto count = (const int32_t *)c.opt(a[10], c10::kInt, {1});
    int32_t *st = c.status(a[11]);
    kvc_stream_t stream = c.stream(a[12]);
    if (!c.ok || inter < 0 || Hq <= 0 || T > INT32_MAX || heads > INT32_MAX || half > (1 << 20)) return unhandled();
    return PyLong_FromLong(f_write(&c.cache, qkv, c.L * heads * c.D, (int32_t)T, count, (int32_t)Hq, qw, kw, (float)eps, inv,
                                   (int32_t)(2 * half), inter ? KVC_ROPE_INTERLEAVED : 0, pos, map, out, st, stream));
}

// (cache, bounds, block_pos, from_len, d_status, stream)
PyObject *bounds(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 6 || !f_bounds) return unhandled();
    Call c(a[0], true);
    auto b = c.arg(a[1], c.type, {c.rows, c.pages, 2, c.D});
    auto pos = (int32_t *)c.arg(a[2], c10::kInt, {c.rows, c.pages});
    auto from = (const int32_t *)c.opt(a[3], c10::kInt, {c.rows});
    int32_t *st = c.status(a[4]);
    kvc_stream_t stream = c.stream(a[5]);
    if (!c.ok) return unhandled();
    return PyLong_FromLong(f_bounds(&c.cache, from, b, pos, st, stream));
}

// (cache, bounds, block_pos, q, q_pos, block_list, block_count, workspace, sink_blocks, recent_blocks, d_status, stream)
PyObject *select(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 12 || !f_select) return unhandled();
    Call c(a[0], true);
    const int64_t Hq = c.size(a[3], 4, 2), k = c.size(a[5], 2, 1);
    auto b = c.arg(a[1], c.type, {c.rows, c.pages, 2, c.D});
    auto pos = (const int32_t *)c.arg(a[2], c10::kInt, {c.rows, c.pages});
    auto q = c.arg(a[3], c.type, {c.S, c.L, Hq, c.D});
    auto qp = (const int32_t *)c.arg(a[4], c10::kInt, {c.S});
    auto list = (int32_t *)c.arg(a[5], c10::kInt, {c.rows, k});
    auto count = (int32_t *)c.arg(a[6], c10::kInt, {c.rows});
    size_t bytes = 0;
    void *ws = c.work(a[7], bytes);
    const int64_t sink = c.number(a[8], INT32_MIN, INT32_MAX), recent = c.number(a[9], INT32_MIN, INT32_MAX);
    int32_t *st = c.status(a[10]);
    kvc_stream_t stream = c.stream(a[11]);
    if (!c.ok || Hq > INT32_MAX || k > INT32_MAX) return unhandled();
    return PyLong_FromLong(f_select(&c.cache, b, pos, q, qp, (int32_t)Hq, (int32_t)k, (int32_t)sink, (int32_t)recent, list, count,
                                    ws, bytes, st, stream));
}

// (cache, q, q_pos, out, lse, workspace, block_list, block_count, d_status, stream)
PyObject *attend(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 10 || !f_attend || (a[6] == Py_None) != (a[7] == Py_None)) return unhandled();
    Call c(a[0], true);
    const int64_t Hq = c.size(a[1], 4, 2), apart = a[6] == Py_None ? 0 : c.size(a[6], 2, 1);
    auto q = c.arg(a[1], c.type, {c.S, c.L, Hq, c.D});
    auto qp = (const int32_t *)c.arg(a[2], c10::kInt, {c.S});
    auto out = (float *)c.arg(a[3], c10::kFloat, {c.S, c.L, Hq, c.D});
    auto lse = (float *)c.arg(a[4], c10::kFloat, {c.S, c.L, Hq});
    size_t bytes = 0;
    void *ws = c.work(a[5], bytes);
    auto list = (const int32_t *)c.opt(a[6], c10::kInt, {c.rows, apart});
    auto count = (const int32_t *)c.opt(a[7], c10::kInt, {c.rows});
    int32_t *st = c.status(a[8]);
    kvc_stream_t stream = c.stream(a[9]);
    if (!c.ok || Hq > INT32_MAX || apart > INT32_MAX) return unhandled();
    return PyLong_FromLong(f_attend(&c.cache, q, qp, (int32_t)Hq, list, (int32_t)apart, count, out, lse, ws, bytes, st, stream));
}

// bind(handle): the entry points of the library that dlopen returned `handle` for
PyObject *bind(PyObject *, PyObject *handle) {
    void *h = PyLong_AsVoidPtr(handle);
    if (!h) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no library handle");
        return nullptr;
    }
    f_reserve = (decltype(f_reserve))dlsym(h, "kvc_reserve_slots");
    f_write = (decltype(f_write))dlsym(h, "kvc_norm_rope_write");
    f_bounds = (decltype(f_bounds))dlsym(h, "kvc_block_bounds");
    f_select = (decltype(f_select))dlsym(h, "kvc_select_blocks");
    f_attend = (decltype(f_attend))dlsym(h, "kvc_block_attention");
    Py_RETURN_NONE;
}

// C++ exceptions (from torch's calls) end at the module's border: the Python function then handles the call
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    try {
        return F(self, a, n);
    } catch (...) {
        return unhandled();
    }
}

PyMethodDef methods[] = {
    {"bind", bind, METH_O, nullptr},
    {"reserve", (PyCFunction)(void (*)(void))guarded<reserve>, METH_FASTCALL, nullptr},
    {"write", (PyCFunction)(void (*)(void))guarded<write>, METH_FASTCALL, nullptr},
    {"bounds", (PyCFunction)(void (*)(void))guarded<bounds>, METH_FASTCALL, nullptr},
    {"select", (PyCFunction)(void (*)(void))guarded<select>, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void (*)(void))guarded<attend>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

// Torch's tensor layout and the interpreter's are compiled in, so the module loads only into those it was built for (KVC_TORCH:
// the version of torch).
bool built_for_this() {
    const std::string python = std::to_string(PY_MAJOR_VERSION) + "." + std::to_string(PY_MINOR_VERSION) + ".";
    if (std::strncmp(Py_GetVersion(), python.c_str(), python.size()) != 0) return false;
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
    PyObject *text = version ? PyObject_Str(version) : nullptr;
    const char *have = text ? PyUnicode_AsUTF8(text) : nullptr;
    const bool same = have && std::strcmp(have, KVC_TORCH) == 0;
    Py_XDECREF(text);
    Py_XDECREF(version);
    Py_XDECREF(torch);
    PyErr_Clear();
    return same;
}

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) {
    if (!built_for_this()) {
        PyErr_SetString(PyExc_ImportError, "_bind.so was built for torch " KVC_TORCH " and another interpreter or torch is running");
        return nullptr;
    }
    struct {
        PyObject **to;
        const char *name;
    } names[] = {{&s_k_pool, "k_pool"}, {&s_v_pool, "v_pool"}, {&s_table, "block_table"}, {&s_len, "row_len"},
                 {&s_pos, "slot_pos"}, {&s_label, "slot_label"}, {&s_seqs, "num_seqs"}, {&s_layers, "num_layers"},
                 {&s_heads, "num_kv_heads"}, {&s_stream, "cuda_stream"}};
    for (auto &n : names)
        if (!(*n.to = PyUnicode_InternFromString(n.name))) return nullptr;
    return PyModule_Create(&module);
}
