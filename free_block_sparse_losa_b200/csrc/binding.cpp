// Argument marshalling of the streaming calls, in place of a ctypes call per argument: their small forms (one token, a short
// cache) take a few microseconds on the GPU, and checking ten tensors in Python takes twice that. It checks every tensor
// against the call's descriptors as the Python binding does for the other calls (dtype, size, layout, then device; an int
// is a raw device pointer), takes the current stream and calls the C entry point. No computation happens here.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <utility>

#include "losa.h"

namespace {

decltype(&losa_rope_apply) g_rope_apply = nullptr;
decltype(&losa_cache_append) g_cache_append = nullptr;
decltype(&losa_cache_attn) g_cache_attn = nullptr;
decltype(&losa_cache_sparse_attn) g_cache_sparse_attn = nullptr;

struct Refused {  // becomes a ValueError; empty: a Python error is set already
    std::string why;
};

std::string text_of(PyObject* o) {
    PyObject* s = PyObject_Str(o);
    std::string r = s ? PyUnicode_AsUTF8(s) : "?";
    Py_XDECREF(s);
    return r;
}

std::string shape_of(const at::Tensor& t) {
    std::string r = "(";
    for (int64_t i = 0; i < t.dim(); ++i) r += (i ? ", " : "") + std::to_string(t.size(i));
    return r + (t.dim() == 1 ? ",)" : ")");
}

const char* name_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "float32";
        case at::kBFloat16: return "bfloat16";
        case at::kInt: return "int32";
        default: return "float8_e4m3fn";
    }
}

// Pointers of a call's arguments; the devices are checked at the end, behind everything else.
class Args {
  public:
    const at::Tensor& tensor(PyObject* o, const char* name) {
        if (!THPVariable_Check(o)) throw Refused{std::string(name) + ": expected a tensor"};
        return THPVariable_Unpack(o);
    }
    // A contiguous buffer of at least numel elements (numel < 0: any number), NULL for None, or a raw pointer.
    void* buffer(PyObject* o, const char* name, at::ScalarType type, int64_t numel, bool any_type = false) {
        if (o == Py_None) return nullptr;
        if (PyLong_Check(o)) {
            void* p = PyLong_AsVoidPtr(o);
            if (PyErr_Occurred()) throw Refused{};
            return p;
        }
        const at::Tensor& t = tensor(o, name);
        if (!any_type) check_type(o, t, name, type);
        if (numel >= 0 && t.numel() < numel)
            throw Refused{std::string(name) + ": holds " + std::to_string(t.numel()) + " elements, the shape needs " +
                          std::to_string(numel)};
        if (!t.is_contiguous()) throw Refused{std::string(name) + ": expected a contiguous tensor"};
        note(o, t, name);
        return t.data_ptr();
    }
    // Any strides but a contiguous last dimension.
    void* strided(PyObject* o, const char* name, at::ScalarType type) {
        const at::Tensor& t = tensor(o, name);
        check_type(o, t, name, type);
        if (t.stride(-1) != 1 && t.size(-1) > 1)
            throw Refused{std::string(name) + ": the last dimension must be contiguous"};
        note(o, t, name);
        return t.data_ptr();
    }
    void check_devices() const {
        int here = -1;
        for (int i = 0; i < n_; ++i)
            if (!seen_[i].second->is_cuda()) throw Refused{std::string(seen_[i].first) + ": expected a CUDA tensor"};
        for (int i = 0; i < n_; ++i) {
            if (here < 0) here = c10::cuda::current_device();
            if (seen_[i].second->get_device() != here)
                throw Refused{std::string(seen_[i].first) + ": lives on " + seen_[i].second->device().str() +
                              ", the current device is cuda:" + std::to_string(here)};
        }
    }

  private:
    void check_type(PyObject* o, const at::Tensor& t, const char* name, at::ScalarType type) {
        if (t.scalar_type() == type) return;
        PyObject* d = PyObject_GetAttrString(o, "dtype");
        const std::string got = d ? text_of(d) : "?";
        Py_XDECREF(d);
        throw Refused{std::string(name) + ": expected torch." + name_of(type) + ", got " + got};
    }
    void note(PyObject*, const at::Tensor& t, const char* name) {
        if (n_ < 20) seen_[n_++] = {name, &t};
    }
    std::pair<const char*, const at::Tensor*> seen_[20];
    int n_ = 0;
};

// The memory of a ctypes structure.
template <typename T> class Struct {
  public:
    Struct(PyObject* o, const char* name) {
        if (o == Py_None) return;
        if (PyObject_GetBuffer(o, &view_, PyBUF_SIMPLE) != 0) throw Refused{};
        held_ = true;
        if (view_.len != (Py_ssize_t)sizeof(T)) {
            PyBuffer_Release(&view_);
            held_ = false;
            throw Refused{std::string(name) + ": expected the call's structure"};
        }
    }
    ~Struct() {
        if (held_) PyBuffer_Release(&view_);
    }
    Struct(const Struct&) = delete;
    const T* get() const { return held_ ? static_cast<const T*>(view_.buf) : nullptr; }
    const T* operator->() const { return get(); }

  private:
    Py_buffer view_;
    bool held_ = false;
};

cudaStream_t stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* raw = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!raw) throw Refused{};
    void* p = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw Refused{};
    return static_cast<cudaStream_t>(p);
}

int64_t whole(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}
int32_t int32_of(PyObject* o, const char* name) {
    const int64_t v = whole(o);
    if (v < INT32_MIN || v > INT32_MAX) throw Refused{std::string(name) + ": out of range"};
    return (int32_t)v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return (float)v;
}

at::ScalarType float_type(PyObject* o, const at::Tensor& t, const char* name) {
    const at::ScalarType s = t.scalar_type();
    if (s == at::kBFloat16 || s == at::kFloat) return s;
    PyObject* d = PyObject_GetAttrString(o, "dtype");
    const std::string got = d ? text_of(d) : "?";
    Py_XDECREF(d);
    throw Refused{std::string(name) + ": expected torch.bfloat16 or torch.float32, got " + got};
}
int32_t code_of(at::ScalarType t) { return t == at::kBFloat16 ? LOSA_DTYPE_BF16 : LOSA_DTYPE_F32; }

int32_t extent(int64_t n, const char* name) {
    if (n > INT32_MAX) throw Refused{std::string(name) + ": too large"};
    return (int32_t)n;
}

int64_t at_least_0(int64_t n) { return n > 0 ? n : 0; }

struct Pool {
    void *k8, *v8;
    float *k_scale, *v_scale;
    int32_t *table, *lens;
};
Pool pool_of(Args& a, const losa_cache* c, PyObject* const* o) {  // k8, v8, k_scale, v_scale, page_table, lens
    const int64_t n = at_least_0(c->n_pages) * at_least_0(c->kv_heads), seqs = at_least_0(c->seqs);
    const int64_t codes = n * at_least_0(c->page_tokens) * at_least_0(c->head_dim);
    Pool p;
    p.k8 = a.buffer(o[0], "k8", at::kFloat8_e4m3fn, codes);
    p.v8 = a.buffer(o[1], "v8", at::kFloat8_e4m3fn, codes);
    p.k_scale = (float*)a.buffer(o[2], "k_scale", at::kFloat, n);
    p.v_scale = (float*)a.buffer(o[3], "v_scale", at::kFloat, n);
    p.table = (int32_t*)a.buffer(o[4], "page_table", at::kInt, seqs * at_least_0(c->table_stride));
    p.lens = (int32_t*)a.buffer(o[5], "lens", at::kInt, seqs);
    return p;
}

// The C call itself runs without the interpreter's lock, as one by ctypes does: a launch may wait for room in its queue, and
// other threads go on meanwhile. Its arguments are read before.
template <typename F> losa_status unlocked(F call) {
    losa_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = call();
    Py_END_ALLOW_THREADS;
    return st;
}

// Runs f, turning what it throws into a Python error; returns the status as an int.
template <typename F> PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)f());
    } catch (const Refused& r) {
        if (!r.why.empty()) PyErr_SetString(PyExc_ValueError, r.why.c_str());
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// rope, x, y, rotate, inverse, positions, start, stream
PyObject* rope_apply(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        Struct<losa_rope> rope(o[0], "rope");
        if (!rope.get()) throw Refused{"rope: expected the call's structure"};
        Args a;
        const at::Tensor &x = a.tensor(o[1], "x"), &y = a.tensor(o[2], "y");
        const at::ScalarType type = float_type(o[1], x, "x");
        if (x.dim() != 5 || y.dim() != 5 || x.size(4) != rope->head_dim || y.size(4) != rope->head_dim)
            throw Refused{"x, y: shapes " + shape_of(x) + ", " + shape_of(y) + ", expected (parts, batch, tokens, heads, " +
                          std::to_string(rope->head_dim) + ")"};
        void *px = a.strided(o[1], "x", type), *py = a.strided(o[2], "y", type);
        const int32_t* pos = (const int32_t*)a.buffer(o[5], "positions", at::kInt, 3 * x.size(1) * x.size(2));
        const int32_t* start = (const int32_t*)a.buffer(o[6], "start", at::kInt, x.size(1));
        a.check_devices();
        losa_token_view v[2];
        for (int i = 0; i < 2; ++i) {
            const at::Tensor& t = i ? y : x;
            const char* name = i ? "y" : "x";
            v[i] = {extent(t.size(0), name), extent(t.size(1), name), extent(t.size(2), name), extent(t.size(3), name),
                    t.stride(0), t.stride(1), t.stride(2), t.stride(3)};
        }
        const uint32_t rotate = (uint32_t)whole(o[3]);
        const bool inverse = truth(o[4]);
        cudaStream_t stream = stream_of(o[7]);
        return unlocked([&] {
            return g_rope_apply(rope.get(), code_of(type), &v[0], px, &v[1], py, rotate, inverse, pos, start, stream);
        });
    });
}

// cache, k, v, k8, v8, k_scale, v_scale, page_table, lens, new_tokens, indptr, new_lens, rope, positions, stream
PyObject* cache_append(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        Struct<losa_cache> cache(o[0], "cache");
        Struct<losa_rope> rope(o[12], "rope");
        if (!cache.get()) throw Refused{"cache: expected the call's structure"};
        Args a;
        const at::Tensor &k = a.tensor(o[1], "k"), &v = a.tensor(o[2], "v");
        const at::ScalarType type = float_type(o[1], k, "k");
        if (k.dim() != 3 || k.size(1) != cache->kv_heads || k.size(2) != cache->head_dim || v.sizes() != k.sizes())
            throw Refused{"k, v: shapes " + shape_of(k) + ", " + shape_of(v) + ", expected (tokens, " +
                          std::to_string(cache->kv_heads) + ", " + std::to_string(cache->head_dim) + ") of both"};
        const Pool p = pool_of(a, cache.get(), o + 3);
        void *pk = a.strided(o[1], "k", type), *pv = a.strided(o[2], "v", type);
        const int64_t seqs = at_least_0(cache->seqs);
        const int32_t* indptr = (const int32_t*)a.buffer(o[10], "indptr", at::kInt, seqs + 1);
        int32_t* new_lens = (int32_t*)a.buffer(o[11], "new_lens", at::kInt, seqs);
        const int32_t* pos = (const int32_t*)a.buffer(o[13], "positions", at::kInt, 3 * k.size(0));
        a.check_devices();
        const int64_t ks[2] = {k.stride(0), k.stride(1)}, vs[2] = {v.stride(0), v.stride(1)}, total = k.size(0);
        const int32_t new_tokens = int32_of(o[9], "new_tokens");
        cudaStream_t stream = stream_of(o[14]);
        return unlocked([&] {
            return g_cache_append(cache.get(), rope.get(), code_of(type), pk, ks[0], ks[1], pv, vs[0], vs[1], total,
                                  new_tokens, indptr, pos, p.table, p.lens, new_lens, p.k8, p.v8, p.k_scale, p.v_scale,
                                  stream);
        });
    });
}

// cache, q, k8, v8, k_scale, v_scale, page_table, lens, scale, o, lse, causal, max_len, workspace, ws_bytes, stream
PyObject* cache_attn(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        Struct<losa_cache> cache(o[0], "cache");
        if (!cache.get()) throw Refused{"cache: expected the call's structure"};
        Args a;
        const at::Tensor &q = a.tensor(o[1], "q"), &out = a.tensor(o[9], "o");
        if (q.dim() != 4 || q.size(0) != cache->seqs || q.size(3) != cache->head_dim || out.sizes() != q.sizes())
            throw Refused{"q, o: shapes " + shape_of(q) + ", " + shape_of(out) + ", expected (" +
                          std::to_string(cache->seqs) + ", tokens, heads, " + std::to_string(cache->head_dim) + ") of both"};
        const Pool p = pool_of(a, cache.get(), o + 2);
        void *pq = a.strided(o[1], "q", at::kBFloat16), *po = a.strided(o[9], "o", at::kBFloat16);
        float* lse = (float*)a.buffer(o[10], "lse", at::kFloat, q.size(0) * q.size(1) * q.size(2));
        void* ws = a.buffer(o[13], "workspace", at::kFloat, -1, true);
        size_t ws_bytes = 0;
        const bool says = o[14] != Py_None;
        if (says) {
            const int64_t b = whole(o[14]);
            if (b < 0) throw Refused{"ws_bytes: out of range"};
            ws_bytes = (size_t)b;
        }
        if (o[13] != Py_None && THPVariable_Check(o[13])) {
            const at::Tensor& w = THPVariable_Unpack(o[13]);
            const size_t have = (size_t)w.numel() * w.element_size();
            if (says && have < ws_bytes)
                throw Refused{"workspace: holds " + std::to_string(have) + " bytes, ws_bytes says " + std::to_string(ws_bytes)};
            if (!says) ws_bytes = have;
        }  // a raw pointer without its size counts as empty, which is enough for calls that need no workspace
        a.check_devices();
        const int32_t heads = extent(q.size(2), "q"), tokens = extent(q.size(1), "q"), causal = truth(o[11]);
        const int64_t qs[3] = {q.stride(0), q.stride(1), q.stride(2)};
        const int64_t os[3] = {out.stride(0), out.stride(1), out.stride(2)};
        const float scale = real(o[8]);
        const int32_t max_len = int32_of(o[12], "max_len");
        cudaStream_t stream = stream_of(o[15]);
        return unlocked([&] {
            return g_cache_attn(cache.get(), heads, tokens, causal, pq, qs[0], qs[1], qs[2], p.table, p.lens, p.k8, p.v8,
                                p.k_scale, p.v_scale, scale, max_len, po, os[0], os[1], os[2], lse, ws, ws_bytes, stream);
        });
    });
}

// shape, cache, q, k8, v8, k_scale, v_scale, page_table, lens, scale, o, indptr, kv_block_idx, order, lse, stream
PyObject* cache_sparse_attn(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        Struct<losa_shape> shape(o[0], "shape");
        Struct<losa_cache> cache(o[1], "cache");
        if (!shape.get() || !cache.get()) throw Refused{"shape, cache: expected the call's structures"};
        Args a;
        const Pool p = pool_of(a, cache.get(), o + 3);
        const int64_t rows = at_least_0(shape->heads) * at_least_0(shape->n_padded);
        const int64_t items = shape->block_q > 0 ? at_least_0(shape->heads) * (at_least_0(shape->n_padded) / shape->block_q) : 0;
        const int64_t tokens = rows * at_least_0(shape->head_dim);
        void* q = a.buffer(o[2], "q", at::kBFloat16, tokens);
        const int32_t* indptr = (const int32_t*)a.buffer(o[11], "indptr", at::kInt, items + 1);
        const int32_t* idx = (const int32_t*)a.buffer(o[12], "kv_block_idx", at::kInt, -1);
        const int32_t* order = (const int32_t*)a.buffer(o[13], "order", at::kInt, items);
        void* out = a.buffer(o[10], "o", at::kBFloat16, tokens);
        float* lse = (float*)a.buffer(o[14], "lse", at::kFloat, rows);
        a.check_devices();
        const float scale = real(o[9]);
        cudaStream_t stream = stream_of(o[15]);
        return unlocked([&] {
            return g_cache_sparse_attn(shape.get(), cache.get(), q, p.table, p.lens, p.k8, p.v8, p.k_scale, p.v_scale, scale,
                                       indptr, idx, order, out, lse, stream);
        });
    });
}

// Addresses of the four entry points.
PyObject* bind(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded(n, 4, [&] {
        void* p[4];
        for (int i = 0; i < 4; ++i) {
            p[i] = PyLong_AsVoidPtr(o[i]);
            if (PyErr_Occurred()) throw Refused{};
        }
        g_rope_apply = reinterpret_cast<decltype(g_rope_apply)>(p[0]);
        g_cache_append = reinterpret_cast<decltype(g_cache_append)>(p[1]);
        g_cache_attn = reinterpret_cast<decltype(g_cache_attn)>(p[2]);
        g_cache_sparse_attn = reinterpret_cast<decltype(g_cache_sparse_attn)>(p[3]);
        return 0;
    });
}

#define LOSA_METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {LOSA_METHOD(rope_apply), LOSA_METHOD(cache_append), LOSA_METHOD(cache_attn),
                         LOSA_METHOD(cache_sparse_attn), LOSA_METHOD(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Argument marshalling of the streaming calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
