// binding.cpp -- the Python side of the calls a decode step makes: reads the torch
// tensors' addresses, sizes and types, checks them and calls the C entry point
// (include/pkv.h).  A CPython module of its own (_binding.so); ops.py holds the
// documented functions and marshals the others through ctypes, whose conversions
// take several times as long as the calls themselves (10 us against 3).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <exception>
#include <optional>
#include <string>

#include "pkv.h"

namespace {

// A Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyErr_FormatV(type, fmt, ap);
    va_end(ap);
    throw Raised{};
}

// Attribute names, interned once.
struct Names {
#define PKV_NAMES(X) \
    X(kind) X(k) X(v) X(k_scale) X(v_scale) X(v_zero) X(v_group) X(block_tables) X(context_lens) X(q_len) X(sliding_window) \
        X(freq) X(rotary_dim) X(layout) X(mscale) X(softcap) X(distance_slopes) X(doc_starts) X(prefix_lens) X(cuda_stream)
#define PKV_FIELD(n) PyObject* n = nullptr;
    PKV_NAMES(PKV_FIELD)
#undef PKV_FIELD
    bool init() {
#define PKV_INTERN(n) \
    if (!(n = PyUnicode_InternFromString(#n))) return false;
        PKV_NAMES(PKV_INTERN)
#undef PKV_INTERN
        return true;
    }
} names;

// An owned reference.
struct Ref {
    PyObject* o;
    explicit Ref(PyObject* x) : o(x) {
        if (!o) throw Raised{};
    }
    ~Ref() { Py_DECREF(o); }
    Ref(const Ref&) = delete;
    Ref& operator=(const Ref&) = delete;
};

// An attribute as an integer, from whatever int() takes.
long as_long(PyObject* obj, PyObject* name) {
    Ref a(PyObject_GetAttr(obj, name)), whole(PyNumber_Long(a.o));
    const long v = PyLong_AsLong(whole.o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

double as_double(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

int32_t fits(long v, const char* name) {
    if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_ValueError, "%s does not fit 32 bits", name);
    return int32_t(v);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) raise(PyExc_ValueError, "%s must be a torch tensor", name);
    return THPVariable_Unpack(o);
}

// An attribute that is a tensor or None; keeps it alive.
struct TensorAttr {
    Ref ref;
    const at::Tensor* t;
    TensorAttr(PyObject* obj, PyObject* name, const char* text)
        : ref(PyObject_GetAttr(obj, name)), t(ref.o == Py_None ? nullptr : &tensor(ref.o, text)) {}
};

// What the calls have in common: the device they run on, which every tensor has to live on, and its stream.
struct Call {
    mutable int current = -1;

    // asked for when a CUDA tensor is there: without a GPU torch has no current device to name
    int device() const {
        if (current < 0) current = c10::cuda::current_device();
        return current;
    }

    void where(const at::Tensor& t) const {
        if (!t.is_cuda()) raise(PyExc_ValueError, "pkv tensors must live on a CUDA device");
        if (t.get_device() != device())
            raise(PyExc_ValueError, "pkv tensors must live on the current CUDA device (%d), not cuda:%d", device(),
                  int(t.get_device()));
    }
    void* ptr(const at::Tensor& t) const {
        where(t);
        if (!t.is_contiguous()) raise(PyExc_ValueError, "pkv tensors must be contiguous");
        return t.data_ptr();
    }
    void* ptr(const TensorAttr& a) const { return a.t ? ptr(*a.t) : nullptr; }
    uint32_t* err(PyObject* o) const {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor(o, "err_flags");
        if ((t.scalar_type() != at::kInt && t.scalar_type() != at::ScalarType::UInt32) || t.numel() < 1)
            raise(PyExc_ValueError, "err_flags must be a device int32/uint32 tensor");
        return static_cast<uint32_t*>(ptr(t));
    }
    pkv_stream_t stream(PyObject* o) const {
        if (o == Py_None)
            return reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device())).stream());
        Ref a(PyObject_GetAttr(o, names.cuda_stream));
        void* s = PyLong_AsVoidPtr(a.o);
        if (!s && PyErr_Occurred()) throw Raised{};
        return static_cast<pkv_stream_t>(s);
    }
};

bool half_type(const at::Tensor& t, pkv_dtype* d) {
    if (t.scalar_type() == at::kBFloat16) *d = PKV_BF16;
    else if (t.scalar_type() == at::kHalf) *d = PKV_F16;
    else return false;
    return true;
}

pkv_dtype any_type(const at::Tensor& t, const char* name) {
    pkv_dtype d = PKV_F32;
    if (t.scalar_type() != at::kFloat && !half_type(t, &d))
        raise(PyExc_ValueError, "%s must be float16, bfloat16 or float32", name);
    return d;
}

// A cache's kind and sizes; its addresses after place().  The sizes are checked first, so that what they
// refuse is refused before any tensor's device matters.
struct CacheArg {
    TensorAttr k, v, ks, vs, vz;
    pkv_cache c;
    explicit CacheArg(PyObject* o)
        : k(o, names.k, "cache.k"), v(o, names.v, "cache.v"), ks(o, names.k_scale, "cache.k_scale"),
          vs(o, names.v_scale, "cache.v_scale"), vz(o, names.v_zero, "cache.v_zero") {
        Ref kind(PyObject_GetAttr(o, names.kind));
        const char* s = PyUnicode_AsUTF8(kind.o);
        if (!s) throw Raised{};
        static const char* const kinds[] = {"f16", "bf16", "k8v4", "i8", "e4m3"};
        int32_t id = 0;
        while (id < 5 && std::string(s) != kinds[id]) ++id;
        if (id == 5) raise(PyExc_KeyError, "'%s'", s);
        if (!k.t || !v.t || k.t->dim() != 4) raise(PyExc_ValueError, "a cache's k and v are [num_blocks, 16, num_kv_heads, head_dim]");
        const auto z = k.t->sizes();
        if (id == PKV_CACHE_I8 || id == PKV_CACHE_E4M3) {
            auto codes = [&](const at::Tensor& t) {
                if (id == PKV_CACHE_I8) return t.scalar_type() == at::kChar;
                return t.scalar_type() == at::ScalarType::Float8_e4m3fn || t.scalar_type() == at::kByte;
            };
            if (!codes(*k.t) || !codes(*v.t))
                raise(PyExc_ValueError, "a %s cache holds %s codes", s, id == PKV_CACHE_I8 ? "torch.int8" : "torch.float8_e4m3fn");
            auto scales = [&](const TensorAttr& a) {
                return a.t && a.t->scalar_type() == at::kFloat && a.t->dim() == 2 && a.t->size(0) == z[0] && a.t->size(1) == z[2];
            };
            if (v.t->sizes() != z || !scales(ks) || !scales(vs))
                raise(PyExc_ValueError, "a %s cache has k and v of one shape and float32 scales [num_blocks, num_kv_heads]", s);
        } else {
            // the bytes that k's shape implies, whatever type the tensors call them
            const int64_t rows = z[0] * z[1] * z[2];
            auto holds = [&](const TensorAttr& a, int64_t bytes, const char* name) {
                if (!a.t || int64_t(a.t->nbytes()) < bytes)
                    raise(PyExc_ValueError, "a %s cache's %s is smaller than k's shape asks for", s, name);
            };
            const bool packed = id == PKV_CACHE_K8V4;
            holds(k, rows * z[3] * (packed ? 1 : 2), "k");
            holds(v, packed ? rows * z[3] / 2 : rows * z[3] * 2, "v");
            if (packed) {
                holds(ks, rows * 2, "k_scale");
                holds(vs, rows * (z[3] / 32) * 2, "v_scale");
                holds(vz, rows * (z[3] / 32) * 2, "v_zero");
            }
        }
        c = pkv_cache{id, fits(z[0], "num_blocks"), fits(z[1], "block_size"), fits(z[2], "num_kv_heads"),
                      fits(z[3], "head_dim"), fits(as_long(o, names.v_group), "v_group"), nullptr, nullptr, nullptr, nullptr, nullptr};
    }
    void place(const Call& call) {
        c.k = call.ptr(k);
        c.v = call.ptr(v);
        c.k_scale = call.ptr(ks);
        c.v_scale = call.ptr(vs);
        c.v_zero = call.ptr(vz);
    }
};

// A batch's sizes; its addresses after place().
struct SeqsArg {
    TensorAttr bt, cl;
    pkv_seqs s;
    explicit SeqsArg(PyObject* o) : bt(o, names.block_tables, "block_tables"), cl(o, names.context_lens, "context_lens") {
        if (!bt.t || !cl.t || bt.t->scalar_type() != at::kInt || cl.t->scalar_type() != at::kInt)
            raise(PyExc_ValueError, "block_tables and context_lens must be int32");
        if (bt.t->dim() != 2) raise(PyExc_ValueError, "block_tables must be [num_seqs, max_blocks]");
        s = pkv_seqs{nullptr, nullptr, fits(bt.t->size(0), "num_seqs"), fits(bt.t->size(1), "max_blocks"),
                     fits(as_long(o, names.q_len), "q_len"), fits(as_long(o, names.sliding_window), "sliding_window")};
        if (cl.t->numel() < s.num_seqs) raise(PyExc_ValueError, "context_lens must be [num_seqs]");
    }
    void place(const Call& call) {
        s.block_tables = static_cast<const int32_t*>(call.ptr(bt));
        s.context_lens = static_cast<const int32_t*>(call.ptr(cl));
    }
};

// Address and row stride of a [tokens, heads, head_dim] view whose rows are contiguous.
struct Rows {
    void* data;
    int64_t stride;
};
Rows rows(const Call& call, PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != shape)
        raise(PyExc_ValueError, "%s must be %s [%lld, %lld, %lld]", name, c10::toString(type), (long long)shape[0],
              (long long)shape[1], (long long)shape[2]);
    call.where(t);
    const auto st = t.strides();
    // no element, no stride that matters (torch keeps what an empty view came with)
    if (t.numel() > 0 && (st[2] != 1 || (st[1] != shape[2] && shape[1] > 1))) raise(PyExc_ValueError, "%s: a token's heads must be contiguous", name);
    // one row (or none): any stride will do
    return {t.data_ptr(), shape[0] > 1 ? st[0] : shape[1] * shape[2]};
}

// The library's functions, looked up in the build that ops.py selects.
struct Lib {
    decltype(&pkv_rope_and_cache) rope_and_cache;
    decltype(&pkv_quantize_kv_blocks) quantize_kv_blocks;
    decltype(&pkv_paged_attention_scored) paged_attention_scored;
    decltype(&pkv_paged_attention_balanced) paged_attention_balanced;
    decltype(&pkv_gather_kv_cache_dequant) gather_kv_cache_dequant;
    decltype(&pkv_reshape_and_cache) reshape_and_cache;
    decltype(&pkv_quantize_kv) quantize_kv;
    decltype(&pkv_key_bounds) key_bounds;
    decltype(&pkv_select_pages) select_pages;
    decltype(&pkv_paged_attention_selected) paged_attention_selected;
} lib;
void* handle = nullptr;

// Run f without the interpreter lock, as ctypes does.
template <class F>
PyObject* status_of(F f) {
    pkv_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

// A Python-callable body: C++ exceptions stay inside.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    try {
        if (!handle) raise(PyExc_RuntimeError, "the library is not loaded");
        if (n != want) raise(PyExc_TypeError, "%zd arguments, not %zd", want, n);
        return f();
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject* py_load(PyObject*, PyObject* arg) {
    const char* path = PyUnicode_AsUTF8(arg);
    if (!path) return nullptr;
    void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!h) {
        PyErr_SetString(PyExc_RuntimeError, dlerror());
        return nullptr;
    }
    Lib l{};
#define PKV_LOOKUP(n)                                                  \
    l.n = reinterpret_cast<decltype(l.n)>(dlsym(h, "pkv_" #n));        \
    if (!l.n) {                                                        \
        PyErr_SetString(PyExc_RuntimeError, "pkv_" #n " is missing");  \
        return nullptr;                                                \
    }
    PKV_LOOKUP(rope_and_cache)
    PKV_LOOKUP(quantize_kv_blocks)
    PKV_LOOKUP(paged_attention_scored)
    PKV_LOOKUP(paged_attention_balanced)
    PKV_LOOKUP(gather_kv_cache_dequant)
    PKV_LOOKUP(reshape_and_cache)
    PKV_LOOKUP(quantize_kv)
    PKV_LOOKUP(key_bounds)
    PKV_LOOKUP(select_pages)
    PKV_LOOKUP(paged_attention_selected)
#undef PKV_LOOKUP
    lib = l;
    handle = h;   // kept for the life of the process
    Py_RETURN_NONE;
}

// (q_out, q, k, v, rope, positions, cache, slot_mapping, k_out, err_flags, stream)
PyObject* py_rope_and_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const Call call;
        const at::Tensor& q = tensor(a[1], "q");
        pkv_dtype dt;
        if (!half_type(q, &dt)) raise(PyExc_ValueError, "q must be float16 or bfloat16");
        if (q.dim() != 3) raise(PyExc_ValueError, "q must be [num_tokens, num_heads, head_dim]");
        const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
        const at::Tensor& k = tensor(a[2], "k");
        if (k.dim() != 3) raise(PyExc_ValueError, "k must be [num_tokens, num_kv_heads, head_dim]");
        const int64_t Hkv = k.size(1), qz[3] = {T, H, D}, kz[3] = {T, Hkv, D};
        const at::ScalarType ty = q.scalar_type();
        const at::Tensor& pos = tensor(a[5], "positions");
        if (pos.scalar_type() != at::kLong || pos.numel() != T)
            raise(PyExc_ValueError, "positions must be int64 [num_tokens]");
        const Rows rq = rows(call, a[1], "q", qz, ty), ro = rows(call, a[0], "q_out", qz, ty), rk = rows(call, a[2], "k", kz, ty);
        const Rows rko = a[8] == Py_None ? Rows{nullptr, 0} : rows(call, a[8], "k_out", kz, ty);
        Rows rv{nullptr, 0};
        const int64_t* slots = nullptr;
        std::optional<CacheArg> cache;
        if (a[6] != Py_None) {
            if (a[3] == Py_None || a[7] == Py_None) raise(PyExc_ValueError, "a cache write needs v and slot_mapping");
            const at::Tensor& s = tensor(a[7], "slot_mapping");
            if (s.scalar_type() != at::kLong || s.numel() != T) raise(PyExc_ValueError, "slot_mapping must be int64 [num_tokens]");
            cache.emplace(a[6]);
            cache->place(call);
            slots = static_cast<const int64_t*>(call.ptr(s));
            rv = rows(call, a[3], "v", kz, ty);
        }
        TensorAttr freq(a[4], names.freq, "freq");
        const long rotary = as_long(a[4], names.rotary_dim);
        if (!freq.t || freq.t->scalar_type() != at::kLong || freq.t->numel() * 2 != rotary)
            raise(PyExc_ValueError, "freq must be int64 [rotary_dim / 2]");
        Ref layout(PyObject_GetAttr(a[4], names.layout)), mscale(PyObject_GetAttr(a[4], names.mscale));
        const char* ls = PyUnicode_AsUTF8(layout.o);
        if (!ls) throw Raised{};
        const std::string lay(ls);
        if (lay != "half" && lay != "interleaved") raise(PyExc_ValueError, "layout '%s': 'half' or 'interleaved'", ls);
        const pkv_rope r{static_cast<const uint64_t*>(call.ptr(freq)), fits(rotary, "rotary_dim"),
                         lay == "half" ? PKV_ROPE_HALF : PKV_ROPE_INTERLEAVED, float(as_double(mscale.o))};
        uint32_t* err = call.err(a[9]);
        const pkv_stream_t stream = call.stream(a[10]);
        const int64_t* pp = static_cast<const int64_t*>(call.ptr(pos));
        const int32_t h = fits(H, "num_heads"), hkv = fits(Hkv, "num_kv_heads"), d = fits(D, "head_dim"), t = fits(T, "num_tokens");
        return status_of([&] {
            return lib.rope_and_cache(cache ? &cache->c : nullptr, &r, ro.data, ro.stride, rq.data, rq.stride, h, rko.data,
                                      rko.stride, rk.data, rk.stride, rv.data, rv.stride, hkv, d, dt, pp, slots, t, err, stream);
        });
    });
}

// (cache, k_new, v_new, seqs, cu_new_lens, err_flags, stream)
PyObject* py_quantize_kv_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        const Call call;
        const at::Tensor &k = tensor(a[1], "k_new"), &v = tensor(a[2], "v_new");
        pkv_dtype dt;
        if (!half_type(k, &dt) || v.scalar_type() != k.scalar_type())
            raise(PyExc_ValueError, "k_new / v_new must both be float16 or both bfloat16");
        CacheArg c(a[0]);
        SeqsArg s(a[3]);
        if (k.dim() != 3 || k.size(1) != c.c.num_kv_heads || k.size(2) != c.c.head_dim || v.sizes() != k.sizes())
            raise(PyExc_ValueError, "k_new / v_new must be [num_tokens, num_kv_heads, head_dim]");
        c.place(call);
        s.place(call);
        const Rows rk = rows(call, a[1], "k_new", k.sizes(), k.scalar_type()), rv = rows(call, a[2], "v_new", k.sizes(), k.scalar_type());
        if (s.cl.t->numel() != s.s.num_seqs) raise(PyExc_ValueError, "context_lens must be [num_seqs]");
        const int32_t* cu = nullptr;
        if (a[4] != Py_None) {
            const at::Tensor& t = tensor(a[4], "cu_new_lens");
            if (t.scalar_type() != at::kInt || t.numel() != int64_t(s.s.num_seqs) + 1)
                raise(PyExc_ValueError, "cu_new_lens must be int32 [num_seqs + 1]");
            cu = static_cast<const int32_t*>(call.ptr(t));
        }
        const int32_t tokens = fits(k.size(0), "num_tokens");
        uint32_t* err = call.err(a[5]);
        const pkv_stream_t stream = call.stream(a[6]);
        return status_of([&] { return lib.quantize_kv_blocks(&c.c, rk.data, rk.stride, rv.data, rv.stride, dt, tokens, cu, &s.s, err, stream); });
    });
}

// (out, q, scale, cache, seqs, scores, workspace, err_flags, stream)
PyObject* py_paged_attention_scored(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const Call call;
        CacheArg c(a[3]);
        SeqsArg s(a[4]);
        const at::Tensor &out = tensor(a[0], "out"), &q = tensor(a[1], "q"), &ws = tensor(a[6], "workspace");
        if (q.dim() != 3 || q.size(0) != int64_t(s.s.num_seqs) * s.s.q_len || q.size(2) != c.c.head_dim ||
            out.sizes() != q.sizes() || s.cl.t->numel() != s.s.num_seqs)
            raise(PyExc_ValueError, "q and out must be [num_seqs * q_len, num_heads, head_dim], context_lens [num_seqs]");
        pkv_dtype qt;
        if (!half_type(q, &qt)) raise(PyExc_ValueError, "q must be float16 or bfloat16");
        const pkv_dtype ot = any_type(out, "out");
        const int64_t H = q.size(1);
        TensorAttr slopes(a[5], names.distance_slopes, "distance_slopes"), starts(a[5], names.doc_starts, "doc_starts"),
            prefix(a[5], names.prefix_lens, "prefix_lens");
        if (slopes.t && (slopes.t->scalar_type() != at::kFloat || slopes.t->numel() != H))
            raise(PyExc_ValueError, "distance_slopes must be float32 [%lld]", (long long)H);
        for (const TensorAttr* t : {&starts, &prefix})
            if (t->t && (t->t->scalar_type() != at::kInt || t->t->numel() != s.s.num_seqs))
                raise(PyExc_ValueError, "%s must be int32 [%d]", t == &starts ? "doc_starts" : "prefix_lens", int(s.s.num_seqs));
        c.place(call);
        s.place(call);
        Ref cap(PyObject_GetAttr(a[5], names.softcap));
        const pkv_scores sc{float(as_double(cap.o)), static_cast<const float*>(call.ptr(slopes)),
                            static_cast<const int32_t*>(call.ptr(starts)), static_cast<const int32_t*>(call.ptr(prefix))};
        const float scale = float(as_double(a[2]));
        void *op = call.ptr(out), *wp = call.ptr(ws);
        const void* qp = call.ptr(q);
        const int32_t h = fits(H, "num_heads");
        uint32_t* err = call.err(a[7]);
        const pkv_stream_t stream = call.stream(a[8]);
        return status_of([&] {
            return lib.paged_attention_scored(op, ot, qp, qt, h, scale, &c.c, &s.s, &sc, wp, ws.nbytes(), err, stream);
        });
    });
}

// (out, q, scale, cache, seqs, workspace, err_flags, stream)
PyObject* py_paged_attention_balanced(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        const Call call;
        CacheArg c(a[3]);
        SeqsArg s(a[4]);
        const at::Tensor &out = tensor(a[0], "out"), &q = tensor(a[1], "q"), &ws = tensor(a[5], "workspace");
        if (q.dim() < 2) raise(PyExc_ValueError, "q must be [num_seqs * q_len, num_heads, head_dim]");
        // buffers of a larger batch are taken (their first rows), smaller ones are not
        const int64_t needed = int64_t(s.s.num_seqs) * s.s.q_len * q.size(1) * c.c.head_dim;
        if (q.numel() < needed || out.numel() < needed)
            raise(PyExc_ValueError, "q and out must be [num_seqs * q_len, num_heads, head_dim]");
        const pkv_dtype ot = any_type(out, "out"), qt = any_type(q, "q");
        c.place(call);
        s.place(call);
        const float scale = float(as_double(a[2]));
        void *op = call.ptr(out), *wp = call.ptr(ws);
        const void* qp = call.ptr(q);
        const int32_t h = fits(q.size(1), "num_heads");
        uint32_t* err = call.err(a[6]);
        const pkv_stream_t stream = call.stream(a[7]);
        return status_of(
            [&] { return lib.paged_attention_balanced(op, ot, qp, qt, h, scale, &c.c, &s.s, wp, ws.nbytes(), err, stream); });
    });
}

// (k_out, v_out, cu_seq_lens, cache, seqs, err_flags, stream)
PyObject* py_gather_kv_cache_dequant(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        const Call call;
        const at::Tensor &k = tensor(a[0], "k_out"), &v = tensor(a[1], "v_out"), &cu = tensor(a[2], "cu_seq_lens");
        if (cu.scalar_type() != at::kInt) raise(PyExc_ValueError, "cu_seq_lens must be int32");
        pkv_dtype dt;
        if (!half_type(k, &dt) || v.scalar_type() != k.scalar_type())
            raise(PyExc_ValueError, "k_out / v_out must both be float16 or both bfloat16");
        CacheArg c(a[3]);
        SeqsArg s(a[4]);
        if (k.sizes() != v.sizes() || (c.c.head_dim > 0 && c.c.num_kv_heads > 0 && k.numel() % (int64_t(c.c.num_kv_heads) * c.c.head_dim) != 0))
            raise(PyExc_ValueError, "k_out and v_out must both be [cu_seq_lens[num_seqs], num_kv_heads, head_dim]");
        if (cu.numel() < int64_t(s.s.num_seqs) + 1) raise(PyExc_ValueError, "cu_seq_lens must be int32 [num_seqs + 1]");
        c.place(call);
        s.place(call);
        void *kp = call.ptr(k), *vp = call.ptr(v);
        const int32_t* cp = static_cast<const int32_t*>(call.ptr(cu));
        uint32_t* err = call.err(a[5]);
        const pkv_stream_t stream = call.stream(a[6]);
        return status_of([&] { return lib.gather_kv_cache_dequant(kp, vp, dt, cp, &c.c, &s.s, err, stream); });
    });
}

// The cache writes by slot: (cache, k_new, v_new, slot_mapping, err_flags, stream).  type(cache, k_new, v_new) refuses tensors that
// the call would read as what they are not.
template <class Type, class F>
PyObject* write_by_slot(PyObject* const* a, Py_ssize_t n, Type type, F f) {
    return guarded(n, 6, [&] {
        const Call call;
        const at::Tensor &k = tensor(a[1], "k_new"), &v = tensor(a[2], "v_new"), &slots = tensor(a[3], "slot_mapping");
        if (slots.scalar_type() != at::kLong) raise(PyExc_ValueError, "slot_mapping must be int64");
        CacheArg c(a[0]);
        type(c, k, v);
        const int64_t needed = slots.numel() * c.c.num_kv_heads * c.c.head_dim;
        if (k.numel() < needed || v.numel() < needed)
            raise(PyExc_ValueError, "k_new / v_new must be [num_tokens, num_kv_heads, head_dim]");
        c.place(call);
        const void *kp = call.ptr(k), *vp = call.ptr(v);
        const int64_t* sp = static_cast<const int64_t*>(call.ptr(slots));
        const int32_t tokens = fits(slots.numel(), "num_tokens");
        uint32_t* err = call.err(a[4]);
        const pkv_stream_t stream = call.stream(a[5]);
        return status_of([&] { return f(c.c, k, kp, vp, sp, tokens, err, stream); });
    });
}

PyObject* py_reshape_and_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    // the cache's type, or the type that the cache's own tensors give its 16 bits; the library refuses the other kinds
    auto type = [](const CacheArg& c, const at::Tensor& k, const at::Tensor& v) {
        if (c.c.kind != PKV_CACHE_F16 && c.c.kind != PKV_CACHE_BF16) return;
        const at::ScalarType own = c.c.kind == PKV_CACHE_BF16 ? at::kBFloat16 : at::kHalf;
        auto fits_cache = [&](const at::Tensor& t) {
            return t.scalar_type() == own || (t.scalar_type() == c.k.t->scalar_type() && t.element_size() == 2);
        };
        if (!fits_cache(k) || !fits_cache(v)) raise(PyExc_ValueError, "k_new / v_new must be %s, as the cache is", c10::toString(own));
    };
    return write_by_slot(a, n, type, [](const pkv_cache& c, const at::Tensor&, const void* k, const void* v, const int64_t* slots,
                                        int32_t tokens, uint32_t* err, pkv_stream_t stream) {
        return lib.reshape_and_cache(&c, k, v, slots, tokens, err, stream);
    });
}

PyObject* py_quantize_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
    auto type = [](const CacheArg&, const at::Tensor& k, const at::Tensor& v) {
        if (v.scalar_type() != k.scalar_type()) raise(PyExc_ValueError, "k_new / v_new must be of one type");
    };
    return write_by_slot(a, n, type, [](const pkv_cache& c, const at::Tensor& kt, const void* k, const void* v, const int64_t* slots,
                                        int32_t tokens, uint32_t* err, pkv_stream_t stream) {
        pkv_dtype dt = PKV_F32;   // which the call refuses
        half_type(kt, &dt);
        return lib.quantize_kv(&c, k, v, dt, slots, tokens, err, stream);
    });
}

// A cache's key bounds, of their type and shape.
const at::Tensor& bounds_tensor(PyObject* o, const CacheArg& c) {
    const at::Tensor& b = tensor(o, "bounds");
    const at::ScalarType t = b.scalar_type();
    const bool fits_type = c.c.kind == PKV_CACHE_BF16 ? t == at::kBFloat16
                         : c.c.kind == PKV_CACHE_I8   ? t == at::kChar
                         : c.c.kind == PKV_CACHE_E4M3 ? t == at::ScalarType::Float8_e4m3fn || t == at::kByte
                                                      : t == at::kHalf;
    const int64_t shape[4] = {c.c.num_blocks, c.c.num_kv_heads, 2, c.c.head_dim};
    if (!fits_type || b.sizes() != at::IntArrayRef(shape, 4))
        raise(PyExc_ValueError, "bounds must be [num_blocks, num_kv_heads, 2, head_dim] of the cache's key type (k8v4: float16)");
    return b;
}

// int32 [num_seqs + 1] or None
const int32_t* prefix_sums(const Call& call, PyObject* o, const char* name, int32_t num_seqs) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kInt || t.numel() != int64_t(num_seqs) + 1)
        raise(PyExc_ValueError, "%s must be int32 [num_seqs + 1]", name);
    return static_cast<const int32_t*>(call.ptr(t));
}

// The lists of pages of each (query token, kv head): their address and width.
int32_t page_lists(const at::Tensor& lists, const at::Tensor& counts, int64_t rows, int32_t kv_heads) {
    if (lists.scalar_type() != at::kInt || counts.scalar_type() != at::kInt)
        raise(PyExc_ValueError, "page_lists / page_counts must be int32");
    if (lists.dim() != 3 || lists.size(0) != rows || lists.size(1) != kv_heads || counts.dim() != 2 || counts.size(0) != rows ||
        counts.size(1) != kv_heads)
        raise(PyExc_ValueError, "page_lists must be [num_rows, num_kv_heads, max_pages] and page_counts [num_rows, num_kv_heads]");
    return fits(lists.size(2), "max_pages");
}

// (bounds, cache, seqs, cu_new_lens, err_flags, stream)
PyObject* py_key_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const Call call;
        CacheArg c(a[1]);
        SeqsArg s(a[2]);
        const at::Tensor& b = bounds_tensor(a[0], c);
        if (s.cl.t->numel() != s.s.num_seqs) raise(PyExc_ValueError, "context_lens must be [num_seqs]");
        c.place(call);
        s.place(call);
        void* bp = call.ptr(b);
        const int32_t* cu = prefix_sums(call, a[3], "cu_new_lens", s.s.num_seqs);
        uint32_t* err = call.err(a[4]);
        const pkv_stream_t stream = call.stream(a[5]);
        return status_of([&] { return lib.key_bounds(bp, &c.c, cu, &s.s, err, stream); });
    });
}

// (page_lists, page_counts, q, bounds, cache, seqs, cu_q_lens, keep_first, keep_last, err_flags, stream)
PyObject* py_select_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const Call call;
        const at::Tensor &lists = tensor(a[0], "page_lists"), &counts = tensor(a[1], "page_counts"), &q = tensor(a[2], "q");
        CacheArg c(a[4]);
        SeqsArg s(a[5]);
        const at::Tensor& b = bounds_tensor(a[3], c);
        pkv_dtype qt;
        if (!half_type(q, &qt)) raise(PyExc_ValueError, "q must be float16 or bfloat16");
        if (q.dim() != 3 || q.size(2) != c.c.head_dim || s.cl.t->numel() != s.s.num_seqs)
            raise(PyExc_ValueError, "q must be [num_rows, num_heads, head_dim], context_lens [num_seqs]");
        const int32_t pages = page_lists(lists, counts, q.size(0), c.c.num_kv_heads);
        const long first = PyLong_AsLong(a[7]), last = PyLong_AsLong(a[8]);
        if (PyErr_Occurred()) throw Raised{};
        c.place(call);
        s.place(call);
        int32_t *lp = static_cast<int32_t*>(call.ptr(lists)), *cp = static_cast<int32_t*>(call.ptr(counts));
        const void *qp = call.ptr(q), *bp = call.ptr(b);
        const int32_t* cu = prefix_sums(call, a[6], "cu_q_lens", s.s.num_seqs);
        const int32_t h = fits(q.size(1), "num_heads"), rows = fits(q.size(0), "num_rows"), kf = fits(first, "keep_first"),
                      kl = fits(last, "keep_last");
        uint32_t* err = call.err(a[9]);
        const pkv_stream_t stream = call.stream(a[10]);
        return status_of([&] { return lib.select_pages(lp, cp, pages, kf, kl, qp, qt, h, rows, bp, &c.c, cu, &s.s, err, stream); });
    });
}

// (out, q, scale, cache, seqs, page_lists, page_counts, cu_q_lens, err_flags, stream)
PyObject* py_paged_attention_selected(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const Call call;
        CacheArg c(a[3]);
        SeqsArg s(a[4]);
        const at::Tensor &out = tensor(a[0], "out"), &q = tensor(a[1], "q"), &lists = tensor(a[5], "page_lists"),
                         &counts = tensor(a[6], "page_counts");
        if (q.dim() != 3 || q.size(2) != c.c.head_dim || out.sizes() != q.sizes() || s.cl.t->numel() != s.s.num_seqs)
            raise(PyExc_ValueError, "q and out must be [num_rows, num_heads, head_dim], context_lens [num_seqs]");
        pkv_dtype qt;
        if (!half_type(q, &qt)) raise(PyExc_ValueError, "q must be float16 or bfloat16");
        const pkv_dtype ot = any_type(out, "out");
        const int32_t pages = page_lists(lists, counts, q.size(0), c.c.num_kv_heads);
        c.place(call);
        s.place(call);
        const float scale = float(as_double(a[2]));
        void* op = call.ptr(out);
        const void* qp = call.ptr(q);
        const int32_t *lp = static_cast<const int32_t*>(call.ptr(lists)), *cp = static_cast<const int32_t*>(call.ptr(counts));
        const int32_t* cu = prefix_sums(call, a[7], "cu_q_lens", s.s.num_seqs);
        const int32_t h = fits(q.size(1), "num_heads"), rows = fits(q.size(0), "num_rows");
        uint32_t* err = call.err(a[8]);
        const pkv_stream_t stream = call.stream(a[9]);
        return status_of([&] {
            return lib.paged_attention_selected(op, ot, qp, qt, h, rows, scale, &c.c, cu, &s.s, lp, cp, pages, err, stream);
        });
    });
}

#define PKV_METHOD(n) {#n, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_##n)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"load", py_load, METH_O, nullptr},
                         PKV_METHOD(rope_and_cache),
                         PKV_METHOD(quantize_kv_blocks),
                         PKV_METHOD(paged_attention_scored),
                         PKV_METHOD(paged_attention_balanced),
                         PKV_METHOD(gather_kv_cache_dequant),
                         PKV_METHOD(reshape_and_cache),
                         PKV_METHOD(quantize_kv),
                         PKV_METHOD(key_bounds),
                         PKV_METHOD(select_pages),
                         PKV_METHOD(paged_attention_selected),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    if (!names.init()) return nullptr;
    return PyModule_Create(&module);
}
