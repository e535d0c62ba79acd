// Direct calls of the bounded-cache entry points with torch tensors.
//
// A decode call of a small batch takes 3 to 5 us on the GPU.  Checking its
// tensors in Python and passing 21 to 24 arguments through ctypes took 6 us of
// host time; the same checks here take a tenth of one, and the call costs
// little more than its launch.  This module decides nothing: a call whose
// arguments are not plain contiguous tensors of the right types and shapes on
// the current device is answered with kAskPython, and engine.py then says what
// is wrong or makes the call through ctypes.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "pagedkv.h"

namespace {

constexpr long kAskPython = -1;

// A tensor argument, or null where it is something else.
const at::Tensor* tensor(PyObject* o) {
    return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

struct Args {
    PyObject* const* v;
    c10::DeviceIndex dev = -1;
    bool ok = true;

    // argument i: contiguous, of type t, on the device of the first tensor taken
    const at::Tensor* take(int i, at::ScalarType t, int64_t dims) {
        const at::Tensor* x = ok ? tensor(v[i]) : nullptr;
        if (!x || !x->is_cuda() || x->scalar_type() != t || x->dim() != dims || !x->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        if (dev < 0) dev = x->get_device();
        if (x->get_device() != dev) ok = false;
        return ok ? x : nullptr;
    }
    int integer(int i) {
        if (!ok || !PyLong_CheckExact(v[i])) {
            ok = false;
            return 0;
        }
        int overflow = 0;
        const long x = PyLong_AsLongAndOverflow(v[i], &overflow);
        if (overflow || x < INT32_MIN || x > INT32_MAX) ok = false;
        return (int)x;
    }
    // a float, or 1 / sqrt(D) for None
    float scale(int i, int64_t D) {
        if (v[i] == Py_None) return (float)(1.0 / std::sqrt((double)D));
        if (!PyFloat_CheckExact(v[i])) {
            ok = false;
            return 0.f;
        }
        return (float)PyFloat_AS_DOUBLE(v[i]);
    }
    // torch's current stream on the tensors' device, which must be current
    void* stream() {
        if (!ok || c10::cuda::current_device() != dev) {
            ok = false;
            return nullptr;
        }
        return c10::cuda::getCurrentCUDAStream(dev).stream();
    }
};

bool small(const at::Tensor& t) {  // sizes that the C entry points can be told
    for (const int64_t n : t.sizes())
        if (n > INT32_MAX) return false;
    return true;
}

pkv_dtype code(at::ScalarType t) { return t == at::kHalf ? PKV_F16 : PKV_BF16; }

// The tensors that every call has: caches [NB, bs, Hkv, D] and tables [S, MB].
struct Caches {
    const at::Tensor *k, *v, *tables;
    at::ScalarType type;
    int NB, bs, Hkv, D, S, MB;
    bool take(Args& a, int ik, int iv, int it) {
        const at::Tensor* any = tensor(a.v[ik]);
        if (!any || (any->scalar_type() != at::kHalf && any->scalar_type() != at::kBFloat16)) return a.ok = false;
        type = any->scalar_type();
        k = a.take(ik, type, 4);
        v = a.take(iv, type, 4);
        tables = a.take(it, at::kInt, 2);
        if (!a.ok || v->sizes() != k->sizes() || !small(*k) || !small(*tables)) return a.ok = false;
        NB = (int)k->size(0);
        bs = (int)k->size(1);
        Hkv = (int)k->size(2);
        D = (int)k->size(3);
        S = (int)tables->size(0);
        MB = (int)tables->size(1);
        return true;
    }
};

// q and out [S, H, D], context_lens [S]; returns H
int query(Args& a, const Caches& c, int iq, int io, int il, const at::Tensor** q, const at::Tensor** out,
          const at::Tensor** lens) {
    *q = a.take(iq, c.type, 3);
    *out = a.take(io, c.type, 3);
    *lens = a.take(il, at::kInt, 1);
    if (!a.ok || (*q)->size(0) != c.S || (*q)->size(2) != c.D || (*out)->sizes() != (*q)->sizes() ||
        (*lens)->size(0) != c.S || !small(**q)) {
        a.ok = false;
        return 0;
    }
    return (int)(*q)->size(1);
}

PyObject* answer(long status) { return PyLong_FromLong(status); }

// window(out, q, k_cache, v_cache, block_tables, context_lens, window,
//        sink_tokens, scale, max_context_len, workspace)
PyObject* window(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 11) return answer(kAskPython);
    Args a{args};
    Caches c;
    const at::Tensor *q, *out, *lens;
    if (!c.take(a, 2, 3, 4)) return answer(kAskPython);
    const int H = query(a, c, 1, 0, 5, &q, &out, &lens);
    const int win = a.integer(6), sinks = a.integer(7), most = a.integer(9);
    const float scale = a.scale(8, c.D);
    const at::Tensor* ws = a.take(10, at::kByte, 1);
    void* stream = a.stream();
    if (!a.ok) return answer(kAskPython);
    return answer(pkv_paged_attention_decode_window(
        out->data_ptr(), q->data_ptr(), c.k->data_ptr(), c.v->data_ptr(),
        static_cast<const int32_t*>(c.tables->data_ptr()), static_cast<const int32_t*>(lens->data_ptr()), c.S, H,
        c.Hkv, c.D, c.bs, c.NB, c.MB, most, win, sinks, scale, code(c.type), ws->data_ptr(),
        (size_t)ws->numel(), stream));
}

// accumulate(out, scores, q, k_cache, v_cache, block_tables, context_lens,
//            scale, max_context_len, workspace)
PyObject* accumulate(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 10) return answer(kAskPython);
    Args a{args};
    Caches c;
    const at::Tensor *q, *out, *lens;
    if (!c.take(a, 3, 4, 5)) return answer(kAskPython);
    const int H = query(a, c, 2, 0, 6, &q, &out, &lens);
    const at::Tensor* scores = a.take(1, at::kFloat, 3);
    const float scale = a.scale(7, c.D);
    const int most = a.integer(8);
    const at::Tensor* ws = a.take(9, at::kByte, 1);
    void* stream = a.stream();
    if (!a.ok || scores->size(0) != c.S || scores->size(1) != c.Hkv) return answer(kAskPython);
    return answer(pkv_paged_attention_decode_accumulate(
        out->data_ptr(), static_cast<float*>(scores->data_ptr()), q->data_ptr(), c.k->data_ptr(),
        c.v->data_ptr(), static_cast<const int32_t*>(c.tables->data_ptr()),
        static_cast<const int32_t*>(lens->data_ptr()), c.S, H, c.Hkv, c.D, c.bs, c.NB, c.MB, most,
        scores->size(2), scale, code(c.type), ws->data_ptr(), (size_t)ws->numel(), stream));
}

// evict(k_cache, v_cache, scores, positions, block_tables, context_lens,
//       token_counts, new_context_lens, budget, recent_tokens, sink_tokens,
//       scores_out, positions_out, max_context_len, workspace)
PyObject* evict(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 15) return answer(kAskPython);
    Args a{args};
    Caches c;
    if (!c.take(a, 0, 1, 4)) return answer(kAskPython);
    const at::Tensor* scores = a.take(2, at::kFloat, 3);
    const at::Tensor* positions = a.take(3, at::kInt, 3);
    const at::Tensor* lens = a.take(5, at::kInt, 1);
    const at::Tensor* seen = a.take(6, at::kInt, 1);
    const at::Tensor* fresh = a.take(7, at::kInt, 1);
    const int budget = a.integer(8), recent = a.integer(9), sinks = a.integer(10), most = a.integer(13);
    const at::Tensor* scores_out = a.take(11, at::kFloat, 3);
    const at::Tensor* positions_out = a.take(12, at::kInt, 3);
    const at::Tensor* ws = a.take(14, at::kByte, 1);
    void* stream = a.stream();
    if (!a.ok || scores->size(0) != c.S || scores->size(1) != c.Hkv || positions->sizes() != scores->sizes() ||
        scores_out->sizes() != scores->sizes() || positions_out->sizes() != scores->sizes() ||
        lens->size(0) != c.S || seen->size(0) != c.S || fresh->size(0) != c.S)
        return answer(kAskPython);
    return answer(pkv_evict_tokens(
        c.k->data_ptr(), c.v->data_ptr(), static_cast<const float*>(scores->data_ptr()),
        static_cast<const int32_t*>(positions->data_ptr()), static_cast<const int32_t*>(c.tables->data_ptr()),
        static_cast<const int32_t*>(lens->data_ptr()), static_cast<const int32_t*>(seen->data_ptr()),
        static_cast<float*>(scores_out->data_ptr()), static_cast<int32_t*>(positions_out->data_ptr()),
        static_cast<int32_t*>(fresh->data_ptr()), c.S, c.Hkv, c.D, c.bs, c.NB, c.MB, most, scores->size(2),
        budget, recent, sinks, code(c.type), ws->data_ptr(), (size_t)ws->numel(), stream));
}

// rows of tokens [T, heads, D] of type t, each token's contiguous; the
// elements from one token to the next
const at::Tensor* token_rows(Args& a, int i, at::ScalarType t, int64_t T, int64_t heads, int64_t D, int64_t* stride) {
    const at::Tensor* x = a.ok ? tensor(a.v[i]) : nullptr;
    if (!x || !x->is_cuda() || x->scalar_type() != t || x->dim() != 3 || x->size(0) != T ||
        (heads >= 0 && x->size(1) != heads) || x->size(2) != D || x->numel() == 0 || x->stride(2) != 1 ||
        (x->size(1) > 1 && x->stride(1) != D) || !small(*x) || x->get_device() != a.dev) {
        a.ok = false;
        return nullptr;
    }
    *stride = T > 1 ? x->stride(0) : x->size(1) * D;
    return x;
}

// 4-bit caches [NB, Hkv, bs, RB] of head_dim D, arguments ik and iv.
struct Caches4 {
    const at::Tensor *k, *v;
    int NB, Hkv, bs;
    bool take(Args& a, int ik, int iv, int64_t D) {
        k = a.take(ik, at::kByte, 4);
        v = a.take(iv, at::kByte, 4);
        if (!a.ok || v->sizes() != k->sizes() || !small(*k) || D < 0 || D > 128 ||
            (size_t)k->size(3) != pkv_cache_q4_row_bytes((int)D))
            return a.ok = false;
        NB = (int)k->size(0);
        Hkv = (int)k->size(1);
        bs = (int)k->size(2);
        return true;
    }
};

// The 16-bit type, the first extent and the head_dim of o, a tensor of three dims.
bool rows_like(PyObject* o, at::ScalarType* type, int64_t* T, int64_t* D) {
    const at::Tensor* x = tensor(o);
    if (!x || x->dim() != 3 || (x->scalar_type() != at::kHalf && x->scalar_type() != at::kBFloat16)) return false;
    *type = x->scalar_type();
    *T = x->size(0);
    *D = x->size(2);
    return true;
}

// rotate(q4, key, value, k_cache, v_cache, block_tables, seq_idx, pos,
//        slot_mapping, rotary_table, query, query_out, rotary_pos, interleaved)
PyObject* rotate(PyObject*, PyObject* const* args, Py_ssize_t n) {
    at::ScalarType type;
    int64_t T, D;
    if (n != 14 || !PyBool_Check(args[0]) || !PyBool_Check(args[13]) || !rows_like(args[1], &type, &T, &D))
        return answer(kAskPython);
    Args a{args};
    const bool q4 = args[0] == Py_True;
    int NB, bs, Hkv;
    const at::Tensor *k, *v;
    if (q4) {
        Caches4 c;
        if (!c.take(a, 3, 4, D)) return answer(kAskPython);
        k = c.k, v = c.v, NB = c.NB, bs = c.bs, Hkv = c.Hkv;
    } else {
        k = a.take(3, type, 4);
        v = a.take(4, type, 4);
        if (!a.ok || v->sizes() != k->sizes() || !small(*k) || k->size(3) != D) return answer(kAskPython);
        NB = (int)k->size(0);
        bs = (int)k->size(1);
        Hkv = (int)k->size(2);
    }
    int64_t ks = 0, vs = 0, qs = 0, qos = 0;
    const at::Tensor* key = token_rows(a, 1, type, T, Hkv, D, &ks);
    const at::Tensor* value = token_rows(a, 2, type, T, Hkv, D, &vs);
    const at::Tensor* tables = a.take(5, at::kInt, 2);
    const at::Tensor* seq = a.take(6, at::kInt, 1);
    const at::Tensor* pos = a.take(7, at::kInt, 1);
    const at::Tensor* slots = a.take(8, at::kLong, 1);
    const at::Tensor* table = args[9] == Py_None ? nullptr : a.take(9, at::kFloat, 2);
    const at::Tensor* turn = args[12] == Py_None ? nullptr : a.take(12, at::kInt, 1);
    const at::Tensor *query = nullptr, *query_out = nullptr;
    if (args[10] != Py_None) {
        query = token_rows(a, 10, type, T, -1, D, &qs);
        query_out = token_rows(a, 11, type, T, query ? query->size(1) : 0, D, &qos);
    } else if (args[11] != Py_None) {
        return answer(kAskPython);
    }
    void* stream = a.stream();
    if (!a.ok || seq->size(0) != T || pos->size(0) != T || slots->size(0) != T || (turn && turn->size(0) != T) ||
        !small(*tables) || (table && !small(*table)))
        return answer(kAskPython);
    auto call = q4 ? pkv_rotate_and_cache_q4 : pkv_rotate_and_cache;
    return answer(call(
        key->data_ptr(), ks, value->data_ptr(), vs, query ? query->data_ptr() : nullptr, qs,
        query_out ? query_out->data_ptr() : nullptr, qos, k->data_ptr(), v->data_ptr(),
        static_cast<const int32_t*>(tables->data_ptr()), static_cast<const int32_t*>(seq->data_ptr()),
        static_cast<const int32_t*>(pos->data_ptr()),
        turn ? static_cast<const int32_t*>(turn->data_ptr()) : nullptr,
        table ? static_cast<const float*>(table->data_ptr()) : nullptr, table ? (int)table->size(0) : 0,
        table ? (int)table->size(1) : 0, args[13] == Py_True, static_cast<int64_t*>(slots->data_ptr()), (int)T,
        (int)tables->size(0), query ? (int)query->size(1) : 0, Hkv, (int)D, bs, NB, (int)tables->size(1), code(type),
        stream));
}

// gather(key, value, k_cache, v_cache, slot_mapping)
PyObject* gather(PyObject*, PyObject* const* args, Py_ssize_t n) {
    at::ScalarType type;
    int64_t T, D, ks = 0, vs = 0;
    if (n != 5 || !rows_like(args[0], &type, &T, &D)) return answer(kAskPython);
    Args a{args};
    Caches4 c;
    if (!c.take(a, 2, 3, D)) return answer(kAskPython);
    const at::Tensor* key = token_rows(a, 0, type, T, c.Hkv, D, &ks);
    const at::Tensor* value = token_rows(a, 1, type, T, c.Hkv, D, &vs);
    const at::Tensor* slots = a.take(4, at::kLong, 1);
    void* stream = a.stream();
    if (!a.ok || slots->size(0) != T) return answer(kAskPython);
    return answer(pkv_gather_cache_q4(key->data_ptr(), ks, value->data_ptr(), vs, c.k->data_ptr(), c.v->data_ptr(),
                                      static_cast<const int64_t*>(slots->data_ptr()), (int)T, c.Hkv, (int)D, c.bs,
                                      c.NB, code(type), stream));
}

// decode_q4(out, q, k_cache, v_cache, block_tables, context_lens, scale,
//           max_context_len, workspace)
PyObject* decode_q4(PyObject*, PyObject* const* args, Py_ssize_t n) {
    at::ScalarType type;
    int64_t S, D;
    if (n != 9 || !rows_like(args[1], &type, &S, &D)) return answer(kAskPython);
    Args a{args};
    Caches4 c;
    if (!c.take(a, 2, 3, D)) return answer(kAskPython);
    const at::Tensor* q = a.take(1, type, 3);
    const at::Tensor* out = a.take(0, type, 3);
    const at::Tensor* tables = a.take(4, at::kInt, 2);
    const at::Tensor* lens = a.take(5, at::kInt, 1);
    const float scale = a.scale(6, D);
    const int most = a.integer(7);
    const at::Tensor* ws = a.take(8, at::kByte, 1);
    void* stream = a.stream();
    if (!a.ok || out->sizes() != q->sizes() || tables->size(0) != S || lens->size(0) != S || !small(*q) ||
        !small(*tables))
        return answer(kAskPython);
    return answer(pkv_paged_attention_decode_q4(
        out->data_ptr(), q->data_ptr(), c.k->data_ptr(), c.v->data_ptr(),
        static_cast<const int32_t*>(tables->data_ptr()), static_cast<const int32_t*>(lens->data_ptr()), (int)S,
        (int)q->size(1), c.Hkv, (int)D, c.bs, c.NB, (int)tables->size(1), most, scale, code(type), ws->data_ptr(),
        (size_t)ws->numel(), stream));
}

// C++ exceptions (torch's device query) end here.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    try {
        return F(self, args, n);
    } catch (const std::exception&) {
        return answer(kAskPython);
    }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction entry() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>));
}

PyMethodDef methods[] = {
    {"window", entry<window>(), METH_FASTCALL, "pkv_paged_attention_decode_window with tensors"},
    {"accumulate", entry<accumulate>(), METH_FASTCALL, "pkv_paged_attention_decode_accumulate with tensors"},
    {"evict", entry<evict>(), METH_FASTCALL, "pkv_evict_tokens with tensors"},
    {"rotate", entry<rotate>(), METH_FASTCALL, "pkv_rotate_and_cache and pkv_rotate_and_cache_q4 with tensors"},
    {"gather", entry<gather>(), METH_FASTCALL, "pkv_gather_cache_q4 with tensors"},
    {"decode_q4", entry<decode_q4>(), METH_FASTCALL, "pkv_paged_attention_decode_q4 with tensors"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch that this was built against, the only one that it may be used with.
PyMODINIT_FUNC PyInit__tensor_bind() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", PKV_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
