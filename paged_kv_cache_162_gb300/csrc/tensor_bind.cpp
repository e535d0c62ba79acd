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
