// The calls of the softmax-attention layer, marshalled natively: serving makes them once a token and layer, on
// kernels of a few microseconds, where the interpreter's part of a call (10 us) is longer than the kernel.  Each
// function takes the plain case (contiguous CUDA tensors of the expected types on the current device, results and
// workspace made here, the current stream) and returns
//     the result(s),
//     None   where a tensor is anything else: gdn.py's general marshalling then takes the call, or says what is wrong,
//     an int a gdn_status other than GDN_OK.
// Sizes and values are checked where every caller's are, in the C calls.
// The module is not linked to libgdn.so: gdn.py hands it the entry points of the copy that it has loaded (bind), so that
// importing it maps no second one, and both ways call the same library whatever lies at its path by now.
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "gdn.h"

namespace {

using at::Tensor;

// libgdn's entry points that are called here, by name; NULL until bind.
#define GDN_ENTRIES(X)                                                                                            \
    X(gdn_qk_norm_rope_fwd) X(gdn_qk_norm_rope_bwd_workspace_size) X(gdn_qk_norm_rope_bwd)                        \
    X(gdn_attn_fwd_workspace_size) X(gdn_attn_fwd) X(gdn_attn_bwd_workspace_size) X(gdn_attn_bwd)                 \
    X(gdn_kv_append) X(gdn_attn_decode_workspace_size) X(gdn_attn_decode)
struct Entries {
#define X(f) decltype(&::f) f = nullptr;
    GDN_ENTRIES(X)
#undef X
    bool bound = false;
} lib;

// The tensors of one call: all like the first in place, and each of its own type.
struct Inputs {
    bool plain = true;
    int device;
    at::ScalarType dtype = at::ScalarType::Undefined;

    const Tensor* first(PyObject* o, int64_t dims) {
        if (!THPVariable_Check(o)) return reject();
        const Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.get_device() != c10::cuda::current_device() || !t.is_contiguous() || t.dim() != dims)
            return reject();
        device = t.get_device();
        dtype = t.scalar_type();
        if (dtype != at::kBFloat16 && dtype != at::kFloat) return reject();
        return &t;
    }
    const Tensor* other(PyObject* o, at::ScalarType type, int64_t dims) {
        if (!plain || !THPVariable_Check(o)) return reject();
        const Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.get_device() != device || t.scalar_type() != type || !t.is_contiguous() || t.dim() != dims)
            return reject();
        return &t;
    }
    const Tensor* optional(PyObject* o, at::ScalarType type, int64_t dims) {
        return o == Py_None ? nullptr : other(o, type, dims);
    }
    void require(bool ok) { plain = plain && ok; }
    const Tensor* reject() {
        plain = false;
        return nullptr;
    }
};

bool real(PyObject* o, double* x) {
    *x = PyFloat_AsDouble(o);
    if (*x != -1.0 || !PyErr_Occurred()) return true;
    PyErr_Clear();
    return false;
}
bool whole(PyObject* o, int64_t* x) {
    *x = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
    if (!PyLong_Check(o)) return false;
    if (*x != -1 || !PyErr_Occurred()) return true;
    PyErr_Clear();
    return false;
}

const void* at_of(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
int32_t dtype_of(at::ScalarType t) { return t == at::kBFloat16 ? GDN_BF16 : GDN_F32; }
void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

// inv_freq, q_norm_w, k_norm_w, norm_eps, interleaved, rot_scale from args[0] on.
bool norm_of(PyObject* const* args, int64_t d, Inputs& in, gdn_qk_norm* n) {
    const Tensor *f = in.optional(args[0], at::kFloat, 1), *qw = in.optional(args[1], in.dtype, 1),
                 *kw = in.optional(args[2], in.dtype, 1);
    double eps, scale;
    int64_t il;
    if (!in.plain || !real(args[3], &eps) || !whole(args[4], &il) || !real(args[5], &scale)) return false;
    if ((qw && qw->size(0) != d) || (kw && kw->size(0) != d)) return false;
    *n = gdn_qk_norm{at_of(qw), at_of(kw), static_cast<const float*>(at_of(f)), f ? 2 * f->size(0) : 0, (int32_t)il, (float)eps, (float)scale};
    return true;
}

template <class F>
gdn_status unlocked(F call) {
    gdn_status s;
    Py_BEGIN_ALLOW_THREADS
    s = call();
    Py_END_ALLOW_THREADS
    return s;
}

// Runs a call with a workspace of `need` bytes made here.
template <class A>
gdn_status run(gdn_status (*call)(const A*, void*, size_t, gdn_stream), const A& a, size_t need, const Tensor& like, int device) {
    Tensor ws;
    if (need) ws = at::empty({(int64_t)need}, like.options().dtype(at::kByte));
    void* p = need ? ws.data_ptr() : nullptr;
    return unlocked([&] { return call(&a, p, need, stream_of(device)); });
}

// A tuple of tensors (None for NULL).
PyObject* tuple(std::initializer_list<const Tensor*> x) {
    PyObject* t = PyTuple_New((Py_ssize_t)x.size());
    Py_ssize_t i = 0;
    for (const Tensor* e : x) {
        PyObject* o = t ? (e ? THPVariable_Wrap(*e) : Py_NewRef(Py_None)) : nullptr;
        if (t && !o) Py_CLEAR(t);
        if (t) PyTuple_SET_ITEM(t, i++, o);
    }
    return t;
}

// q, k or None, positions or None, and what norm_of reads, from args[0] on; false if they are not plain.
template <class A>
bool qk_of(PyObject* const* args, Inputs& in, A* a, const Tensor** q, const Tensor** k) {
    if (!(*q = in.first(args[0], 3))) return false;
    *k = in.optional(args[1], in.dtype, 3);
    const Tensor* pos = in.optional(args[2], at::kInt, 1);
    a->T = (*q)->size(0);
    a->Hq = (*q)->size(1);
    a->d = (*q)->size(2);
    if (!norm_of(args + 3, a->d, in, &a->norm)) return false;
    if (*k) in.require((*k)->size(0) == a->T && (*k)->size(2) == a->d);
    if (pos) in.require(pos->size(0) == a->T);
    if (!in.plain) return false;
    a->q = (*q)->data_ptr();
    a->k = at_of(*k);
    a->positions = static_cast<const int32_t*>(at_of(pos));
    a->Hk = *k ? (*k)->size(1) : 0;
    a->dtype = dtype_of(in.dtype);
    return true;
}

// (q, k or None, positions or None, inv_freq, q_norm_w, k_norm_w, norm_eps, interleaved, rot_scale) -> (q_out, k_out)
PyObject* qk_norm_rope_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9 || !lib.bound) Py_RETURN_NONE;
    Inputs in;
    gdn_qk_fwd_args a{};
    const Tensor *q, *k;
    if (!qk_of(args, in, &a, &q, &k)) Py_RETURN_NONE;
    Tensor qo = at::empty(q->sizes(), q->options()), ko;
    if (k) ko = at::empty(k->sizes(), k->options());
    a.q_out = qo.data_ptr();
    a.k_out = k ? ko.data_ptr() : nullptr;
    const gdn_status s = unlocked([&] { return lib.gdn_qk_norm_rope_fwd(&a, stream_of(in.device)); });
    if (s) return PyLong_FromLong(s);
    return tuple({&qo, k ? &ko : nullptr});
    END_HANDLE_TH_ERRORS
}

// (the forward's nine, grad_q, grad_k or None) -> (dq, dk, dq_norm_w, dk_norm_w), None for those that do not apply
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 11 || !lib.bound) Py_RETURN_NONE;
    Inputs in;
    gdn_qk_bwd_args a{};
    const Tensor *q, *k;
    if (!qk_of(args, in, &a, &q, &k)) Py_RETURN_NONE;
    const Tensor *gq = in.other(args[9], in.dtype, 3), *gk = in.optional(args[10], in.dtype, 3);
    if (!in.plain || gq->sizes() != q->sizes() || (k != nullptr) != (gk != nullptr) || (k && gk->sizes() != k->sizes())) Py_RETURN_NONE;
    Tensor dq = at::empty(q->sizes(), q->options()), dk, dqw, dkw;
    const auto f32 = q->options().dtype(at::kFloat);
    if (k) dk = at::empty(k->sizes(), k->options());
    if (a.norm.q_norm_w) dqw = at::empty({a.d}, f32);
    if (a.norm.k_norm_w) dkw = at::empty({a.d}, f32);
    a.grad_q_out = gq->data_ptr();
    a.grad_k_out = at_of(gk);
    a.grad_q = dq.data_ptr();
    a.grad_k = k ? dk.data_ptr() : nullptr;
    a.grad_q_norm_w = a.norm.q_norm_w ? dqw.data_ptr<float>() : nullptr;
    a.grad_k_norm_w = a.norm.k_norm_w ? dkw.data_ptr<float>() : nullptr;
    const gdn_status s = run(lib.gdn_qk_norm_rope_bwd, a, lib.gdn_qk_norm_rope_bwd_workspace_size(&a), dq, in.device);
    if (s) return PyLong_FromLong(s);
    return tuple({&dq, k ? &dk : nullptr, a.norm.q_norm_w ? &dqw : nullptr, a.norm.k_norm_w ? &dkw : nullptr});
    END_HANDLE_TH_ERRORS
}

// q, k, v, cu_seqlens, scale or None, window; false if they are not plain.
template <class A>
bool attn_of(PyObject* qo, PyObject* ko, PyObject* vo, PyObject* cuo, PyObject* scale, PyObject* window, Inputs& in, A* a,
             const Tensor** q, const Tensor** k) {
    if (!(*q = in.first(qo, 3))) return false;
    *k = in.other(ko, in.dtype, 3);
    const Tensor *v = in.other(vo, in.dtype, 3), *cu = in.other(cuo, at::kInt, 1);
    if (!in.plain || cu->size(0) < 1 || (*k)->size(0) != (*q)->size(0) || (*k)->size(2) != (*q)->size(2) || v->sizes() != (*k)->sizes())
        return false;
    double c = 1.0 / std::sqrt((double)(*q)->size(2));
    if ((scale != Py_None && !real(scale, &c)) || !whole(window, &a->window)) return false;
    a->q = (*q)->data_ptr();
    a->k = (*k)->data_ptr();
    a->v = v->data_ptr();
    a->cu_seqlens = static_cast<const int32_t*>(cu->data_ptr());
    a->T = (*q)->size(0);
    a->nseq = cu->size(0) - 1;
    a->Hq = (*q)->size(1);
    a->Hk = (*k)->size(1);
    a->d = (*q)->size(2);
    a->scale = (float)c;
    a->dtype = dtype_of(in.dtype);
    return true;
}
// (q, k, v, cu_seqlens on the device, scale or None, window, bwd_cache or None) -> o
PyObject* attn_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7 || !lib.bound) Py_RETURN_NONE;
    Inputs in;
    gdn_attn_fwd_args a{};
    const Tensor *q, *k;
    if (!attn_of(args[0], args[1], args[2], args[3], args[4], args[5], in, &a, &q, &k)) Py_RETURN_NONE;
    const Tensor* cache = in.optional(args[6], at::kByte, 1);
    if (!in.plain) Py_RETURN_NONE;
    Tensor o = at::empty(q->sizes(), q->options());
    a.o = o.data_ptr();
    a.bwd_cache = cache ? cache->data_ptr() : nullptr;
    a.bwd_cache_bytes = cache ? (size_t)cache->size(0) : 0;
    const gdn_status s = run(lib.gdn_attn_fwd, a, lib.gdn_attn_fwd_workspace_size(&a), o, in.device);
    return s ? PyLong_FromLong(s) : THPVariable_Wrap(o);
    END_HANDLE_TH_ERRORS
}

// (q, k, v, cu_seqlens on the device, scale or None, window, o, grad_o, fwd_cache) -> (dq, dk, dv)
PyObject* attn_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9 || !lib.bound) Py_RETURN_NONE;
    Inputs in;
    gdn_attn_bwd_args a{};
    const Tensor *q, *k;
    if (!attn_of(args[0], args[1], args[2], args[3], args[4], args[5], in, &a, &q, &k)) Py_RETURN_NONE;
    const Tensor *o = in.other(args[6], in.dtype, 3), *go = in.other(args[7], in.dtype, 3), *cache = in.other(args[8], at::kByte, 1);
    if (!in.plain || o->sizes() != q->sizes() || go->sizes() != q->sizes()) Py_RETURN_NONE;
    Tensor dq = at::empty(q->sizes(), q->options()), dk = at::empty(k->sizes(), k->options()), dv = at::empty(k->sizes(), k->options());
    a.o = o->data_ptr();
    a.grad_o = go->data_ptr();
    a.grad_q = dq.data_ptr();
    a.grad_k = dk.data_ptr();
    a.grad_v = dv.data_ptr();
    a.fwd_cache = cache->data_ptr();
    a.fwd_cache_bytes = (size_t)cache->size(0);
    const gdn_status s = run(lib.gdn_attn_bwd, a, lib.gdn_attn_bwd_workspace_size(&a), dq, in.device);
    if (s) return PyLong_FromLong(s);
    return tuple({&dq, &dk, &dv});
    END_HANDLE_TH_ERRORS
}

// The paged cache's arguments; false if they are not plain.
template <class A>
bool cache_of(PyObject* const* args, Inputs& in, int64_t nseq, int64_t Hk, int64_t d, A* a) {
    const Tensor *kc = in.other(args[0], in.dtype, 4), *vc = in.other(args[1], in.dtype, 4), *tab = in.other(args[2], at::kInt, 2),
                 *ctx = in.other(args[3], at::kInt, 1);
    if (!in.plain || vc->sizes() != kc->sizes() || kc->size(2) != Hk || kc->size(3) != d || tab->size(0) != nseq || ctx->size(0) != nseq)
        return false;
    a->k_cache = kc->data_ptr();
    a->v_cache = vc->data_ptr();
    a->block_table = static_cast<const int32_t*>(tab->data_ptr());
    a->context_lens = static_cast<const int32_t*>(ctx->data_ptr());
    a->num_pages = kc->size(0);
    a->page_size = kc->size(1);
    a->max_pages = tab->size(1);
    return true;
}

// (k, v, k_cache, v_cache, block_table, context_lens, cu_seqlens on the device or None, q or None, inv_freq, q_norm_w,
// k_norm_w, norm_eps, interleaved, rot_scale, want_k) -> (q_out, k_out)
PyObject* kv_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 15 || !lib.bound) Py_RETURN_NONE;
    Inputs in;
    const Tensor* k = in.first(args[0], 3);
    if (!k) Py_RETURN_NONE;
    const Tensor *v = in.other(args[1], in.dtype, 3), *cu = in.optional(args[6], at::kInt, 1), *q = in.optional(args[7], in.dtype, 3);
    gdn_kv_append_args a{};
    a.T = k->size(0);
    a.Hk = k->size(1);
    a.d = k->size(2);
    if (!in.plain || v->sizes() != k->sizes() || (cu && cu->size(0) < 1) || (q && (q->size(0) != a.T || q->size(2) != a.d)))
        Py_RETURN_NONE;
    a.nseq = cu ? cu->size(0) - 1 : a.T;
    const int want_k = PyObject_IsTrue(args[14]);
    if (want_k < 0) return nullptr;
    if (!cache_of(args + 2, in, a.nseq, a.Hk, a.d, &a) || !norm_of(args + 8, a.d, in, &a.norm)) Py_RETURN_NONE;
    Tensor qo, ko;
    if (q) qo = at::empty(q->sizes(), q->options());
    if (want_k) ko = at::empty(k->sizes(), k->options());
    a.q = at_of(q);
    a.k = k->data_ptr();
    a.v = v->data_ptr();
    a.cu_seqlens = static_cast<const int32_t*>(at_of(cu));
    a.q_out = q ? qo.data_ptr() : nullptr;
    a.k_out = want_k ? ko.data_ptr() : nullptr;
    a.Hq = q ? q->size(1) : 0;
    a.dtype = dtype_of(in.dtype);
    const gdn_status s = unlocked([&] { return lib.gdn_kv_append(&a, stream_of(in.device)); });
    if (s) return PyLong_FromLong(s);
    return tuple({q ? &qo : nullptr, want_k ? &ko : nullptr});
    END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, block_table, context_lens, scale or None, window, max_context) -> o
PyObject* attn_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 8 || !lib.bound) Py_RETURN_NONE;
    Inputs in;
    const Tensor* q = in.first(args[0], 3);
    if (!q || !THPVariable_Check(args[1]) || THPVariable_Unpack(args[1]).dim() != 4) Py_RETURN_NONE;
    gdn_attn_decode_args a{};
    a.N = q->size(0);
    a.Hq = q->size(1);
    a.Hk = THPVariable_Unpack(args[1]).size(2);
    a.d = q->size(2);
    double scale = 1.0 / std::sqrt((double)a.d);
    if (!cache_of(args + 1, in, a.N, a.Hk, a.d, &a) || (args[5] != Py_None && !real(args[5], &scale)) ||
        !whole(args[6], &a.window) || !whole(args[7], &a.max_context))
        Py_RETURN_NONE;
    Tensor o = at::empty(q->sizes(), q->options());
    a.q = q->data_ptr();
    a.o = o.data_ptr();
    a.scale = (float)scale;
    a.dtype = dtype_of(in.dtype);
    const gdn_status s = run(lib.gdn_attn_decode, a, lib.gdn_attn_decode_workspace_size(&a), o, in.device);
    return s ? PyLong_FromLong(s) : THPVariable_Wrap(o);
    END_HANDLE_TH_ERRORS
}

// ({name: address} of every entry point) -> None
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 1 || !PyDict_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "bind takes the entry points' addresses by name");
        return nullptr;
    }
    Entries e;
#define X(f)                                                                        \
    {                                                                               \
        PyObject* o = PyDict_GetItemString(args[0], #f); /* borrowed */             \
        void* p = o && PyLong_Check(o) ? PyLong_AsVoidPtr(o) : nullptr;             \
        if (!p) {                                                                   \
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, #f);             \
            return nullptr;                                                         \
        }                                                                           \
        e.f = reinterpret_cast<decltype(e.f)>(p);                                   \
    }
    GDN_ENTRIES(X)
#undef X
    e.bound = true;
    lib = e;
    Py_RETURN_NONE;
}

// The names that bind takes.
PyObject* entries(PyObject*, PyObject* const*, Py_ssize_t) {
    const char* names[] = {
#define X(f) #f,
        GDN_ENTRIES(X)
#undef X
    };
    constexpr Py_ssize_t count = sizeof(names) / sizeof(names[0]);
    PyObject* t = PyTuple_New(count);
    for (Py_ssize_t i = 0; t && i < count; ++i) {
        PyObject* o = PyUnicode_FromString(names[i]);
        if (!o) Py_CLEAR(t);
        else PyTuple_SET_ITEM(t, i, o);
    }
    return t;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<qk_norm_rope_fwd>("qk_norm_rope_fwd"), method<qk_norm_rope_bwd>("qk_norm_rope_bwd"),
                         method<attn_fwd>("attn_fwd"), method<attn_bwd>("attn_bwd"), method<kv_append>("kv_append"),
                         method<attn_decode>("attn_decode"), method<bind>("bind"), method<entries>("entries"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_calls(void) { return PyModule_Create(&module); }
