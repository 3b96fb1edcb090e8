// binding.cpp -- Python entry points of the decode step's operators between
// its GEMVs.  They do what the package's ctypes calls do -- read addresses,
// shapes and strides off the tensors, check them, take the current stream
// and call the C ABI -- but in compiled code: these calls' kernels take 2 to
// 6 us for a few tokens, and marshalling them in Python took 8 to 11 us a
// call on top of the 4 us of the launch.
//
// A function returns its result, or the status code (an int) of a refused
// call; tensors of a wrong shape or type raise ValueError, a result that does
// not fit the device torch's OutOfMemoryError, as from the package's other calls.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <stdexcept>

#include "../../include/qgemv.h"

namespace {

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

inline void need(bool ok, const char *what)
{
    if (!ok) throw Refused(what);
}

// The tensor of an argument, nullptr for None.
const at::Tensor *tensor(PyObject *o, const char *what)
{
    if (o == Py_None) return nullptr;
    need(THPVariable_Check(o), what);
    const at::Tensor &t = THPVariable_Unpack(o);
    need(t.is_cuda(), what);
    return &t;
}

// A structure of the C ABI where the Python object keeps it (a ctypes
// structure's buffer, held during the call), nullptr for None.  An address
// kept beside the object instead would outlive it in the object's copies.
template <typename S>
class Structure {
public:
    Structure(PyObject *o, const char *what)
    {
        if (o == Py_None) return;
        if (PyObject_GetBuffer(o, &view_, PyBUF_SIMPLE) != 0) {
            PyErr_Clear();
            throw Refused(what);
        }
        if (view_.len != static_cast<Py_ssize_t>(sizeof(S)) || reinterpret_cast<uintptr_t>(view_.buf) % alignof(S)) {
            PyBuffer_Release(&view_);
            throw Refused(what);
        }
    }
    ~Structure()
    {
        if (view_.buf) PyBuffer_Release(&view_);
    }
    Structure(const Structure &) = delete;
    Structure &operator=(const Structure &) = delete;
    const S *get() const { return static_cast<const S *>(view_.buf); }

private:
    Py_buffer view_ = {};
};

// The handle of a stream argument (an integer).
void *handle(PyObject *o)
{
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refused("a stream's handle");
    return p;
}

qgemv_stream_t stream_of(PyObject *o, const at::Tensor &t)
{
    if (o == Py_None)
        return reinterpret_cast<qgemv_stream_t>(c10::cuda::getCurrentCUDAStream(t.device().index()).stream());
    return reinterpret_cast<qgemv_stream_t>(handle(o));
}

qgemv_dtype type_of(const at::Tensor &t, const char *what)
{
    switch (t.scalar_type()) {
    case at::kFloat: return QGEMV_F32;
    case at::kHalf: return QGEMV_F16;
    case at::kBFloat16: return QGEMV_BF16;
    default: throw Refused(what);
    }
}

at::ScalarType scalar_of(qgemv_dtype t)
{
    return t == QGEMV_F32 ? at::kFloat : t == QGEMV_F16 ? at::kHalf : at::kBFloat16;
}

const int32_t *int32s(const at::Tensor *t, int64_t n, const char *what)
{
    if (!t) return nullptr;
    need(t->scalar_type() == at::kInt && t->is_contiguous() && t->numel() >= n, what);
    return t->const_data_ptr<int32_t>();
}

// [tokens][heads][head_dim] with contiguous, adjacent heads; the token stride.
int64_t heads(const at::Tensor &t, const char *what)
{
    need(t.dim() == 3 && t.stride(2) == 1 && (t.size(1) == 1 || t.stride(1) == t.size(2)), what);
    return t.stride(0);
}

// A new contiguous tensor beside another (without a way through the
// dispatcher: it is a third of a call), from the memory of the stream that
// the call runs on: a block that the current stream has just let go may still
// be in use there.
at::Tensor beside(const at::Tensor &t, at::IntArrayRef sizes, at::ScalarType type, PyObject *stream)
{
    if (stream == Py_None) return at::detail::empty_cuda(sizes, type, t.device(), std::nullopt);
    const c10::cuda::CUDAStreamGuard there(
        c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle(stream)), t.device().index()));
    return at::detail::empty_cuda(sizes, type, t.device(), std::nullopt);
}

void raise_out_of_memory(const char *what)
{
    PyObject *torch = PyImport_ImportModule("torch");
    PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, what);
    Py_XDECREF(type);
    Py_XDECREF(torch);
}

template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f) noexcept
{
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused &e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        raise_out_of_memory(e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// rope_kv(plan, q, k, v, pos, slots, cache, out, stream) -> out
PyObject *rope_kv(PyObject *, PyObject *const *a, Py_ssize_t n) noexcept
{
    return guarded(n, 9, [&]() -> PyObject * {
        const Structure<qgemv_rope_plan> plan_at(a[0], "rope_kv: plan");
        const Structure<qgemv_kv_cache> cache_at(a[6], "rope_kv: cache");
        const auto *plan = plan_at.get();
        const auto *cache = cache_at.get();
        const at::Tensor *q = tensor(a[1], "rope_kv: q"), *k = tensor(a[2], "rope_kv: k"), *v = tensor(a[3], "rope_kv: v"),
                         *pos = tensor(a[4], "rope_kv: pos"), *slots = tensor(a[5], "rope_kv: slots"),
                         *out = tensor(a[7], "rope_kv: out");
        const at::Tensor *some = q ? q : k;
        need(some && pos && !k == !v, "rope_kv: q, or k and v, and pos");
        need(some->dim() == 3, "rope_kv: [tokens][heads][head_dim]");
        const int64_t tokens = some->size(0), d = some->size(2);
        const qgemv_dtype type = type_of(*some, "rope_kv: fp32, f16 or bf16");
        int64_t qs = 0, ks = 0, vs = 0, os = 0;
        if (k) {
            ks = heads(*k, "rope_kv: k [tokens][heads][head_dim] with adjacent heads");
            vs = heads(*v, "rope_kv: v [tokens][heads][head_dim] with adjacent heads");
            need(cache && slots, "rope_kv: k and v need a cache and slots");
            need(k->sizes() == v->sizes() && k->size(0) == tokens && k->size(1) == cache->n_heads && k->size(2) == d &&
                     k->scalar_type() == some->scalar_type() && v->scalar_type() == some->scalar_type(),
                 "rope_kv: k and v of q's type and tokens, with the cache's heads");
        }
        at::Tensor made;
        if (q) {
            qs = heads(*q, "rope_kv: q [tokens][heads][head_dim] with adjacent heads");
            if (!out) {
                made = beside(*q, q->sizes(), cache ? scalar_of(cache->type) : q->scalar_type(), a[8]);
                out = &made;
            }
            need(out->sizes() == q->sizes(), "rope_kv: out of q's shape");
            os = heads(*out, "rope_kv: out [tokens][heads][head_dim] with adjacent heads");
        }
        const qgemv_status s = qgemv_rope_kv(
            plan, q ? q->const_data_ptr() : nullptr, k ? k->const_data_ptr() : nullptr, v ? v->const_data_ptr() : nullptr,
            type, qs, ks, vs, int32s(pos, tokens, "rope_kv: pos int32 [tokens]"),
            int32s(slots, tokens, "rope_kv: slots int32 [tokens]"), tokens, q ? static_cast<int>(q->size(1)) : 0,
            static_cast<int>(d), q ? out->data_ptr() : nullptr, q ? type_of(*out, "rope_kv: out's type") : QGEMV_F32, os,
            k ? cache : nullptr, stream_of(a[8], *some));
        if (s != QGEMV_OK) return PyLong_FromLong(s);
        if (made.defined()) return THPVariable_Wrap(std::move(made));
        return Py_NewRef(q ? a[7] : Py_None);
    });
}

// Strides between tokens and heads of [n_seqs][n_q][heads][d] or [tokens][heads][d].
void token_strides(const at::Tensor &t, const qgemv_attn_batch &b, int d, int64_t &token, int64_t &head, const char *what)
{
    const int64_t tokens = static_cast<int64_t>(b.n_seqs) * b.n_q;
    if (t.dim() == 4) {
        need(t.size(0) == b.n_seqs && t.size(1) == b.n_q && t.size(2) == b.n_q_heads && t.size(3) == d && t.stride(3) == 1, what);
        // a dimension of size one has no stride of its own
        token = b.n_q > 1 ? t.stride(1) : t.stride(0);
        need(b.n_q == 1 || b.n_seqs == 1 || t.stride(0) == b.n_q * token, what);
        head = t.stride(2);
    } else {
        need(t.dim() == 3 && t.size(0) == tokens && t.size(1) == b.n_q_heads && t.size(2) == d && t.stride(2) == 1, what);
        token = t.stride(0);
        head = t.stride(1);
    }
}

// attn_prefix(q, cache, batch, ws, out, lse, stream) -> out
PyObject *attn_prefix(PyObject *, PyObject *const *a, Py_ssize_t n) noexcept
{
    return guarded(n, 7, [&]() -> PyObject * {
        const Structure<qgemv_kv_cache> cache_at(a[1], "attn_prefix: cache");
        const Structure<qgemv_attn_batch> batch_at(a[2], "attn_prefix: batch");
        const at::Tensor *q = tensor(a[0], "attn_prefix: q"), *ws = tensor(a[3], "attn_prefix: ws"),
                         *out = tensor(a[4], "attn_prefix: out"), *lse = tensor(a[5], "attn_prefix: lse");
        const auto *cache = cache_at.get();
        const auto *batch = batch_at.get();
        need(q && ws && cache && batch, "attn_prefix: q, a batch and its workspace");
        need(type_of(*q, "attn_prefix: q of the cache's type") == cache->type, "attn_prefix: q of the cache's type");
        need(ws->is_contiguous(), "attn_prefix: a contiguous workspace");
        int64_t qt, qh, ot, oh;
        token_strides(*q, *batch, cache->head_dim, qt, qh, "attn_prefix: q and out [n_seqs][n_q][heads][head_dim], evenly spaced");
        at::Tensor made;
        if (!out) {
            made = beside(*q, q->sizes(), q->scalar_type(), a[6]);
            out = &made;
        }
        token_strides(*out, *batch, cache->head_dim, ot, oh, "attn_prefix: q and out [n_seqs][n_q][heads][head_dim], evenly spaced");
        if (lse)
            need(lse->scalar_type() == at::kFloat && lse->is_contiguous() &&
                     lse->numel() == static_cast<int64_t>(batch->n_seqs) * batch->n_q * batch->n_q_heads,
                 "attn_prefix: lse fp32 [tokens][heads]");
        const qgemv_status s = qgemv_attn_prefix(
            q->const_data_ptr(), qt, qh, cache, batch, out->data_ptr(), type_of(*out, "attn_prefix: out's type"), ot, oh,
            lse ? lse->data_ptr<float>() : nullptr, ws->data_ptr(), ws->nbytes(), stream_of(a[6], *q));
        if (s != QGEMV_OK) return PyLong_FromLong(s);
        return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[4]);
    });
}

// logits_rules(x, spec, ws, out, idx, val, stream) -> (idx, val)
PyObject *logits_rules(PyObject *, PyObject *const *a, Py_ssize_t n) noexcept
{
    return guarded(n, 7, [&]() -> PyObject * {
        const Structure<qgemv_logits_spec> spec_at(a[1], "logits_rules: rules");
        const at::Tensor *x = tensor(a[0], "logits_rules: x"), *ws = tensor(a[2], "logits_rules: ws"),
                         *out = tensor(a[3], "logits_rules: out"), *idx = tensor(a[4], "logits_rules: idx"),
                         *val = tensor(a[5], "logits_rules: val");
        const auto *spec = spec_at.get();
        need(x && ws && spec, "logits_rules: x, rules and a workspace");
        need(x->dim() == 2 && x->size(0) == spec->rows && x->size(1) == spec->vocab && x->stride(1) == 1,
             "logits_rules: x [rows][vocab]");
        need(ws->is_contiguous(), "logits_rules: a contiguous workspace");
        if (out)
            need(out->sizes() == x->sizes() && out->stride(1) == 1 && out->scalar_type() == x->scalar_type(),
                 "logits_rules: out of x's shape and type");
        at::Tensor made_idx, made_val;
        if (!idx) made_idx = beside(*x, {spec->rows}, at::kLong, a[6]);
        if (!val) made_val = beside(*x, {spec->rows}, at::kFloat, a[6]);
        if (!idx) idx = &made_idx;
        if (!val) val = &made_val;
        need(idx->scalar_type() == at::kLong && idx->is_contiguous() && idx->numel() == spec->rows &&
                 val->scalar_type() == at::kFloat && val->is_contiguous() && val->numel() == spec->rows,
             "logits_rules: idx int64 and val fp32 [rows]");
        const qgemv_status s = qgemv_logits_rules(
            x->const_data_ptr(), type_of(*x, "logits_rules: fp32, f16 or bf16"), x->stride(0), spec,
            out ? out->data_ptr() : nullptr, out ? out->stride(0) : 0, idx->data_ptr<int64_t>(), val->data_ptr<float>(),
            ws->data_ptr(), ws->nbytes(), stream_of(a[6], *x));
        if (s != QGEMV_OK) return PyLong_FromLong(s);
        PyObject *r = PyTuple_New(2);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, made_idx.defined() ? THPVariable_Wrap(std::move(made_idx)) : Py_NewRef(a[4]));
        PyTuple_SET_ITEM(r, 1, made_val.defined() ? THPVariable_Wrap(std::move(made_val)) : Py_NewRef(a[5]));
        return r;
    });
}

// An argument's tensor on the device of another, nullptr for None.
const at::Tensor *tensor_beside(PyObject *o, const at::Tensor *some, const char *what)
{
    const at::Tensor *t = tensor(o, what);
    need(!t || !some || t->device() == some->device(), what);
    return t;
}

// An array of structures of the C ABI in a Python object's buffer.
template <typename S>
class Structures {
public:
    Structures(PyObject *o, const char *what)
    {
        if (PyObject_GetBuffer(o, &view_, PyBUF_SIMPLE) != 0) {
            PyErr_Clear();
            throw Refused(what);
        }
        if (view_.len == 0 || view_.len % static_cast<Py_ssize_t>(sizeof(S)) ||
            reinterpret_cast<uintptr_t>(view_.buf) % alignof(S)) {
            PyBuffer_Release(&view_);
            throw Refused(what);
        }
    }
    ~Structures() { PyBuffer_Release(&view_); }
    Structures(const Structures &) = delete;
    Structures &operator=(const Structures &) = delete;
    const S *get() const { return static_cast<const S *>(view_.buf); }
    int size() const { return static_cast<int>(view_.len / static_cast<Py_ssize_t>(sizeof(S))); }

private:
    Py_buffer view_ = {};
};

// norm_rope_kv(plan, norm, q, k, v, pos, slots, cache, out, k_out, stream) -> out
PyObject *norm_rope_kv(PyObject *, PyObject *const *a, Py_ssize_t n) noexcept
{
    return guarded(n, 11, [&]() -> PyObject * {
        const Structure<qgemv_rope_plan> plan_at(a[0], "norm_rope_kv: plan");
        const Structure<qgemv_qk_norm> norm_at(a[1], "norm_rope_kv: norm");
        const Structure<qgemv_kv_cache> cache_at(a[7], "norm_rope_kv: cache");
        const auto *cache = cache_at.get();
        const at::Tensor *q = tensor(a[2], "norm_rope_kv: q"), *k = tensor_beside(a[3], q, "norm_rope_kv: k");
        const at::Tensor *some = q ? q : k;
        need(some, "norm_rope_kv: q or k");
        const at::Tensor *v = tensor_beside(a[4], some, "norm_rope_kv: v"), *pos = tensor_beside(a[5], some, "norm_rope_kv: pos"),
                         *slots = tensor_beside(a[6], some, "norm_rope_kv: slots"),
                         *out = tensor_beside(a[8], some, "norm_rope_kv: out"),
                         *k_out = tensor_beside(a[9], some, "norm_rope_kv: k_out");
        need(pos, "norm_rope_kv: pos");
        need(some->dim() == 3, "norm_rope_kv: [tokens][heads][head_dim]");
        const int64_t tokens = some->size(0), d = some->size(2);
        const qgemv_dtype type = type_of(*some, "norm_rope_kv: fp32, f16 or bf16");
        const c10::cuda::CUDAGuard device(some->device());
        int64_t qs = 0, ks = 0, vs = 0, os = 0, kos = 0;
        if (k) {
            ks = heads(*k, "norm_rope_kv: k [tokens][heads][head_dim] with adjacent heads");
            need(k->size(0) == tokens && k->size(2) == d && k->scalar_type() == some->scalar_type(),
                 "norm_rope_kv: k of q's type and tokens");
            if (cache) {
                need(v && slots && !k_out, "norm_rope_kv: with a cache, v and slots, no k_out");
                vs = heads(*v, "norm_rope_kv: v [tokens][heads][head_dim] with adjacent heads");
                need(v->sizes() == k->sizes() && v->scalar_type() == k->scalar_type(), "norm_rope_kv: v of k's shape and type");
            } else {
                need(k_out && !v && !slots && k_out->sizes() == k->sizes(),
                     "norm_rope_kv: without a cache, k_out of k's shape, no v and no slots");
                kos = heads(*k_out, "norm_rope_kv: k_out [tokens][heads][head_dim] with adjacent heads");
            }
        } else {
            need(!v && !k_out, "norm_rope_kv: v and k_out need k");
        }
        at::Tensor made;
        qgemv_dtype q_type = QGEMV_F32;
        if (q) {
            qs = heads(*q, "norm_rope_kv: q [tokens][heads][head_dim] with adjacent heads");
            if (!out) {
                made = beside(*q, q->sizes(), cache ? scalar_of(cache->type) : q->scalar_type(), a[10]);
                out = &made;
            }
            need(out->sizes() == q->sizes(), "norm_rope_kv: out of q's shape");
            os = heads(*out, "norm_rope_kv: out [tokens][heads][head_dim] with adjacent heads");
            q_type = type_of(*out, "norm_rope_kv: out's type");
        }
        const qgemv_status s = qgemv_norm_rope_kv(
            plan_at.get(), norm_at.get(), q ? q->const_data_ptr() : nullptr, k ? k->const_data_ptr() : nullptr,
            k && v ? v->const_data_ptr() : nullptr, type, qs, ks, vs, int32s(pos, tokens, "norm_rope_kv: pos int32 [tokens]"),
            int32s(slots, tokens, "norm_rope_kv: slots int32 [tokens]"), tokens, q ? static_cast<int>(q->size(1)) : 0,
            k ? static_cast<int>(k->size(1)) : 0, static_cast<int>(d), q ? out->data_ptr() : nullptr, q_type, os,
            k_out ? k_out->data_ptr() : nullptr, k_out ? type_of(*k_out, "norm_rope_kv: k_out's type") : QGEMV_F32, kos,
            k ? cache : nullptr, stream_of(a[10], *some));
        if (s != QGEMV_OK) return PyLong_FromLong(s);
        if (made.defined()) return THPVariable_Wrap(std::move(made));
        return Py_NewRef(q ? a[8] : Py_None);
    });
}

// kv8_append(k, v, cache, batch, first, max_new, stream) -> None
PyObject *kv8_append(PyObject *, PyObject *const *a, Py_ssize_t n) noexcept
{
    return guarded(n, 7, [&]() -> PyObject * {
        const Structure<qgemv_kv8_cache> cache_at(a[2], "kv8_append: cache");
        const Structure<qgemv_kv8_batch> batch_at(a[3], "kv8_append: batch");
        const at::Tensor *k = tensor(a[0], "kv8_append: k"), *v = tensor_beside(a[1], k, "kv8_append: v"),
                         *first = tensor_beside(a[4], k, "kv8_append: first");
        const auto *cache = cache_at.get();
        const auto *batch = batch_at.get();
        need(k && v && cache && batch, "kv8_append: k, v and a batch");
        const int64_t ks = heads(*k, "kv8_append: k [tokens][heads][head_dim] with adjacent heads");
        const int64_t vs = heads(*v, "kv8_append: v [tokens][heads][head_dim] with adjacent heads");
        need(k->sizes() == v->sizes() && k->scalar_type() == v->scalar_type() && k->size(1) == cache->n_heads &&
                 k->size(2) == cache->head_dim,
             "kv8_append: k and v of one shape and type, with the cache's heads");
        long most = batch->n_q;
        if (a[5] != Py_None) {
            most = PyLong_AsLong(a[5]);
            need(!(most == -1 && PyErr_Occurred()) && most >= 0 && most <= (1 << 30), "kv8_append: max_new");
        } else if (first) {
            most = std::min<long>(k->size(0), 1 << 30);
        }
        const c10::cuda::CUDAGuard device(k->device());
        const qgemv_status s =
            qgemv_kv8_append(k->const_data_ptr(), v->const_data_ptr(), type_of(*k, "kv8_append: fp32, f16 or bf16"), ks, vs,
                             k->size(0), cache, batch, int32s(first, batch->n_seqs + 1, "kv8_append: first int32 [n_seqs + 1]"),
                             static_cast<int>(most), stream_of(a[6], *k));
        if (s != QGEMV_OK) return PyLong_FromLong(s);
        return Py_NewRef(Py_None);
    });
}

// attn_kv8(q, cache, batch, ws, out, lse, stream) -> out
PyObject *attn_kv8(PyObject *, PyObject *const *a, Py_ssize_t n) noexcept
{
    return guarded(n, 7, [&]() -> PyObject * {
        const Structure<qgemv_kv8_cache> cache_at(a[1], "attn_kv8: cache");
        const Structure<qgemv_kv8_batch> batch_at(a[2], "attn_kv8: batch");
        const at::Tensor *q = tensor(a[0], "attn_kv8: q"), *ws = tensor_beside(a[3], q, "attn_kv8: ws"),
                         *out = tensor_beside(a[4], q, "attn_kv8: out"), *lse = tensor_beside(a[5], q, "attn_kv8: lse");
        const auto *cache = cache_at.get();
        const auto *batch = batch_at.get();
        need(q && ws && cache && batch, "attn_kv8: q, a batch and its workspace");
        need(ws->is_contiguous(), "attn_kv8: a contiguous workspace");
        const qgemv_attn_batch shape = {batch->n_seqs, batch->n_q, batch->n_q_heads, 0, nullptr, nullptr, nullptr, 0, 0, 0.0f};
        const c10::cuda::CUDAGuard device(q->device());
        int64_t qt, qh, ot, oh;
        token_strides(*q, shape, cache->head_dim, qt, qh, "attn_kv8: q and out [n_seqs][n_q][heads][head_dim], evenly spaced");
        at::Tensor made;
        if (!out) {
            made = beside(*q, q->sizes(), q->scalar_type(), a[6]);
            out = &made;
        }
        token_strides(*out, shape, cache->head_dim, ot, oh, "attn_kv8: q and out [n_seqs][n_q][heads][head_dim], evenly spaced");
        if (lse)
            need(lse->scalar_type() == at::kFloat && lse->is_contiguous() &&
                     lse->numel() == static_cast<int64_t>(batch->n_seqs) * batch->n_q * batch->n_q_heads,
                 "attn_kv8: lse fp32 [tokens][heads]");
        const qgemv_status s = qgemv_attn_kv8(
            q->const_data_ptr(), type_of(*q, "attn_kv8: q f16 or bf16"), qt, qh, cache, batch, out->data_ptr(),
            type_of(*out, "attn_kv8: out's type"), ot, oh, lse ? lse->data_ptr<float>() : nullptr, ws->data_ptr(), ws->nbytes(),
            stream_of(a[6], *q));
        if (s != QGEMV_OK) return PyLong_FromLong(s);
        return made.defined() ? THPVariable_Wrap(std::move(made)) : Py_NewRef(a[4]);
    });
}

// beam_select(x, spec, ws, score, token, parent, stream) -> (score, token, parent)
PyObject *beam_select(PyObject *, PyObject *const *a, Py_ssize_t n) noexcept
{
    return guarded(n, 7, [&]() -> PyObject * {
        const Structure<qgemv_beam_spec> spec_at(a[1], "beam_select: step");
        const at::Tensor *x = tensor(a[0], "beam_select: x"), *ws = tensor_beside(a[2], x, "beam_select: ws");
        const auto *spec = spec_at.get();
        need(x && ws && spec, "beam_select: x, a step and a workspace");
        need(x->dim() == 2 && x->size(0) == static_cast<int64_t>(spec->n_groups) * spec->n_beams && x->size(1) == spec->vocab &&
                 (x->size(1) == 1 || x->stride(1) == 1),
             "beam_select: x [groups * beams][vocab]");
        need(ws->is_contiguous(), "beam_select: a contiguous workspace");
        const c10::cuda::CUDAGuard device(x->device());
        const at::ScalarType types[3] = {at::kFloat, at::kLong, at::kInt};
        at::Tensor made[3];
        const at::Tensor *r[3];
        for (int i = 0; i < 3; ++i) {
            r[i] = tensor_beside(a[3 + i], x, "beam_select: score, token and parent");
            if (!r[i]) {
                made[i] = beside(*x, {spec->n_groups, spec->n_best}, types[i], a[6]);
                r[i] = &made[i];
            }
            need(r[i]->scalar_type() == types[i] && r[i]->is_contiguous() &&
                     r[i]->numel() == static_cast<int64_t>(spec->n_groups) * spec->n_best,
                 "beam_select: score fp32, token int64, parent int32 [groups][n_best]");
        }
        const qgemv_status s = qgemv_beam_select(x->const_data_ptr(), type_of(*x, "beam_select: fp32, f16 or bf16"), x->stride(0),
                                                 spec, r[0]->data_ptr<float>(), r[1]->data_ptr<int64_t>(),
                                                 r[2]->data_ptr<int32_t>(), ws->data_ptr(), ws->nbytes(), stream_of(a[6], *x));
        if (s != QGEMV_OK) return PyLong_FromLong(s);
        PyObject *t = PyTuple_New(3);
        if (!t) return nullptr;
        for (int i = 0; i < 3; ++i)
            PyTuple_SET_ITEM(t, i, made[i].defined() ? THPVariable_Wrap(std::move(made[i])) : Py_NewRef(a[3 + i]));
        return t;
    });
}

// fork_pages(caches, eight_bit, parents, lens, pages, fresh, pages_out, lens_out, stream) -> None
PyObject *fork_pages(PyObject *, PyObject *const *a, Py_ssize_t n) noexcept
{
    return guarded(n, 9, [&]() -> PyObject * {
        const bool eight = a[1] == Py_True;
        const at::Tensor *parents = tensor(a[2], "fork_pages: parents"), *lens = tensor_beside(a[3], parents, "fork_pages: lens"),
                         *pages = tensor_beside(a[4], parents, "fork_pages: pages"),
                         *fresh = tensor_beside(a[5], parents, "fork_pages: fresh"),
                         *pages_out = tensor_beside(a[6], parents, "fork_pages: pages_out"),
                         *lens_out = tensor_beside(a[7], parents, "fork_pages: lens_out");
        need(parents && lens && pages && fresh && pages_out && lens_out, "fork_pages: parents, lens, pages, fresh and results");
        const auto table = [](const at::Tensor &t) {
            need(t.dim() == 2 && t.scalar_type() == at::kInt && (t.size(1) == 1 || t.stride(1) == 1),
                 "fork_pages: pages and pages_out int32 [rows][columns]");
        };
        table(*pages);
        table(*pages_out);
        const int64_t most = 1 << 20;
        const int64_t n_out = parents->numel(), n_in = pages->size(0), columns = pages->size(1);
        need(n_out <= most && n_in <= most && columns <= INT32_MAX && pages_out->size(0) == n_out && pages_out->size(1) == columns &&
                 lens->numel() == n_in && fresh->numel() == n_out && lens_out->numel() == n_out,
             "fork_pages: rows of lens and pages, of parents, fresh and the results, columns");
        const qgemv_fork f = {static_cast<int>(n_in),
                              static_cast<int>(n_out),
                              static_cast<int>(columns),
                              int32s(parents, n_out, "fork_pages: parents int32"),
                              int32s(lens, n_in, "fork_pages: lens int32"),
                              pages->const_data_ptr<int32_t>(),
                              pages->stride(0),
                              int32s(fresh, n_out, "fork_pages: fresh int32"),
                              pages_out->data_ptr<int32_t>(),
                              pages_out->stride(0),
                              const_cast<int32_t *>(int32s(lens_out, n_out, "fork_pages: lens_out int32"))};
        const c10::cuda::CUDAGuard device(parents->device());
        qgemv_status s;
        if (eight) {
            const Structures<qgemv_kv8_cache> c(a[0], "fork_pages: caches");
            s = qgemv_fork_pages(&f, nullptr, c.get(), c.size(), stream_of(a[8], *parents));
        } else {
            const Structures<qgemv_kv_cache> c(a[0], "fork_pages: caches");
            s = qgemv_fork_pages(&f, c.get(), nullptr, c.size(), stream_of(a[8], *parents));
        }
        if (s != QGEMV_OK) return PyLong_FromLong(s);
        return Py_NewRef(Py_None);
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t) noexcept>
PyCFunction fast()
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {{"rope_kv", fast<rope_kv>(), METH_FASTCALL, nullptr},
                         {"attn_prefix", fast<attn_prefix>(), METH_FASTCALL, nullptr},
                         {"logits_rules", fast<logits_rules>(), METH_FASTCALL, nullptr},
                         {"norm_rope_kv", fast<norm_rope_kv>(), METH_FASTCALL, nullptr},
                         {"kv8_append", fast<kv8_append>(), METH_FASTCALL, nullptr},
                         {"attn_kv8", fast<attn_kv8>(), METH_FASTCALL, nullptr},
                         {"beam_select", fast<beam_select>(), METH_FASTCALL, nullptr},
                         {"fork_pages", fast<fork_pages>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
