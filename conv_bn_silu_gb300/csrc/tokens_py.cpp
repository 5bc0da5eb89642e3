// tokens_py.cpp -- the token operators' calls from Python: checks of tensors,
// the outputs' allocation and the C ABI's call in one step, since a
// single-token step is as long as its calls' host time (on the Arm host a call
// through ctypes took 11 to 24 us, its kernel 1 to 15).  Argument marshalling
// only: the computing calls are those of include/cbs.h.
//
// A call returns its tensors, or the (negative) status of the C call; what a
// tensor is not fit for raises ValueError here.
#include <Python.h>

#include <initializer_list>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/cbs.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused {};   // a Python error is set

[[noreturn]] void refuse(const char *name, const char *why) {
    PyErr_Format(PyExc_ValueError, "%s: %s", name, why);
    throw Refused{};
}

// A CUDA tensor, on the device of `like` if one is given: addresses of another
// device's memory must not reach a kernel.
const Tensor &tensor(PyObject *o, const char *name, const Tensor *like = nullptr) {
    if (!THPVariable_Check(o)) refuse(name, "expected a CUDA tensor");
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(name, "expected a CUDA tensor");
    if (like && t.device() != like->device()) refuse(name, "on another device");
    return t;
}

// A contiguous tensor of a type and shape (-1: any extent).
const Tensor &dense(PyObject *o, const char *name, const Tensor *like, ScalarType type, std::initializer_list<int64_t> shape) {
    const Tensor &t = tensor(o, name, like);
    if (t.scalar_type() != type) refuse(name, "unexpected type");
    if (!t.is_contiguous()) refuse(name, "not contiguous");
    if (t.dim() != (int64_t)shape.size()) refuse(name, "unexpected number of dimensions");
    int64_t d = 0;
    for (const int64_t n : shape) {
        if (n >= 0 && t.size(d) != n) refuse(name, "unexpected shape");
        if (t.size(d) > INT_MAX) refuse(name, "over 2^31 in one dimension");
        ++d;
    }
    return t;
}

bool is_float(ScalarType t) { return t == ScalarType::Float || t == ScalarType::BFloat16; }
int prec(ScalarType t) { return t == ScalarType::Float ? CBS_FP32 : t == ScalarType::BFloat16 ? CBS_BF16 : CBS_INT8; }

// Elements between the tokens of [tokens, heads, head_dim], which may be a slice
// of a fused product's rows.
int64_t token_stride(const Tensor &t, const char *name, ScalarType type, int heads, int head_dim) {
    if (t.scalar_type() != type) refuse(name, "unexpected type");
    if (t.dim() != 3 || t.size(1) != heads || t.size(2) != head_dim || t.size(0) > INT_MAX)
        refuse(name, "expected (tokens, heads, head_dim) of the cache");
    if (t.stride(2) != 1 || (t.stride(1) != head_dim && heads != 1)) refuse(name, "a token's values are not contiguous");
    return t.size(0) > 1 ? t.stride(0) : (int64_t)heads * head_dim;
}

void *stream_of(const Tensor &t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }
Tensor empty(at::IntArrayRef shape, ScalarType type, const Tensor &like) {   // (past the dispatcher, which takes as long again)
    return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
void *pointer(PyObject *o) {
    void *p = o == Py_None ? nullptr : PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Refused{};
    return p;
}
long integer(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}
bool flag(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}
// The device of a layer's or a cache's own arrays, which their owner has checked.
void at_home(const Tensor &t, const char *name, PyObject *device) {
    if (t.get_device() != integer(device)) refuse(name, "not on the device of the layer or cache");
}
PyObject *status(cbs_status s) { return PyLong_FromLong(s); }
PyObject *none() { Py_RETURN_NONE; }
PyObject *triple(PyObject *a, PyObject *b, PyObject *c) {
    PyObject *r = PyTuple_Pack(3, a, b, c);
    Py_DECREF(a);
    Py_DECREF(b);
    Py_DECREF(c);
    return r;
}

// The sequences of a call, their arrays checked.
cbs_sequences sequences(PyObject *starts, PyObject *lens, PyObject *table, int64_t total, const Tensor *like) {
    const Tensor &t = dense(table, "page_table", like, ScalarType::Int, {-1, -1});
    const Tensor &n = dense(lens, "seq_lens", &t, ScalarType::Int, {t.size(0)});
    const Tensor *s0 = starts == Py_None ? nullptr : &dense(starts, "new_start", &t, ScalarType::Int, {t.size(0) + 1});
    cbs_sequences s;
    s.batch = (int)t.size(0);
    s.max_pages = (int)t.size(1);
    s.total = (int)total;
    s.page_table = t.data_ptr<int>();
    s.seq_lens = n.data_ptr<int>();
    s.new_start = s0 ? s0->data_ptr<int>() : nullptr;
    return s;
}

// rmsnorm(x, weight, eps, residual, int8, h_out) -> (y, scale, h)
PyObject *rmsnorm(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x");
    if (!is_float(x.scalar_type())) refuse("x", "expected float32 or bfloat16");
    dense(a[0], "x", nullptr, x.scalar_type(), {-1, -1});
    const int64_t rows = x.size(0), cols = x.size(1);
    const Tensor &w = dense(a[1], "weight", &x, ScalarType::Float, {cols});
    const double eps = PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred()) throw Refused{};
    const bool int8 = flag(a[4]);
    const Tensor *residual = a[3] == Py_None ? nullptr : &dense(a[3], "residual", &x, x.scalar_type(), {rows, cols});
    if (!residual && a[5] != Py_None) refuse("h_out", "without a residual it is x itself");
    Tensor h;
    if (a[5] != Py_None) h = dense(a[5], "h_out", &x, x.scalar_type(), {rows, cols});
    const c10::cuda::CUDAGuard guard(x.device());
    if (residual && !h.defined()) h = empty({rows, cols}, x.scalar_type(), x);
    Tensor y = empty({rows, cols}, int8 ? ScalarType::Char : x.scalar_type(), x), scale;
    if (int8) scale = empty({rows}, ScalarType::Float, x);
    const cbs_status s = cbs_rmsnorm(x.data_ptr(), residual ? residual->data_ptr() : nullptr, w.data_ptr<float>(),
                                     h.defined() ? h.data_ptr() : nullptr, y.data_ptr(), int8 ? scale.data_ptr<float>() : nullptr,
                                     (int)rows, (int)cols, (float)eps, prec(x.scalar_type()), prec(y.scalar_type()), stream_of(x));
    if (s != CBS_OK) return status(s);
    PyObject *h_py = !residual ? Py_NewRef(a[0]) : a[5] != Py_None ? Py_NewRef(a[5]) : THPVariable_Wrap(h);
    return triple(THPVariable_Wrap(y), int8 ? THPVariable_Wrap(scale) : none(), h_py);
}

// dequantize_rows(q, scale, bf16) -> out
PyObject *dequantize_rows(PyObject *const *a) {
    const Tensor &q = dense(a[0], "q", nullptr, ScalarType::Char, {-1, -1});
    const Tensor &scale = dense(a[1], "scale", &q, ScalarType::Float, {q.size(0)});
    const ScalarType type = flag(a[2]) ? ScalarType::BFloat16 : ScalarType::Float;
    const c10::cuda::CUDAGuard guard(q.device());
    Tensor out = empty(q.sizes(), type, q);
    const cbs_status s = cbs_dequantize_rows(q.data_ptr<int8_t>(), scale.data_ptr<float>(), out.data_ptr(), (int)q.size(0),
                                             (int)q.size(1), prec(out.scalar_type()), stream_of(q));
    return s != CBS_OK ? status(s) : THPVariable_Wrap(out);
}

// linear_w4(x, x_scale, out, bf16, device, n, k, group, activation, w, scales, zeros, bias) -> out;
// the layer's own arrays as addresses (their owner has checked and keeps them)
PyObject *linear_w4(PyObject *const *a) {
    const Tensor &x = tensor(a[0], "x");
    const bool int8 = x.scalar_type() == ScalarType::Char;
    if (!int8 && x.scalar_type() != ScalarType::BFloat16) refuse("x", "expected bfloat16 or int8");
    const int n = (int)integer(a[5]), k = (int)integer(a[6]);
    dense(a[0], "x", nullptr, x.scalar_type(), {-1, k});
    at_home(x, "x", a[4]);
    const int64_t rows = x.size(0);
    if ((a[1] != Py_None) != int8) refuse("x_scale", "with int8 inputs, and only with them");
    const Tensor *x_scale = int8 ? &dense(a[1], "x_scale", &x, ScalarType::Float, {rows}) : nullptr;
    Tensor out;
    if (a[2] != Py_None) {
        out = tensor(a[2], "out");
        if (!is_float(out.scalar_type())) refuse("out", "expected float32 or bfloat16");
        dense(a[2], "out", &x, out.scalar_type(), {rows, n});
    }
    const c10::cuda::CUDAGuard guard(x.device());
    if (!out.defined()) out = empty({rows, n}, flag(a[3]) ? ScalarType::BFloat16 : ScalarType::Float, x);
    const cbs_status s = cbs_linear_w4(x.data_ptr(), prec(x.scalar_type()), int8 ? x_scale->data_ptr<float>() : nullptr,
                                       pointer(a[9]), pointer(a[10]), pointer(a[11]), static_cast<const float *>(pointer(a[12])),
                                       out.data_ptr(), prec(out.scalar_type()), (int)rows, n, k, (int)integer(a[7]),
                                       (int)integer(a[8]), stream_of(x));
    if (s != CBS_OK) return status(s);
    return a[2] != Py_None ? Py_NewRef(a[2]) : THPVariable_Wrap(out);
}

// linear_w8(x, x_scale, out, bf16, device, n, k, activation, w, w_scale, bias) -> out; the
// layer's own arrays as addresses
PyObject *linear_w8(PyObject *const *a) {
    const int n = (int)integer(a[5]), k = (int)integer(a[6]);
    const Tensor &x = dense(a[0], "x", nullptr, ScalarType::Char, {-1, k});
    at_home(x, "x", a[4]);
    const int64_t rows = x.size(0);
    const Tensor &x_scale = dense(a[1], "x_scale", &x, ScalarType::Float, {rows});
    Tensor out;
    if (a[2] != Py_None) {
        out = tensor(a[2], "out");
        if (!is_float(out.scalar_type())) refuse("out", "expected float32 or bfloat16");
        dense(a[2], "out", &x, out.scalar_type(), {rows, n});
    }
    const c10::cuda::CUDAGuard guard(x.device());
    if (!out.defined()) out = empty({rows, n}, flag(a[3]) ? ScalarType::BFloat16 : ScalarType::Float, x);
    const cbs_status s = cbs_linear_w8(x.data_ptr<int8_t>(), x_scale.data_ptr<float>(), static_cast<const int8_t *>(pointer(a[8])),
                                       static_cast<const float *>(pointer(a[9])), static_cast<const float *>(pointer(a[10])),
                                       out.data_ptr(), prec(out.scalar_type()), (int)rows, n, k, (int)integer(a[7]), stream_of(x));
    if (s != CBS_OK) return status(s);
    return a[2] != Py_None ? Py_NewRef(a[2]) : THPVariable_Wrap(out);
}

// cache_write(cache, device, k, v, new_start, seq_lens, page_table)
PyObject *cache_write(PyObject *const *a) {
    const auto *c = static_cast<const cbs_cache *>(pointer(a[0]));
    const Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v", &k);
    at_home(k, "k", a[1]);
    if (!is_float(k.scalar_type())) refuse("k", "expected float32 or bfloat16");
    const int64_t ks = token_stride(k, "k", k.scalar_type(), c->kv_heads, c->head_dim);
    const int64_t vs = token_stride(v, "v", k.scalar_type(), c->kv_heads, c->head_dim);
    if (k.size(0) != v.size(0)) refuse("v", "expected the tokens of k");
    const cbs_sequences seqs = sequences(a[4], a[5], a[6], k.size(0), &k);
    const c10::cuda::CUDAGuard guard(k.device());
    const cbs_status s = cbs_cache_write(c, &seqs, k.data_ptr(), ks, v.data_ptr(), vs, prec(k.scalar_type()), stream_of(k));
    if (s != CBS_OK) return status(s);
    Py_RETURN_NONE;
}

// cache_read(cache, device, seq_lens, page_table, max_len, bf16) -> (k, v, None)
PyObject *cache_read(PyObject *const *a) {
    const auto *c = static_cast<const cbs_cache *>(pointer(a[0]));
    const Tensor &like = tensor(a[2], "seq_lens");
    at_home(like, "seq_lens", a[1]);
    const long max_len = integer(a[4]);
    if (max_len < 0 || max_len > INT_MAX) refuse("max_len", "out of range");
    const cbs_sequences seqs = sequences(Py_None, a[2], a[3], 0, &like);
    const c10::cuda::CUDAGuard guard(like.device());
    const ScalarType type = flag(a[5]) ? ScalarType::BFloat16 : ScalarType::Float;
    Tensor k = empty({seqs.batch, max_len, c->kv_heads, c->head_dim}, type, like);
    Tensor v = empty({seqs.batch, max_len, c->kv_heads, c->head_dim}, type, like);
    const cbs_status s = cbs_cache_read(c, &seqs, (int)max_len, k.data_ptr(), v.data_ptr(), prec(type), stream_of(like));
    return s != CBS_OK ? status(s) : triple(THPVariable_Wrap(k), THPVariable_Wrap(v), none());
}

// cache_evict(cache, device, mass, seq_lens, page_table, new_table, keep, recent) -> (kept, new_lens, None)
PyObject *cache_evict(PyObject *const *a) {
    const auto *c = static_cast<const cbs_cache *>(pointer(a[0]));
    const Tensor &mass = dense(a[2], "mass", nullptr, ScalarType::Float, {c->num_pages, c->kv_heads, c->page_size});
    at_home(mass, "mass", a[1]);
    const int64_t batch = dense(a[4], "page_table", &mass, ScalarType::Int, {-1, -1}).size(0);
    const Tensor &table = dense(a[5], "new_table", &mass, ScalarType::Int, {batch, -1});
    const long keep = integer(a[6]), recent = integer(a[7]);
    if (keep < 1 || keep > INT_MAX) refuse("keep", "out of range");
    if (recent < 0 || recent > keep) refuse("recent", "0 to keep");
    const cbs_sequences seqs = sequences(Py_None, a[3], a[4], 0, &mass);
    const c10::cuda::CUDAGuard guard(mass.device());
    Tensor kept = empty({seqs.batch, c->kv_heads, keep}, ScalarType::Int, mass), lens = empty({seqs.batch}, ScalarType::Int, mass);
    const cbs_status s = cbs_cache_evict(c, &seqs, mass.data_ptr<float>(), table.data_ptr<int>(), (int)table.size(1), (int)keep, (int)recent,
                                         kept.data_ptr<int>(), lens.data_ptr<int>(), stream_of(mass));
    return s != CBS_OK ? status(s) : triple(THPVariable_Wrap(kept), THPVariable_Wrap(lens), none());
}

// What the attention calls share: q and out, the sequences, the workspace.
struct Attention {
    const Tensor *q;
    Tensor out;
    int64_t q_stride, out_stride;
    double scale;
    cbs_sequences seqs;
    // The arguments that follow (cache, device, q, new_start, seq_lens, page_table, scale, out).
    // (`more`: checks that come before an address is taken.)
    template <typename More>
    Attention(PyObject *const *a, int heads, More more) {
        const auto *c = static_cast<const cbs_cache *>(pointer(a[0]));
        const int d = c->head_dim;
        q = &tensor(a[2], "q");
        at_home(*q, "q", a[1]);
        q_stride = token_stride(*q, "q", ScalarType::BFloat16, heads, d);
        scale = PyFloat_AsDouble(a[6]);
        if (PyErr_Occurred()) throw Refused{};
        out_stride = (int64_t)heads * d;
        if (a[7] != Py_None) {
            out = tensor(a[7], "out", q);
            out_stride = token_stride(out, "out", ScalarType::BFloat16, heads, d);
            if (out.size(0) != q->size(0)) refuse("out", "expected the tokens of q");
        }
        more(*c);
        seqs = sequences(a[3], a[4], a[5], q->size(0), q);
    }
    void make_out(int heads, int d) {
        if (!out.defined()) out = empty({q->size(0), heads, d}, ScalarType::BFloat16, *q);
    }
    PyObject *result(PyObject *given, cbs_status s) const {
        if (s != CBS_OK) return status(s);
        return given != Py_None ? Py_NewRef(given) : THPVariable_Wrap(out);
    }
};
// A workspace's address.  Used on another stream than its own, its memory is not
// given away before the call has ended.
void *workspace_of(PyObject *o, PyObject *its_stream, const Tensor &like, const c10::cuda::CUDAStream &stream) {
    if (o == Py_None) return nullptr;
    const Tensor &w = tensor(o, "workspace", &like);
    if (stream.stream() != pointer(its_stream)) c10::cuda::CUDACachingAllocator::recordStream(w.storage().data_ptr(), stream);
    return w.data_ptr();
}

// attention(plan, cache, device, q, new_start, seq_lens, page_table, scale, out, workspace, its stream) -> out
PyObject *attention(PyObject *const *a) {
    const auto *p = static_cast<const cbs_attn_plan_t *>(pointer(a[0]));
    const int heads = p->desc.heads;
    Attention t(a + 1, heads, [](const cbs_cache &) {});
    const c10::cuda::CUDAGuard guard(t.q->device());
    t.make_out(heads, p->desc.head_dim);
    const auto stream = c10::cuda::getCurrentCUDAStream(t.q->get_device());
    void *workspace = workspace_of(a[9], a[10], *t.q, stream);
    return t.result(a[8], cbs_paged_attention(p, static_cast<const cbs_cache *>(pointer(a[1])), &t.seqs, t.q->data_ptr(), t.q_stride,
                                              (float)t.scale, t.out.data_ptr(), t.out_stride, workspace, p->workspace_bytes, stream.stream()));
}

// weighed_attention(plan, cache, device, q, new_start, seq_lens, page_table, scale, out, workspace, its stream, mass, decay) -> out
PyObject *weighed_attention(PyObject *const *a) {
    const auto *p = static_cast<const cbs_weighed_plan_t *>(pointer(a[0]));
    const int heads = p->attention.desc.heads;
    const double decay = PyFloat_AsDouble(a[12]);
    if (PyErr_Occurred()) throw Refused{};
    const Tensor *mass = nullptr;
    Attention t(a + 1, heads, [&](const cbs_cache &c) {
        mass = &dense(a[11], "mass", &tensor(a[3], "q"), ScalarType::Float, {c.num_pages, c.kv_heads, c.page_size});
    });
    const c10::cuda::CUDAGuard guard(t.q->device());
    t.make_out(heads, p->attention.desc.head_dim);
    const auto stream = c10::cuda::getCurrentCUDAStream(t.q->get_device());
    void *workspace = workspace_of(a[9], a[10], *t.q, stream);
    return t.result(a[8], cbs_weighed_attention(p, static_cast<const cbs_cache *>(pointer(a[1])), &t.seqs, t.q->data_ptr(), t.q_stride,
                                                (float)t.scale, t.out.data_ptr(), t.out_stride, mass->data_ptr<float>(), (float)decay,
                                                workspace, p->workspace_bytes, stream.stream()));
}

// shared_attention(plan, cache, device, q, new_start, seq_lens, page_table, scale, out, workspace, its stream, group_start,
// prefix_lens, prefix_table) -> out
PyObject *shared_attention(PyObject *const *a) {
    const auto *p = static_cast<const cbs_shared_plan_t *>(pointer(a[0]));
    const int heads = p->desc.heads;
    const Tensor *starts = nullptr, *lens = nullptr, *table = nullptr;
    Attention t(a + 1, heads, [&](const cbs_cache &) {
        const Tensor &q = tensor(a[3], "q");
        table = &dense(a[13], "prefix_table", &q, ScalarType::Int, {-1, -1});
        lens = &dense(a[12], "prefix_lens", &q, ScalarType::Int, {table->size(0)});
        starts = &dense(a[11], "group_start", &q, ScalarType::Int, {table->size(0) + 1});
    });
    const cbs_prefixes prefixes = {starts->data_ptr<int>(), lens->data_ptr<int>(), table->data_ptr<int>(), (int)table->size(0),
                                   (int)table->size(1)};
    const c10::cuda::CUDAGuard guard(t.q->device());
    t.make_out(heads, p->desc.head_dim);
    const auto stream = c10::cuda::getCurrentCUDAStream(t.q->get_device());
    void *workspace = workspace_of(a[9], a[10], *t.q, stream);
    return t.result(a[8], cbs_shared_attention(p, static_cast<const cbs_cache *>(pointer(a[1])), &t.seqs, &prefixes, t.q->data_ptr(),
                                               t.q_stride, (float)t.scale, t.out.data_ptr(), t.out_stride, workspace, p->workspace_bytes,
                                               stream.stream()));
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused &) {
        return nullptr;
    } catch (...) {   // PyTorch's own, as from its own calls: an allocation that failed, for one
        if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

#define CBS_PY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CBS_PY(rmsnorm, 6),     CBS_PY(dequantize_rows, 3), CBS_PY(linear_w4, 13), CBS_PY(cache_write, 7),
                         CBS_PY(cache_read, 6), CBS_PY(attention, 11),       CBS_PY(cache_evict, 8),
                         CBS_PY(linear_w8, 11),  CBS_PY(weighed_attention, 13), CBS_PY(shared_attention, 14), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tokens", "The token operators' calls (see tokens.py).", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tokens() { return PyModule_Create(&module); }
