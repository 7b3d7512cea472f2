// Python binding of the softmax layers' operators: checks a call's tensors,
// allocates its outputs and scratch memory, and calls the C ABI.  Nothing is
// computed here.
//
// These are the calls of a decode step, a few microseconds of GPU time each,
// so the host side counts: the same checks written in Python over ctypes took
// 28 to 45 us a call on the Grace host, most of a small call's time.  Each
// function takes positional arguments only (softmax_layer.py gives them names
// and defaults).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <optional>
#include <string>
#include <utility>

#include "lightning_attn.h"

namespace {

using at::Tensor;

struct PythonError {};  // a Python exception is set

[[noreturn]] void refuse(PyObject *type, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
[[noreturn]] void refuse(PyObject *type, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    PyErr_SetString(type, buf);
    throw PythonError();
}

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}
bool none(PyObject *o) { return o == Py_None; }

double number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw PythonError();
    return x;
}
int32_t integer(PyObject *o, const char *name) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) throw PythonError();
    if (x < INT32_MIN || x > INT32_MAX) refuse(PyExc_ValueError, "%s does not fit 32 bits", name);
    return (int32_t)x;
}
// A size as the C ABI's int32; sizes beyond it are refused here.
int32_t size32(int64_t n, const char *name) {
    if (n > INT32_MAX) refuse(PyExc_ValueError, "%s: a size of %lld is too large", name, (long long)n);
    return (int32_t)n;
}

la_dtype dtype_of(const Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return LA_DTYPE_BF16;
    if (t.scalar_type() == at::kFloat) return LA_DTYPE_FP32;
    refuse(PyExc_TypeError, "unsupported dtype %s (bf16 or fp32)", c10::toString(t.scalar_type()));
}

struct Rows {
    void *p = nullptr;
    int64_t stride = 0;
};

// `n` elements of a one-dimensional tensor from `at` on, sharing its storage.
Tensor part_of(const Tensor &t, int64_t at, int64_t n) {
    Tensor p = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW,
                                                        c10::Storage(t.storage()), t.key_set(),
                                                        t.dtype());
    p.unsafeGetTensorImpl()->set_storage_offset(at);
    p.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    return p;
}

// Device, stream and allocations of one call: every tensor is on the first
// one's device, which is current while the call runs; what the call allocates
// belongs to the stream that it is launched on.  Where that is not the caller's current
// one, the allocator is told that the call's stream uses the inputs and the caller's the
// new outputs: neither is handed out again before both streams are done with it.
class Call {
  public:
    Call(PyObject *first, const char *name, PyObject *stream) {
        const Tensor &t = tensor(first, name);
        if (!t.is_cuda())
            refuse(PyExc_ValueError, "%s must be a CUDA tensor (got %s)", name, t.device().str().c_str());
        device_ = t.device();
        guard_.emplace(device_.index());
        const auto current = c10::cuda::getCurrentCUDAStream(device_.index());
        if (none(stream)) {
            stream_ = current.stream();
        } else {
            PyObject *h = PyObject_GetAttrString(stream, "cuda_stream");
            if (!h) throw PythonError();
            void *raw = PyLong_AsVoidPtr(h);
            Py_DECREF(h);
            if (!raw && PyErr_Occurred()) throw PythonError();
            PyObject *d = PyObject_GetAttrString(stream, "device_index");
            if (!d) throw PythonError();
            const long index = PyLong_AsLong(d);
            Py_DECREF(d);
            if (index == -1 && PyErr_Occurred()) throw PythonError();
            if (index != device_.index())
                refuse(PyExc_ValueError, "stream is on device %ld, the tensors on %s", index,
                                          device_.str().c_str());
            stream_ = static_cast<cudaStream_t>(raw);
            if (stream_ != current.stream()) {
                // the null stream has no external handle; it is the default stream
                own_ = raw ? c10::cuda::getStreamFromExternal(stream_, device_.index())
                           : c10::cuda::getDefaultCUDAStream(device_.index());
                on_.emplace(*own_);
                current_ = current;
            }
        }
        used(t);
    }
    void *stream() const { return stream_; }

    const Tensor &here(PyObject *o, const char *name) const {
        const Tensor &t = tensor(o, name);
        if (t.device() != device_)
            refuse(PyExc_ValueError, "%s must be on %s (got %s)", name, device_.str().c_str(),
                                      t.device().str().c_str());
        used(t);
        return t;
    }
    Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
        const Tensor t = at::detail::empty_cuda(shape, type, device_, std::nullopt);
        if (current_) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *current_);
        return t;
    }
    // [tokens, heads, d], each token's heads contiguous, any stride between tokens
    Rows rows(const Tensor &t, const char *name, int64_t tokens, int64_t heads, int64_t d,
              at::ScalarType type) const {
        if (t.scalar_type() != type || t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads ||
            t.size(2) != d)
            refuse(PyExc_ValueError, "%s must be %s of shape (%lld, %lld, %lld)", name,
                                      c10::toString(type), (long long)tokens, (long long)heads,
                                      (long long)d);
        if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))
            refuse(PyExc_ValueError, "%s: the heads of a token must be contiguous", name);
        return {t.data_ptr(), tokens > 1 ? t.stride(0) : heads * d};
    }
    Rows rows(PyObject *o, const char *name, int64_t tokens, int64_t heads, int64_t d,
              at::ScalarType type) const {
        return rows(here(o, name), name, tokens, heads, d, type);
    }
    // An output of that shape: the caller's, or a new one in `made`.
    Rows output(PyObject *o, const char *name, int64_t tokens, int64_t heads, int64_t d,
                at::ScalarType type, Tensor &made) const {
        made = none(o) ? empty({tokens, heads, d}, type) : here(o, name);
        return rows(made, name, tokens, heads, d, type);
    }
    int32_t *ints(PyObject *o, const char *name, int64_t n) const {
        const Tensor &t = here(o, name);
        if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
            refuse(PyExc_ValueError, "%s must be a contiguous int32 tensor of %lld elements", name,
                                      (long long)n);
        return static_cast<int32_t *>(t.data_ptr());
    }
    const float *weight(PyObject *o, const char *name, int64_t d) const {
        if (none(o)) return nullptr;
        const Tensor &t = here(o, name);
        if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != d || !t.is_contiguous())
            refuse(PyExc_ValueError, "%s must be fp32 [%lld]", name, (long long)d);
        return static_cast<const float *>(t.data_ptr());
    }
    // Scratch memory of at least `need` bytes: the caller's or this call's own.
    std::pair<void *, int64_t> workspace(PyObject *o, int64_t need) {
        if (none(o)) {  // freed to the stream's pool when the call returns
            scratch_ = c10::cuda::CUDACachingAllocator::get()->allocate(need);
            return {scratch_.get(), need};
        }
        const Tensor &t = here(o, "workspace");
        if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
        return {t.data_ptr(), (int64_t)t.nbytes()};
    }

  private:
    // A tensor of the caller's, which the call's stream reads or writes.
    void used(const Tensor &t) const {
        if (own_) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *own_);
    }

    at::Device device_{at::kCUDA, 0};
    cudaStream_t stream_ = nullptr;
    // the call's stream and the caller's, where they differ
    std::optional<c10::cuda::CUDAStream> own_, current_;
    std::optional<c10::cuda::CUDAGuard> guard_;
    std::optional<c10::cuda::CUDAStreamGuard> on_;
    c10::DataPtr scratch_;
};

// A tensor of the caller's has been written: autograd checks the version of what it saved.
// (Tensors made in inference mode have none.)
void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(PyObject *o) {
    if (!none(o)) written(THPVariable_Unpack(o));
}

// Raises the package's error for a status that is not LA_OK.
void check(la_status status, const char *name) {
    if (status == LA_OK) return;
    PyObject *mod = PyImport_ImportModule("lightning_attention_attn_gb300");
    PyObject *r = mod ? PyObject_CallMethod(mod, "_check", "is", (int)status, name) : nullptr;
    Py_XDECREF(r);
    Py_XDECREF(mod);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
    throw PythonError();
}

// The call itself, without the interpreter's lock (a full launch queue blocks).
template <typename F> void launch(const char *name, F f) {
    la_status s;
    Py_BEGIN_ALLOW_THREADS;
    s = f();
    Py_END_ALLOW_THREADS;
    check(s, name);
}

struct Shape {
    int32_t tokens, heads, kv_heads, d;
    at::ScalarType type;
    la_dtype code;
};

Shape shape_of(PyObject *q_, PyObject *k_, bool need_k) {
    const Tensor &q = tensor(q_, "q");
    if (q.dim() != 3) refuse(PyExc_ValueError, "q must have three dimensions: [T, H, d]");
    Shape s{size32(q.size(0), "q"), size32(q.size(1), "q"), 0, size32(q.size(2), "q"), q.scalar_type(),
            dtype_of(q)};
    if (need_k || !none(k_)) {
        const Tensor &k = tensor(k_, "k");
        if (k.dim() != 3) refuse(PyExc_ValueError, "k must be [T, Hkv, d]");
        s.kv_heads = size32(k.size(1), "k");
    }
    return s;
}

struct Rotary {
    const int32_t *positions = nullptr;
    const float *table = nullptr;
    int32_t rows = 0, dim = 0, interleaved = 0;
    const float *qw = nullptr, *kw = nullptr;
    float eps = 0;
};

// positions, table | q_weight, k_weight, eps, interleaved
Rotary rotary_of(const Call &call, PyObject *positions, PyObject *table, PyObject *const *norm,
                 const Shape &s) {
    Rotary r;
    if (!none(table)) {
        const Tensor &t = call.here(table, "table");
        if (t.scalar_type() != at::kFloat || t.dim() != 2 || !t.is_contiguous())
            refuse(PyExc_ValueError, "table must be a contiguous fp32 [positions, rotary_dim] tensor");
        r.table = static_cast<const float *>(t.data_ptr());
        r.rows = size32(t.size(0), "table");
        r.dim = size32(t.size(1), "table");
        r.positions = call.ints(positions, "positions", s.tokens);
    } else if (!none(positions)) {
        refuse(PyExc_ValueError, "positions without a rotary table");
    }
    r.qw = call.weight(norm[0], "q_weight", s.d);
    r.kw = call.weight(norm[1], "k_weight", s.d);
    r.eps = (float)number(norm[2]);
    const int flag = PyObject_IsTrue(norm[3]);
    if (flag < 0) throw PythonError();
    r.interleaved = flag;
    return r;
}

struct Cache {
    void *k, *v;
    int64_t ks, vs;
    int32_t pages, page, kv_heads;
};

int64_t page_stride(const Tensor &t, const char *name, int64_t d, at::ScalarType type) {
    if (t.scalar_type() != type || t.dim() != 4 || t.size(3) != d)
        refuse(PyExc_ValueError, "%s must be %s [pages, Hkv, page_size, %lld]", name,
                                  c10::toString(type), (long long)d);
    const int64_t h = t.size(1), page = t.size(2);
    if (t.stride(3) != 1 || (page > 1 && t.stride(2) != d) || (h > 1 && t.stride(1) != page * d))
        refuse(PyExc_ValueError, "%s: a page must be contiguous", name);
    return t.size(0) > 1 ? t.stride(0) : h * page * d;
}

Cache cache_of(const Call &call, PyObject *k_, PyObject *v_, int64_t d, at::ScalarType type) {
    const Tensor &k = call.here(k_, "k_cache"), &v = call.here(v_, "v_cache");
    Cache c;
    c.ks = page_stride(k, "k_cache", d, type);
    c.vs = page_stride(v, "v_cache", d, type);
    if (k.sizes() != v.sizes()) refuse(PyExc_ValueError, "k_cache and v_cache must have one shape");
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.pages = size32(k.size(0), "k_cache");
    c.kv_heads = size32(k.size(1), "k_cache");
    c.page = size32(k.size(2), "k_cache");
    return c;
}

struct Table {
    int32_t *p;
    int32_t stride, width;
};

Table table_of(const Call &call, PyObject *o, int64_t batch) {
    const Tensor &t = call.here(o, "block_table");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != batch)
        refuse(PyExc_ValueError, "block_table must be int32 [%lld, blocks]", (long long)batch);
    if (t.size(1) > 1 && t.stride(1) != 1)
        refuse(PyExc_ValueError, "a row of block_table must be contiguous");
    const int32_t width = size32(t.size(1), "block_table");
    if (batch > 1 && t.stride(0) < width)
        refuse(PyExc_ValueError, "the rows of block_table overlap");
    return {static_cast<int32_t *>(t.data_ptr()),
            batch > 1 ? size32(t.stride(0), "block_table") : width, width};
}

// out and lse of the attention calls.
Tensor attention_out(const Call &call, PyObject *out, const Shape &s) {
    if (none(out)) return call.empty({s.tokens, s.heads, s.d}, s.type);
    const Tensor &t = call.here(out, "out");
    if (t.scalar_type() != s.type || t.dim() != 3 || t.size(0) != s.tokens ||
        t.size(1) != s.heads || t.size(2) != s.d || !t.is_contiguous())
        refuse(PyExc_ValueError, "out must be contiguous, with the shape and dtype of q");
    return t;
}
float *lse_of(const Call &call, PyObject *lse, const Shape &s) {
    if (none(lse)) return nullptr;
    const Tensor &t = call.here(lse, "lse");
    if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != s.tokens ||
        t.size(1) != s.heads || !t.is_contiguous())
        refuse(PyExc_ValueError, "lse must be a contiguous fp32 [%d, %d]", s.tokens, s.heads);
    return static_cast<float *>(t.data_ptr());
}
float scale_of(PyObject *scale, const Shape &s) {
    return none(scale) ? (float)(1.0 / std::sqrt((double)s.d)) : (float)number(scale);
}
int64_t need_of(int64_t n) {
    if (n < 0) refuse(PyExc_ValueError, "head_dim must be 64 or 128");
    return n;
}

PyObject *wrap(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
template <typename... T> PyObject *tuple(const T &...t) {
    PyObject *r = PyTuple_New(sizeof...(t));
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(r, i++, wrap(t)), ...);
    return r;
}

// q, k, positions, table, q_weight, k_weight, eps, interleaved, q_out, k_out, stream
PyObject *qk_norm_rope(PyObject *const *a) {
    Call call(a[0], "q", a[10]);
    const Shape s = shape_of(a[0], a[1], false);
    const bool has_k = !none(a[1]);
    const Rows q = call.rows(a[0], "q", s.tokens, s.heads, s.d, s.type);
    const Rows k = has_k ? call.rows(a[1], "k", s.tokens, s.kv_heads, s.d, s.type) : Rows();
    const Rotary r = rotary_of(call, a[2], a[3], a + 4, s);
    Tensor q_out, k_out;
    const Rows qo = call.output(a[8], "q_out", s.tokens, s.heads, s.d, s.type, q_out);
    const Rows ko = has_k ? call.output(a[9], "k_out", s.tokens, s.kv_heads, s.d, s.type, k_out) : Rows();
    launch("lightning_attn_qk_norm_rope", [&] {
        return lightning_attn_qk_norm_rope(q.p, q.stride, k.p, k.stride, r.positions, r.table, r.rows,
                                           r.dim, r.interleaved, r.qw, r.kw, r.eps, s.tokens, s.heads,
                                           s.kv_heads, s.d, s.code, qo.p, qo.stride, ko.p, ko.stride,
                                           call.stream());
    });
    written(a[8]);
    if (has_k) written(a[9]);
    return tuple(q_out, k_out);
}

// q, k, positions, table, dq_out, dk_out, q_weight, k_weight, eps, interleaved, dq, dk, workspace,
// stream
PyObject *qk_norm_rope_backward(PyObject *const *a) {
    Call call(a[0], "q", a[13]);
    const Shape s = shape_of(a[0], a[1], false);
    const bool has_k = !none(a[1]);
    const Rows q = call.rows(a[0], "q", s.tokens, s.heads, s.d, s.type);
    const Rows dqo = call.rows(a[4], "dq_out", s.tokens, s.heads, s.d, s.type);
    Rows k, dko, dk;
    if (has_k) {
        k = call.rows(a[1], "k", s.tokens, s.kv_heads, s.d, s.type);
        dko = call.rows(a[5], "dk_out", s.tokens, s.kv_heads, s.d, s.type);
    }
    const Rotary r = rotary_of(call, a[2], a[3], a + 6, s);
    Tensor dq_, dk_, dqw, dkw;
    const Rows dq = call.output(a[10], "dq", s.tokens, s.heads, s.d, s.type, dq_);
    if (has_k) dk = call.output(a[11], "dk", s.tokens, s.kv_heads, s.d, s.type, dk_);
    std::pair<void *, int64_t> ws{nullptr, 0};
    if (r.qw) {
        const Tensor both = call.empty({2 * s.d}, at::kFloat);
        dqw = part_of(both, 0, s.d);
        if (has_k) dkw = part_of(both, s.d, s.d);
        ws = call.workspace(a[12], need_of(lightning_attn_qk_norm_rope_workspace_bytes(s.d)));
    }
    launch("lightning_attn_qk_norm_rope_backward", [&] {
        return lightning_attn_qk_norm_rope_backward(
            q.p, q.stride, k.p, k.stride, r.positions, r.table, r.rows, r.dim, r.interleaved, r.qw,
            r.kw, r.eps, s.tokens, s.heads, s.kv_heads, s.d, s.code, dqo.p, dqo.stride, dko.p,
            dko.stride, dq.p, dq.stride, dk.p, dk.stride,
            dqw.defined() ? static_cast<float *>(dqw.data_ptr()) : nullptr,
            dkw.defined() ? static_cast<float *>(dkw.data_ptr()) : nullptr, ws.first, ws.second,
            call.stream());
    });
    written(a[10]);
    if (has_k) written(a[11]);
    return tuple(dq_, dk_, dqw, dkw);
}

// q, k, v, positions, table, k_cache, v_cache, slots, q_weight, k_weight, eps, interleaved, q_out,
// stream
PyObject *paged_append(PyObject *const *a) {
    Call call(a[0], "q", a[13]);
    const Shape s = shape_of(a[0], a[1], true);
    const Rows q = call.rows(a[0], "q", s.tokens, s.heads, s.d, s.type);
    const Rows k = call.rows(a[1], "k", s.tokens, s.kv_heads, s.d, s.type);
    const Rows v = call.rows(a[2], "v", s.tokens, s.kv_heads, s.d, s.type);
    const Rotary r = rotary_of(call, a[3], a[4], a + 8, s);
    const Cache c = cache_of(call, a[5], a[6], s.d, s.type);
    if (c.kv_heads != s.kv_heads) refuse(PyExc_ValueError, "k_cache has %d heads, k %d", c.kv_heads, s.kv_heads);
    const int32_t *slots = call.ints(a[7], "slots", s.tokens);
    Tensor q_out;
    const Rows qo = call.output(a[12], "q_out", s.tokens, s.heads, s.d, s.type, q_out);
    launch("lightning_attn_paged_append", [&] {
        return lightning_attn_paged_append(
            q.p, q.stride, k.p, k.stride, v.p, v.stride, r.positions, r.table, r.rows, r.dim,
            r.interleaved, r.qw, r.kw, r.eps, s.tokens, s.heads, s.kv_heads, s.d, s.code, qo.p,
            qo.stride, c.k, c.ks, c.v, c.vs, slots, c.pages, c.page, call.stream());
    });
    for (int i : {5, 6, 12}) written(a[i]);
    return wrap(q_out);
}

// q, k_cache, v_cache, block_table, seq_lens, scale, out, lse, workspace, stream
PyObject *paged_decode(PyObject *const *a) {
    Call call(a[0], "q", a[9]);
    const Shape s = shape_of(a[0], Py_None, false);
    const Rows q = call.rows(a[0], "q", s.tokens, s.heads, s.d, s.type);
    const Cache c = cache_of(call, a[1], a[2], s.d, s.type);
    const Table t = table_of(call, a[3], s.tokens);
    const int32_t *lens = call.ints(a[4], "seq_lens", s.tokens);
    const float scale = scale_of(a[5], s);
    const Tensor out = attention_out(call, a[6], s);
    float *lse = lse_of(call, a[7], s);
    const auto ws = call.workspace(a[8], need_of(lightning_attn_paged_decode_workspace_bytes(s.d)));
    launch("lightning_attn_paged_decode", [&] {
        return lightning_attn_paged_decode(q.p, q.stride, c.k, c.ks, c.v, c.vs, t.p, t.stride, t.width,
                                           lens, c.pages, c.page, s.tokens, s.heads, c.kv_heads, s.d,
                                           s.code, scale, out.data_ptr(), lse, ws.first, ws.second,
                                           call.stream());
    });
    for (int i : {6, 7}) written(a[i]);
    return wrap(out);
}

// q, k, v, positions, table, k_cache, v_cache, slots, block_table, seq_lens, q_weight, k_weight, eps,
// interleaved, scale, out, lse, workspace, stream
PyObject *paged_step(PyObject *const *a) {
    Call call(a[0], "q", a[18]);
    const Shape s = shape_of(a[0], a[1], true);
    const Rows q = call.rows(a[0], "q", s.tokens, s.heads, s.d, s.type);
    const Rows k = call.rows(a[1], "k", s.tokens, s.kv_heads, s.d, s.type);
    const Rows v = call.rows(a[2], "v", s.tokens, s.kv_heads, s.d, s.type);
    const Rotary r = rotary_of(call, a[3], a[4], a + 10, s);
    const Cache c = cache_of(call, a[5], a[6], s.d, s.type);
    if (c.kv_heads != s.kv_heads) refuse(PyExc_ValueError, "k_cache has %d heads, k %d", c.kv_heads, s.kv_heads);
    const int32_t *slots = call.ints(a[7], "slots", s.tokens);
    const Table t = table_of(call, a[8], s.tokens);
    const int32_t *lens = call.ints(a[9], "seq_lens", s.tokens);
    const float scale = scale_of(a[14], s);
    const Tensor out = attention_out(call, a[15], s);
    float *lse = lse_of(call, a[16], s);
    const auto ws = call.workspace(
        a[17], need_of(lightning_attn_paged_step_workspace_bytes(s.tokens, std::max(s.heads, 1), s.d)));
    launch("lightning_attn_paged_step", [&] {
        return lightning_attn_paged_step(
            q.p, q.stride, k.p, k.stride, v.p, v.stride, r.positions, r.table, r.rows, r.dim,
            r.interleaved, r.qw, r.kw, r.eps, c.k, c.ks, c.v, c.vs, slots, t.p, t.stride, t.width,
            lens, c.pages, c.page, s.tokens, s.heads, s.kv_heads, s.d, s.code, scale,
            out.data_ptr(), lse, ws.first, ws.second, call.stream());
    });
    for (int i : {5, 6, 15, 16}) written(a[i]);
    return wrap(out);
}

// [pages, Hkv, 2, d] of a cache's pages
int64_t bounds_of(const Call &call, PyObject *o, int64_t pages, int64_t kv_heads, int64_t d,
                  at::ScalarType type, void *&p) {
    const Tensor &t = call.here(o, "bounds");
    const int64_t stride = page_stride(t, "bounds", d, type);
    if (t.size(2) != 2 || (pages >= 0 && (t.size(0) != pages || t.size(1) != kv_heads)))
        refuse(PyExc_ValueError, "bounds must be [pages, Hkv, 2, d]");
    p = t.data_ptr();
    return stride;
}

// k_cache, bounds, block_table, first, seq_lens, stream
PyObject *paged_bounds(PyObject *const *a) {
    Call call(a[0], "k_cache", a[5]);
    const Tensor &k = tensor(a[0], "k_cache");
    if (k.dim() != 4) refuse(PyExc_ValueError, "k_cache must be [pages, Hkv, page_size, d]");
    const la_dtype code = dtype_of(k);
    const int64_t d = k.size(3), ks = page_stride(k, "k_cache", d, k.scalar_type());
    const int32_t pages = size32(k.size(0), "k_cache"), heads = size32(k.size(1), "k_cache");
    const int32_t page = size32(k.size(2), "k_cache");
    void *bounds;
    const int64_t bs = bounds_of(call, a[1], pages, heads, d, k.scalar_type(), bounds);
    const Tensor &bt = tensor(a[2], "block_table");
    if (bt.dim() != 2) refuse(PyExc_ValueError, "block_table must be int32 [B, blocks]");
    const int32_t b = size32(bt.size(0), "block_table");
    const Table t = table_of(call, a[2], b);
    const int32_t *first = call.ints(a[3], "first", b), *lens = call.ints(a[4], "seq_lens", b);
    launch("lightning_attn_paged_bounds", [&] {
        return lightning_attn_paged_bounds(k.data_ptr(), ks, bounds, bs, t.p, t.stride, t.width, first, lens,
                                           pages, page, b, heads, size32(d, "k_cache"), code, call.stream());
    });
    written(a[1]);
    return wrap(THPVariable_Unpack(a[1]));
}

// q, bounds, block_table, seq_lens, page_size, count, keep_first, keep_last, out, workspace, stream
PyObject *paged_select(PyObject *const *a) {
    Call call(a[0], "q", a[10]);
    const Shape s = shape_of(a[0], Py_None, false);
    const Rows q = call.rows(a[0], "q", s.tokens, s.heads, s.d, s.type);
    void *bounds;
    const int64_t bs = bounds_of(call, a[1], -1, 0, s.d, s.type, bounds);
    const Tensor &bt = tensor(a[1], "bounds");
    const int32_t pages = size32(bt.size(0), "bounds"), kv = size32(bt.size(1), "bounds");
    const Table t = table_of(call, a[2], s.tokens);
    const int32_t *lens = call.ints(a[3], "seq_lens", s.tokens);
    const int32_t page = integer(a[4], "page_size"), count = integer(a[5], "count");
    const int32_t first = integer(a[6], "keep_first"), last = integer(a[7], "keep_last");
    if (count < 1) refuse(PyExc_ValueError, "count must be at least 1");
    Tensor out;
    if (none(a[8])) {
        out = call.empty({s.tokens, kv, count}, at::kInt);
    } else {
        out = call.here(a[8], "out");
        if (out.scalar_type() != at::kInt || out.dim() != 3 || out.size(0) != s.tokens ||
            out.size(1) != kv || out.size(2) != count || !out.is_contiguous())
            refuse(PyExc_ValueError, "out must be a contiguous int32 [%d, %d, %d]", s.tokens, kv, count);
    }
    const int64_t need = lightning_attn_paged_select_workspace_bytes(s.tokens, std::max(kv, 1), t.width);
    if (need < 0) refuse(PyExc_ValueError, "too many blocks");
    const auto ws = call.workspace(a[9], std::max<int64_t>(need, 16));
    launch("lightning_attn_paged_select", [&] {
        return lightning_attn_paged_select(q.p, q.stride, bounds, bs, t.p, t.stride, t.width, lens, pages,
                                           page, s.tokens, s.heads, kv, s.d, s.code, count, first, last,
                                           static_cast<int32_t *>(out.data_ptr()), ws.first, ws.second,
                                           call.stream());
    });
    written(a[8]);
    return wrap(out);
}

// q, k_cache, v_cache, block_table, seq_lens, selected, scale, out, lse, workspace, stream
PyObject *paged_sparse_decode(PyObject *const *a) {
    Call call(a[0], "q", a[10]);
    const Shape s = shape_of(a[0], Py_None, false);
    const Rows q = call.rows(a[0], "q", s.tokens, s.heads, s.d, s.type);
    const Cache c = cache_of(call, a[1], a[2], s.d, s.type);
    const Table t = table_of(call, a[3], s.tokens);
    const int32_t *lens = call.ints(a[4], "seq_lens", s.tokens);
    const Tensor &sel = call.here(a[5], "selected");
    if (sel.scalar_type() != at::kInt || sel.dim() != 3 || sel.size(0) != s.tokens ||
        sel.size(1) != c.kv_heads || !sel.is_contiguous())
        refuse(PyExc_ValueError, "selected must be a contiguous int32 [%d, %d, count]", s.tokens, c.kv_heads);
    const int32_t count = size32(sel.size(2), "selected");
    const float scale = scale_of(a[6], s);
    const Tensor out = attention_out(call, a[7], s);
    float *lse = lse_of(call, a[8], s);
    const auto ws = call.workspace(a[9], need_of(lightning_attn_paged_decode_workspace_bytes(s.d)));
    launch("lightning_attn_paged_sparse_decode", [&] {
        return lightning_attn_paged_sparse_decode(
            q.p, q.stride, c.k, c.ks, c.v, c.vs, t.p, t.stride, t.width, lens,
            static_cast<const int32_t *>(sel.data_ptr()), count, c.pages, c.page, s.tokens, s.heads,
            c.kv_heads, s.d, s.code, scale, out.data_ptr(), lse, ws.first, ws.second, call.stream());
    });
    for (int i : {7, 8}) written(a[i]);
    return wrap(out);
}

// q, k_cache, v_cache, prefix_table, prefix_len, block_table, seq_lens, scale, out, lse, workspace,
// stream
PyObject *paged_prefix_decode(PyObject *const *a) {
    Call call(a[0], "q", a[11]);
    const Shape s = shape_of(a[0], Py_None, false);
    const Rows q = call.rows(a[0], "q", s.tokens, s.heads, s.d, s.type);
    const Cache c = cache_of(call, a[1], a[2], s.d, s.type);
    const Tensor &front = tensor(a[3], "prefix_table");
    if (front.dim() != 1) refuse(PyExc_ValueError, "prefix_table must be an int32 [blocks] tensor");
    const int32_t width = size32(front.size(0), "prefix_table");
    const int32_t *pages = call.ints(a[3], "prefix_table", width), *len = call.ints(a[4], "prefix_len", 1);
    const Table t = table_of(call, a[5], s.tokens);
    const int32_t *lens = call.ints(a[6], "seq_lens", s.tokens);
    const float scale = scale_of(a[7], s);
    const Tensor out = attention_out(call, a[8], s);
    float *lse = lse_of(call, a[9], s);
    const int64_t need = lightning_attn_paged_prefix_decode_workspace_bytes(s.tokens, s.heads, c.kv_heads,
                                                                            s.d, s.code);
    if (need < 0)
        refuse(PyExc_ValueError, "%d heads over %d key-value heads of %d, batch %d", s.heads, c.kv_heads, s.d,
               s.tokens);
    const auto ws = call.workspace(a[10], need);
    launch("lightning_attn_paged_prefix_decode", [&] {
        return lightning_attn_paged_prefix_decode(
            q.p, q.stride, c.k, c.ks, c.v, c.vs, pages, width, len, t.p, t.stride, t.width, lens, c.pages,
            c.page, s.tokens, s.heads, c.kv_heads, s.d, s.code, scale, out.data_ptr(), lse, ws.first,
            ws.second, call.stream());
    });
    for (int i : {8, 9}) written(a[i]);
    return wrap(out);
}

// block_table, seq_lens, new_lens, free_pages, free_count, page_size, num_tokens, finished,
// seq_lens_out, free_count_out, stream
PyObject *paged_reserve(PyObject *const *a) {
    Call call(a[0], "block_table", a[10]);
    const Tensor &bt = tensor(a[0], "block_table");
    if (bt.dim() != 2) refuse(PyExc_ValueError, "block_table must be int32 [B, blocks]");
    const int32_t b = size32(bt.size(0), "block_table");
    const Table t = table_of(call, a[0], b);
    int32_t *lens = call.ints(a[1], "seq_lens", b), *fresh = call.ints(a[2], "new_lens", b);
    const Tensor &stack = tensor(a[3], "free_pages");
    if (stack.dim() != 1) refuse(PyExc_ValueError, "free_pages must be an int32 [pages] tensor");
    const int32_t pages = size32(stack.size(0), "free_pages");
    int32_t *free_pages = call.ints(a[3], "free_pages", pages);
    int32_t *count = call.ints(a[4], "free_count", 1);
    const int32_t page = integer(a[5], "page_size"), tokens = integer(a[6], "num_tokens");
    if (tokens < 0) refuse(PyExc_ValueError, "num_tokens < 0");
    const uint8_t *finished = nullptr;
    if (!none(a[7])) {
        const Tensor &f = call.here(a[7], "finished");
        if ((f.scalar_type() != at::kBool && f.scalar_type() != at::kByte) || f.dim() != 1 ||
            f.size(0) != b || !f.is_contiguous())
            refuse(PyExc_ValueError, "finished must be a contiguous bool tensor of %d elements", b);
        finished = static_cast<const uint8_t *>(f.data_ptr());
    }
    int32_t *lens_out = none(a[8]) ? lens : call.ints(a[8], "seq_lens_out", b);
    int32_t *count_out = none(a[9]) ? count : call.ints(a[9], "free_count_out", 1);
    // one allocation for the three int32 outputs, each on a 16-byte boundary
    // (cu_seqlens goes on to the prefill calls, which ask for one)
    const int64_t n = ((int64_t)tokens + 3) / 4 * 4;
    const Tensor all = call.empty({2 * n + b + 1}, at::kInt);
    const Tensor served = call.empty({b}, at::kBool);
    int32_t *base = static_cast<int32_t *>(all.data_ptr());
    launch("lightning_attn_paged_reserve", [&] {
        return lightning_attn_paged_reserve(
            t.p, t.stride, t.width, lens, fresh, finished, b, free_pages, count, pages, page, tokens,
            base, base + n, base + 2 * n, static_cast<uint8_t *>(served.data_ptr()), lens_out,
            count_out, call.stream());
    });
    for (PyObject *o : {a[0], a[3], none(a[8]) ? a[1] : a[8], none(a[9]) ? a[4] : a[9]}) written(o);
    return tuple(part_of(all, 0, tokens), part_of(all, n, tokens), part_of(all, 2 * n, b + 1), served);
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        if (n != N) refuse(PyExc_TypeError, "%d arguments expected, got %d", N, (int)n);
        return F(args);
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define METHOD(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {METHOD(qk_norm_rope, 11), METHOD(qk_norm_rope_backward, 14),
                          METHOD(paged_append, 14), METHOD(paged_decode, 10),
                          METHOD(paged_step, 19),   METHOD(paged_reserve, 11),
                          METHOD(paged_bounds, 6),  METHOD(paged_select, 11),
                          METHOD(paged_sparse_decode, 11), METHOD(paged_prefix_decode, 12),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_lightning_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lightning_binding() { return PyModule_Create(&kModule); }
