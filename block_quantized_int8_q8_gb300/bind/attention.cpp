// attention.cpp -- Python binding of the attention operators (include/mmq.h): argument marshalling only, like the ctypes
// binding of the other entry points in api.py, but in C++ on torch's own tensors.  These operators run once per layer
// and decoding step on a few microseconds of GPU work, and reading a dozen tensors' pointers, types and strides through
// Python attributes takes longer than that (norm and rotation of four tokens: 16 us of host time through ctypes, of which
// the library call with its launch is 3 us).  Every argument is checked here or by the library; errors raise api.MMQError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <cmath>
#include <exception>
#include <string>
#include "../../include/mmq.h"

namespace {

PyObject* g_error = nullptr;               // api.MMQError
PyObject* g_no_memory = nullptr;           // torch.OutOfMemoryError

struct Refused : std::exception {          // becomes api.MMQError
    std::string text;
    explicit Refused(std::string t) : text(std::move(t)) {}
    const char* what() const noexcept override { return text.c_str(); }
};
struct PyRaised {};                        // a Python exception is already set

[[noreturn]] void refuse(const std::string& what, const char* why) { throw Refused(what + ": " + why); }

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) refuse(what, "expected a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor* tensor_or_none(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

long long integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyRaised();
    return v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyRaised();
    return (float)v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PyRaised();
    return v != 0;
}

bool dtype_of(at::ScalarType t, mmq_dtype* d) {
    switch (t) {
        case at::kFloat: *d = MMQ_F32; return true;
        case at::kBFloat16: *d = MMQ_BF16; return true;
        case at::kHalf: *d = MMQ_F16; return true;
        default: return false;
    }
}
at::ScalarType scalar_or(PyObject* o, at::ScalarType otherwise) {
    if (o == Py_None) return otherwise;
    if (!THPDtype_Check(o)) refuse("dtype", "expected a torch dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// The kernels run on the current device; its memory is theirs alone.
thread_local int t_device;                 // during a call: the current device, -1 until it is asked for
void on_device(int device, const char* what) {
    if (t_device < 0) t_device = c10::cuda::current_device();
    if (device != t_device) refuse(what, "is not on the current device");
}

// [tokens][heads][head_dim], the last dimension contiguous
mmq_heads heads(const at::Tensor& t, const char* what) {
    mmq_heads h;
    if (!t.is_cuda() || t.dim() != 3 || !dtype_of(t.scalar_type(), &h.dtype))
        refuse(what, "expected a CUDA tensor [tokens, heads, head_dim] of f32, bf16 or f16");
    if (t.stride(2) != 1) refuse(what, "the last dimension must be contiguous");
    on_device(t.get_device(), what);
    h.data = t.data_ptr();
    h.token_stride = t.stride(0);
    h.head_stride = t.stride(1);
    return h;
}
void* plain(const at::Tensor* t, at::ScalarType type, long long n, const char* what) {
    if (!t) return nullptr;
    if (t->scalar_type() != type) refuse(what, type == at::kInt ? "expected int32" : "expected float32");
    if (!t->is_cuda() || !t->is_contiguous()) refuse(what, "expected a contiguous CUDA tensor");
    if (n >= 0 && t->numel() != n) refuse(what, "has the wrong number of values");
    on_device(t->get_device(), what);
    return t->data_ptr();
}
const float* vector(PyObject* o, long long n, const char* what) {
    return static_cast<const float*>(plain(tensor_or_none(o, what), at::kFloat, n, what));
}

// the structure, or null where neither table is given
const mmq_rotary* rotary(PyObject* cos, PyObject* sin, PyObject* interleaved, mmq_rotary* r) {
    const at::Tensor *c = tensor_or_none(cos, "cos"), *s = tensor_or_none(sin, "sin");
    if (!c && !s) return nullptr;
    if (!c || !s || c->dim() != 2 || c->sizes() != s->sizes())
        refuse("cos, sin", "expected f32 tensors [positions, rot_dim / 2] of one shape");
    r->cos = static_cast<const float*>(plain(c, at::kFloat, -1, "cos"));
    r->sin = static_cast<const float*>(plain(s, at::kFloat, -1, "sin"));
    r->positions = c->size(0);
    r->rot_dim = (int32_t)(2 * c->size(1));
    r->interleaved = truth(interleaved);
    return r;
}

struct PackedCache {
    mmq_kv_cache c;
    int32_t device;
};
const mmq_kv_cache* cache_of(PyObject* o) {
    if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != (Py_ssize_t)sizeof(PackedCache)) refuse("cache", "expected a KVCache");
    const auto* p = reinterpret_cast<const PackedCache*>(PyBytes_AS_STRING(o));
    on_device(p->device, "cache");
    return &p->c;
}

mmq_kv_seqs sequences(PyObject* table, PyObject* lens, PyObject* cu) {
    const at::Tensor &t = tensor(table, "page_table"), &l = tensor(lens, "kv_lens");
    const at::Tensor* c = tensor_or_none(cu, "cu_tokens");
    mmq_kv_seqs q;
    const long long n = l.numel();
    if (n > INT32_MAX) refuse("kv_lens", "too many sequences");
    if (t.dim() != 2 || t.size(0) != n) refuse("page_table", "expected int32 [sequences, pages]");
    q.page_table = static_cast<const int32_t*>(plain(&t, at::kInt, -1, "page_table"));
    q.table_stride = t.size(1);
    q.kv_lens = static_cast<const int32_t*>(plain(&l, at::kInt, -1, "kv_lens"));
    q.cu_tokens = static_cast<const int32_t*>(plain(c, at::kInt, n + 1, "cu_tokens"));
    q.seqs = (int32_t)n;
    return q;
}

// the given output, or a new one of x's shape
at::Tensor output(const at::Tensor& x, PyObject* out, PyObject* dtype, const char* what) {
    if (out == Py_None) return at::empty(x.sizes(), x.options().dtype(scalar_or(dtype, x.scalar_type())));
    const at::Tensor& o = tensor(out, what);
    if (o.sizes() != x.sizes()) refuse(what, "the output has another shape");
    return o;
}

// The call's stream, a handle or None for the current one.  A given stream is the current one while this object lives, so
// that outputs and workspace come from its memory: what the allocator takes back from another stream may still be
// in use there, and a workspace given back when the call returns would be handed out there while the kernels use it.
class OnStream {
    c10::cuda::OptionalCUDAStreamGuard guard;
public:
    explicit OnStream(PyObject* o) {
        if (o == Py_None) return;
        const auto handle = reinterpret_cast<cudaStream_t>((uintptr_t)integer(o));
        guard.reset_stream(c10::cuda::getStreamFromExternal(handle, c10::cuda::current_device()));
    }
    operator mmq_stream_t() const {
        return reinterpret_cast<mmq_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
    }
};

void check(mmq_status st, const char* what) {
    if (st == MMQ_OK) return;
    std::string text = std::string(what) + ": status " + std::to_string((int)st) + " (" + mmq_status_string(st);
    if (st == MMQ_ERR_CUDA) text += std::string("; ") + mmq_last_cuda_error();
    throw Refused(text + ")");
}

void need(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse("binding", "wrong number of arguments");
}

PyObject* none() { Py_RETURN_NONE; }

// q, k, positions, cos, sin, q_weight, k_weight, eps, interleaved, q_out, k_out, dtype, stream
PyObject* qk_norm_rope(PyObject* const* a, Py_ssize_t n) {
    need(n, 13);
    const OnStream stream(a[12]);
    const at::Tensor *q = tensor_or_none(a[0], "q"), *k = tensor_or_none(a[1], "k");
    const at::Tensor* x = q ? q : k;
    if (!x) refuse("qk_norm_rope", "neither q nor k given");
    mmq_heads hq, hqo, hk, hko;
    at::Tensor qo, ko;
    if (q) hq = heads(*q, "q");
    if (k) hk = heads(*k, "k");
    const long long tokens = x->size(0), dim = x->size(2);
    if (q && k && (k->size(0) != tokens || k->size(2) != dim)) refuse("qk_norm_rope", "q and k differ in tokens or head_dim");
    if (q) hqo = heads(qo = output(*q, a[9], a[11], "q_out"), "q_out");
    if (k) hko = heads(ko = output(*k, a[10], a[11], "k_out"), "k_out");
    mmq_rotary r;
    const mmq_rotary* rot = rotary(a[3], a[4], a[8], &r);
    const void* pos = plain(tensor_or_none(a[2], "positions"), at::kInt, tokens, "positions");
    check(mmq_qk_norm_rope(q ? &hq : nullptr, q ? (int)q->size(1) : 0, vector(a[5], dim, "q_weight"), q ? &hqo : nullptr,
                           k ? &hk : nullptr, k ? (int)k->size(1) : 0, vector(a[6], dim, "k_weight"), k ? &hko : nullptr,
                           tokens, (int)dim, static_cast<const int32_t*>(pos), rot, real(a[7]), stream),
          "mmq_qk_norm_rope");
    PyObject* p = q ? THPVariable_Wrap(std::move(qo)) : none();
    PyObject* s = k ? THPVariable_Wrap(std::move(ko)) : none();
    PyObject* both = PyTuple_Pack(2, p, s);
    Py_XDECREF(p);
    Py_XDECREF(s);
    return both;
}

// cache, k, v, page_table, kv_lens, cu_tokens, cos, sin, interleaved, k_weight, eps, q, q_weight, q_out, q_dtype, stream
PyObject* kv_append(PyObject* const* a, Py_ssize_t n) {
    need(n, 16);
    const OnStream stream(a[15]);
    const mmq_kv_cache* c = cache_of(a[0]);
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const at::Tensor* q = tensor_or_none(a[11], "q");
    const mmq_heads hk = heads(k, "k"), hv = heads(v, "v");
    mmq_heads hq, hqo;
    const long long tokens = k.size(0), dim = k.size(2);
    if (v.sizes() != k.sizes() || k.size(1) != c->kv_heads || dim != c->head_dim)
        refuse("kv_append", "k and v are [tokens, kv_heads, head_dim] of the cache");
    at::Tensor qo;
    if (q) {
        hq = heads(*q, "q");
        if (q->size(0) != tokens || q->size(2) != dim) refuse("kv_append", "q and k differ in tokens or head_dim");
        hqo = heads(qo = output(*q, a[13], a[14], "q_out"), "q_out");
    }
    const mmq_kv_seqs sq = sequences(a[3], a[4], a[5]);
    mmq_rotary r;
    const mmq_rotary* rot = rotary(a[6], a[7], a[8], &r);
    check(mmq_kv_append(c, &sq, tokens, &hk, &hv, vector(a[9], dim, "k_weight"), q ? &hq : nullptr,
                        q ? (int)q->size(1) : 0, vector(a[12], dim, "q_weight"), q ? &hqo : nullptr, rot, real(a[10]),
                        stream),
          "mmq_kv_append");
    return q ? THPVariable_Wrap(std::move(qo)) : none();
}

// cache, device tensor, page_table, kv_lens, tokens, cu_tokens, dtype, stream
PyObject* kv_read(PyObject* const* a, Py_ssize_t n) {
    need(n, 8);
    const OnStream stream(a[7]);
    const mmq_kv_cache* c = cache_of(a[0]);
    const long long tokens = integer(a[4]);
    if (tokens < 0) refuse("kv_read", "tokens is negative");
    const auto options = tensor(a[1], "cache").options().dtype(scalar_or(a[6], at::kBFloat16));
    at::Tensor k = at::empty({tokens, c->kv_heads, c->head_dim}, options), v = at::empty(k.sizes(), options);
    const mmq_heads hk = heads(k, "k"), hv = heads(v, "v");
    const mmq_kv_seqs sq = sequences(a[2], a[3], a[5]);
    check(mmq_kv_read(c, &sq, tokens, &hk, &hv, stream), "mmq_kv_read");
    PyObject *p = THPVariable_Wrap(std::move(k)), *s = THPVariable_Wrap(std::move(v));
    PyObject* both = PyTuple_Pack(2, p, s);
    Py_XDECREF(p);
    Py_XDECREF(s);
    return both;
}

// q, cache, page_table, kv_lens, max_kv_len, cu_tokens, max_tokens, scale, causal, window, out, out_dtype, return_lse,
// workspace, stream
PyObject* attention(PyObject* const* a, Py_ssize_t n) {
    need(n, 15);
    const OnStream stream(a[14]);
    const at::Tensor& q = tensor(a[0], "q");
    const mmq_kv_cache* c = cache_of(a[1]);
    const mmq_heads hq = heads(q, "q");
    const long long tokens = q.size(0), h = q.size(1), dim = q.size(2);
    if (dim != c->head_dim) refuse("attention", "q has another head_dim than the cache");
    if (h > INT32_MAX) refuse("attention", "too many heads");
    const mmq_kv_seqs sq = sequences(a[2], a[3], a[5]);
    const long long max_kv = a[4] == Py_None ? sq.table_stride * c->page_size : integer(a[4]);
    const long long max_tokens = a[6] == Py_None ? (sq.cu_tokens ? tokens : 1) : integer(a[6]);
    const float scale = a[7] == Py_None ? 1.f / std::sqrt((float)dim) : real(a[7]);
    at::Tensor out = output(q, a[10], a[11], "out"), lse, ws;
    const mmq_heads ho = heads(out, "out");
    if (truth(a[12])) lse = at::empty({tokens, h}, q.options().dtype(at::kFloat));
    size_t size = 0;
    if (a[13] == Py_None) {
        size = mmq_attention_workspace_bytes(tokens, (int)h, c->kv_heads, (int)dim, sq.seqs, max_tokens, max_kv);
        if (size) ws = at::empty({(long long)size}, q.options().dtype(at::kByte));
    } else {
        ws = tensor(a[13], "workspace");
        if (!ws.is_cuda() || !ws.is_contiguous()) refuse("workspace", "expected a contiguous CUDA tensor");
        on_device(ws.get_device(), "workspace");
        size = (size_t)ws.nbytes();
    }
    check(mmq_attention(&hq, (int)h, c, &sq, tokens, max_tokens, max_kv, scale, truth(a[8]), integer(a[9]), &ho,
                        lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
                        ws.defined() ? ws.data_ptr() : nullptr, size, stream),
          "mmq_attention");
    if (!lse.defined()) return THPVariable_Wrap(std::move(out));
    PyObject *p = THPVariable_Wrap(std::move(out)), *s = THPVariable_Wrap(std::move(lse));
    PyObject* both = PyTuple_Pack(2, p, s);
    Py_XDECREF(p);
    Py_XDECREF(s);
    return both;
}

// k, v, k_scale, v_scale -> (packed cache, pages, kv_heads, page_size, head_dim, block)
PyObject* make_cache(PyObject* const* a, Py_ssize_t n) {
    need(n, 4);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &ks = tensor(a[2], "k_scale"), &vs = tensor(a[3], "v_scale");
    if (k.scalar_type() != at::kChar || v.scalar_type() != at::kChar || k.dim() != 4 || v.sizes() != k.sizes())
        refuse("KVCache", "k and v are int8 tensors of one shape [pages, kv_heads, page_size, head_dim]");
    if (ks.scalar_type() != at::kFloat || vs.scalar_type() != at::kFloat || ks.dim() != 3 || vs.sizes() != ks.sizes() ||
        ks.size(0) != k.size(0) || ks.size(1) != k.size(1) || ks.size(2) <= 0 || k.size(2) % ks.size(2))
        refuse("KVCache", "the scales are f32 tensors [pages, kv_heads, page_size / block]");
    for (const at::Tensor* t : {&k, &v, &ks, &vs})
        if (!t->is_cuda() || !t->is_contiguous() || t->get_device() != k.get_device())
            refuse("KVCache", "expected contiguous CUDA tensors on one device");
    if (k.size(1) > INT32_MAX || k.size(2) > INT32_MAX || k.size(3) > INT32_MAX) refuse("KVCache", "too large");
    PackedCache p{};
    p.device = (int32_t)k.get_device();
    mmq_kv_cache& c = p.c;
    c.k = static_cast<int8_t*>(k.data_ptr());
    c.v = static_cast<int8_t*>(v.data_ptr());
    c.k_scale = static_cast<float*>(ks.data_ptr());
    c.v_scale = static_cast<float*>(vs.data_ptr());
    c.pages = k.size(0);
    c.kv_heads = (int32_t)k.size(1);
    c.page_size = (int32_t)k.size(2);
    c.head_dim = (int32_t)k.size(3);
    c.block = (int32_t)(k.size(2) / ks.size(2));
    return Py_BuildValue("(y#Liiii)", reinterpret_cast<const char*>(&p), (Py_ssize_t)sizeof(p), (long long)c.pages,
                         (int)c.kv_heads, (int)c.page_size, (int)c.head_dim, (int)c.block);
}

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
    t_device = -1;
    try {
        return F(args, n);
    } catch (const PyRaised&) {
        return nullptr;
    } catch (const Refused& e) {
        PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(g_no_memory ? g_no_memory : PyExc_MemoryError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* set_errors(PyObject*, PyObject* types) {
    PyObject *error, *no_memory;
    if (!PyArg_ParseTuple(types, "OO", &error, &no_memory)) return nullptr;
    Py_INCREF(error);
    Py_XSETREF(g_error, error);
    Py_INCREF(no_memory);
    Py_XSETREF(g_no_memory, no_memory);
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(qk_norm_rope), FAST(kv_append), FAST(kv_read), FAST(attention), FAST(make_cache),
                         {"set_errors", set_errors, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attention", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attention(void) { return PyModule_Create(&module); }
