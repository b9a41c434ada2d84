// The operators between the linear layers as functions of torch tensors:
// argument checks, outputs that the caller did not bring, and the call of the
// C entry point (include/fp8act.h). fp8act.py documents them. A decode step's
// operators take a few microseconds on the device; checked in Python, their
// arguments took 5 to 15.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <map>
#include <string>
#include <utility>

#include "../../include/fp8act.h"

namespace {

struct Raised {};  // a Python error is set

[[noreturn]] void raise(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Raised{};
}

std::string text(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + (v.size() == 1 ? ",)" : ")");
}

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

constexpr auto kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kI64 = at::kLong, kU8 = at::kByte,
               kF64 = at::kDouble, kE4m3 = at::kFloat8_e4m3fn;

// The library launches on the current device, which cannot read another one's memory in general: every tensor of a call
// is there. (Asked for once a call.)
thread_local int g_device = -1;
void on_current_device(const at::Tensor& t, const char* name) {
    if (g_device < 0) g_device = c10::cuda::current_device();
    if (t.get_device() != g_device) raise(PyExc_ValueError, std::string(name) + " is not on the current CUDA device");
}

// A contiguous CUDA tensor of a known shape and one of two types.
template <class T>
T* data(const at::Tensor& t, at::ScalarType a, at::ScalarType b, at::IntArrayRef shape, const char* name) {
    if (!t.is_cuda() || (t.scalar_type() != a && t.scalar_type() != b))
        raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor of type " + c10::toString(a) +
                                   (a == b ? "" : std::string(" or ") + c10::toString(b)));
    on_current_device(t, name);
    if (t.sizes() != shape || !t.is_contiguous())
        raise(PyExc_ValueError, std::string(name) + " must be contiguous with shape " + text(shape) + ", got " + text(t.sizes()));
    return static_cast<T*>(t.data_ptr());
}
template <class T = void>
T* data(const at::Tensor& t, at::ScalarType a, at::IntArrayRef shape, const char* name) {
    return data<T>(t, a, a, shape, name);
}
template <class T = void>
T* data(PyObject* o, at::ScalarType a, at::IntArrayRef shape, const char* name) {
    return data<T>(tensor(o, name), a, a, shape, name);
}
template <class T = void>
T* optional(PyObject* o, at::ScalarType a, at::IntArrayRef shape, const char* name) {
    return given(o) ? data<T>(o, a, shape, name) : nullptr;
}

// A bf16 [M, K] tensor of any M and K.
const at::Tensor& matrix(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.scalar_type() != kBf16) raise(PyExc_TypeError, std::string(name) + " must be a bf16 CUDA tensor");
    on_current_device(t, name);
    if (t.dim() != 2 || !t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be a contiguous 2-D tensor");
    return t;
}

int to_int(int64_t v, const char* name) {
    if (v > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " is too large");
    return static_cast<int>(v);
}

cudaStream_t stream_of(PyObject* o) {
    if (!given(o)) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* id = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!id) throw Raised{};
    void* p = PyLong_AsVoidPtr(id);
    Py_DECREF(id);
    if (!p && PyErr_Occurred()) throw Raised{};
    return static_cast<cudaStream_t>(p);
}

PyObject* g_error = nullptr;  // raises fp8act's exception: called with (function, status)

void check(const char* function, int status) {
    if (status == FP8ACT_OK) return;
    PyObject* r = PyObject_CallFunction(g_error, "si", function, status);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, function);
    throw Raised{};
}

template <size_t kN>
PyObject* tuple(const std::array<at::Tensor, kN>& v, size_t n = kN) {
    PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(n));
    for (size_t i = 0; t && i < n; ++i) PyTuple_SET_ITEM(t, static_cast<Py_ssize_t>(i), THPVariable_Wrap(v[i]));
    return t;
}

// The graph capture that `stream` takes part in, 0 for none.
unsigned long long capture_of(cudaStream_t stream) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (stream && cudaStreamGetCaptureInfo(stream, &status, &id) != cudaSuccess) {  // (the legacy stream cannot be captured)
        cudaGetLastError();
        return 0;
    }
    return status == cudaStreamCaptureStatusNone ? 0 : id;
}

// Uninitialised memory for a kernel on `stream`, from that stream's own pool whatever torch's current one is: what used
// it before has ended when the kernel starts, and once let go it is handed out again behind the kernel. In a graph the
// pool is the graph's, which torch knows for its own captures; a capture that the current stream has no part in may not
// be one, and its replays would outlive the memory.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType kind, const at::Tensor& like, cudaStream_t stream) {
    const auto options = like.options().dtype(kind);
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(like.get_device());
    if (current.stream() == stream) return at::empty(shape, options);
    const unsigned long long capture = capture_of(stream);
    if (capture && capture != capture_of(current.stream()))
        raise(PyExc_ValueError, "a call captured on a stream that is not torch's current one needs its outputs and workspace");
    const c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(stream, like.get_device()));
    return at::empty(shape, options);
}

// An output: the caller's tensor, or a new one, which the caller reads on the current stream.
at::Tensor output(PyObject* o, at::ScalarType kind, at::IntArrayRef shape, const at::Tensor& like, cudaStream_t stream,
                  const char* name) {
    if (given(o)) return tensor(o, name);
    at::Tensor t = fresh(shape, kind, like, stream);
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(like.get_device());
    if (current.stream() != stream) t.record_stream(current.unwrap());
    return t;
}

// A workspace: the caller's, or one kept per device and stream (calls of one stream share it; a graph being captured
// gets its own).
struct Workspace {
    at::Tensor keep;
    void* p;
    size_t bytes;
};
Workspace workspace(PyObject* o, size_t need, const at::Tensor& like, cudaStream_t stream) {
    if (given(o)) {
        const at::Tensor& t = tensor(o, "workspace");
        if (!t.is_cuda() || !t.is_contiguous()) raise(PyExc_TypeError, "workspace must be a contiguous CUDA tensor");
        on_current_device(t, "workspace");
        return {t, t.data_ptr(), static_cast<size_t>(t.nbytes())};
    }
    if (need < 16) need = 16;
    const auto make = [&] { return fresh({static_cast<int64_t>(need)}, kU8, like, stream); };
    if (capture_of(stream)) {
        at::Tensor t = make();
        return {t, t.data_ptr(), need};
    }
    static auto* kept = new std::map<std::pair<int, cudaStream_t>, at::Tensor>;  // outlives the CUDA context
    at::Tensor& t = (*kept)[{like.get_device(), stream}];
    if (!t.defined() || t.nbytes() < need) t = make();
    return {t, t.data_ptr(), static_cast<size_t>(t.nbytes())};
}

fp8act_kv_cache cache_of(PyObject* o) {
    PyObject* items = PySequence_Fast(o, "the cache must be (k, v, k_scale, v_scale)");
    if (!items) throw Raised{};
    if (PySequence_Fast_GET_SIZE(items) != 4) {
        Py_DECREF(items);
        raise(PyExc_ValueError, "the cache must be (k, v, k_scale, v_scale)");
    }
    PyObject* const* it = PySequence_Fast_ITEMS(items);
    fp8act_kv_cache c = {};
    try {
        const at::Tensor& k = tensor(it[0], "cache.k");
        if (k.dim() != 4)
            raise(PyExc_ValueError, "the cache's codes must be 4-D [pages, kv_heads, page_size, head_dim]");
        const at::IntArrayRef shape = k.sizes(), rows = shape.slice(0, 3);
        c.k_e4m3 = data<void>(k, kU8, kE4m3, shape, "cache.k");
        c.v_e4m3 = data<void>(tensor(it[1], "cache.v"), kU8, kE4m3, shape, "cache.v");
        c.k_scale = data<float>(it[2], kF32, rows, "cache.k_scale");
        c.v_scale = data<float>(it[3], kF32, rows, "cache.v_scale");
        c.num_pages = to_int(shape[0], "the cache");
        c.kv_heads = to_int(shape[1], "the cache");
        c.page_size = to_int(shape[2], "the cache");
        c.head_dim = to_int(shape[3], "the cache");
    } catch (...) {
        Py_DECREF(items);
        throw;
    }
    Py_DECREF(items);
    return c;
}

// A bf16 [tokens, heads, dim] tensor whose tokens may be apart (columns of wider rows); its token stride.
int64_t heads_of(const at::Tensor& t, int64_t heads, int64_t dim, const char* name) {
    if (!t.is_cuda() || t.scalar_type() != kBf16) raise(PyExc_TypeError, std::string(name) + " must be a bf16 CUDA tensor");
    on_current_device(t, name);
    if (t.dim() != 3 || t.size(2) != dim || (heads >= 0 && t.size(1) != heads))
        raise(PyExc_ValueError, std::string(name) + " must be [tokens, heads, " + std::to_string(dim) + "], got " + text(t.sizes()));
    if (t.stride(2) != 1 || (t.stride(1) != dim && t.size(1) > 1))
        raise(PyExc_ValueError, std::string(name) + ": the heads of a token must be contiguous");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * dim;  // (the stride of a single token is not used)
}

// (x, weight, residual, eps, weight_offset, q, sa, residual_out, stream) -> (q, sa[, residual_out])
PyObject* rmsnorm_quant(PyObject* const* a) {
    const at::Tensor& x = matrix(a[0], "x");
    const int64_t M = x.size(0), K = x.size(1);
    const void* w = data(a[1], kBf16, {K}, "weight");
    const double eps = PyFloat_AsDouble(a[3]), offset = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) throw Raised{};
    cudaStream_t stream = stream_of(a[8]);
    at::Tensor q = output(a[5], kU8, {M, K}, x, stream, "q"), sa = output(a[6], kF32, {M, K / 128}, x, stream, "sa"), out;
    void* qp = data<void>(q, kU8, kE4m3, {M, K}, "q");
    float* sp = data<float>(sa, kF32, {M, K / 128}, "sa");
    const void* r = nullptr;
    void* op = nullptr;
    if (given(a[2])) {
        r = data(a[2], kBf16, {M, K}, "residual");
        out = output(a[7], kBf16, {M, K}, x, stream, "residual_out");
        op = data(out, kBf16, {M, K}, "residual_out");
    } else if (given(a[7])) {
        raise(PyExc_ValueError, "residual_out without a residual");
    }
    check("fp8_rmsnorm_quant",
          fp8_rmsnorm_quant(x.data_ptr(), r, w, static_cast<float>(eps), static_cast<float>(offset), to_int(M, "M"),
                            to_int(K, "K"), qp, sp, op, stream));
    return tuple<3>({q, sa, out}, given(a[2]) ? 3 : 2);
}

// (gate_up, q, sa, stream) -> (q, sa)
PyObject* silu_mul_quant(PyObject* const* a) {
    const at::Tensor& x = matrix(a[0], "gate_up");
    if (x.size(1) % 2) raise(PyExc_ValueError, "gate_up must have an even number of columns");
    const int64_t M = x.size(0), I = x.size(1) / 2;
    cudaStream_t stream = stream_of(a[3]);
    at::Tensor q = output(a[1], kU8, {M, I}, x, stream, "q"), sa = output(a[2], kF32, {M, I / 128}, x, stream, "sa");
    void* qp = data<void>(q, kU8, kE4m3, {M, I}, "q");
    float* sp = data<float>(sa, kF32, {M, I / 128}, "sa");
    check("fp8_silu_mul_quant",
          fp8_silu_mul_quant(x.data_ptr(), to_int(M, "M"), to_int(I, "I"), qp, sp, stream));
    return tuple<2>({q, sa});
}

// (k, v, slots, cache, stream)
PyObject* kv_append(PyObject* const* a) {
    const fp8act_kv_cache c = cache_of(a[3]);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const int64_t ks = heads_of(k, c.kv_heads, c.head_dim, "k"), vs = heads_of(v, c.kv_heads, c.head_dim, "v"), T = k.size(0);
    if (v.size(0) != T) raise(PyExc_ValueError, "k and v have different numbers of tokens");
    const int64_t* slots = data<int64_t>(a[2], kI64, {T}, "slots");
    check("fp8_kv_append",
          fp8_kv_append(k.data_ptr(), v.data_ptr(), slots, to_int(T, "T"), ks, vs, &c, stream_of(a[4])));
    Py_RETURN_NONE;
}

// (q, k, v, positions, inv_freq, slots, cache, q_weight, k_weight, eps, weight_offset, axes, interleaved, rope_scale,
//  q_out, stream) -> q_out
PyObject* rope_append(PyObject* const* a) {
    const fp8act_kv_cache c = cache_of(a[6]);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &pos = tensor(a[3], "positions"),
                     &freq = tensor(a[4], "inv_freq");
    const int64_t D = c.head_dim, qs = heads_of(q, -1, D, "q"), ks = heads_of(k, c.kv_heads, D, "k"),
                  vs = heads_of(v, c.kv_heads, D, "v"), T = q.size(0), Hq = q.size(1);
    if (k.size(0) != T || v.size(0) != T) raise(PyExc_ValueError, "q, k and v have different numbers of tokens");
    if (pos.dim() != 1 && pos.dim() != 2) raise(PyExc_ValueError, "positions must be [T] or [axes, T]");
    const int64_t axes = pos.dim() == 2 ? pos.size(0) : 1;
    const int64_t* pp = pos.dim() == 2 ? data<int64_t>(pos, kI64, {axes, T}, "positions") : data<int64_t>(pos, kI64, {T}, "positions");
    if (freq.dim() != 1) raise(PyExc_ValueError, "inv_freq must be 1-D");
    const int64_t half = freq.size(0);
    const double* fp = data<double>(freq, kF64, {half}, "inv_freq");
    const int64_t* slots = data<int64_t>(a[5], kI64, {T}, "slots");
    const void *wq = optional(a[7], kBf16, {D}, "q_weight"), *wk = optional(a[8], kBf16, {D}, "k_weight");
    const int* ap = optional<int>(a[11], kI32, {half}, "axes");
    const double eps = PyFloat_AsDouble(a[9]), offset = PyFloat_AsDouble(a[10]), scale = PyFloat_AsDouble(a[13]);
    if (PyErr_Occurred()) throw Raised{};
    const int interleaved = PyObject_IsTrue(a[12]);
    if (interleaved < 0) throw Raised{};
    cudaStream_t stream = stream_of(a[15]);
    at::Tensor out = output(a[14], kBf16, {T, Hq, D}, q, stream, "q_out");
    void* op = data(out, kBf16, {T, Hq, D}, "q_out");
    check("fp8_rope_append",
          fp8_rope_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, wq, wk, static_cast<float>(eps),
                          static_cast<float>(offset), pp, fp, ap, to_int(axes, "axes"), to_int(2 * half, "inv_freq"), interleaved,
                          static_cast<float>(scale), slots, to_int(T, "T"), to_int(Hq, "q_heads"), &c, op, stream));
    return THPVariable_Wrap(out);
}

int to_count(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < INT32_MIN) raise(PyExc_ValueError, std::string(name) + " is too small");
    return to_int(v, name);
}

// What attention and its weights have in common: (q, cache, page_table, kv_lens, cu_q, max_q_len, softmax_scale).
struct Rows {
    fp8act_kv_cache c;
    const at::Tensor& q;
    int64_t q_stride, T, Hq;
    int pages, B, max_q;
    const int *table, *lens, *cu;
    double scale;
};
Rows rows_of(PyObject* const* a) {
    const fp8act_kv_cache c = cache_of(a[1]);
    const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[2], "page_table");
    const int64_t qs = heads_of(q, -1, c.head_dim, "q"), T = q.size(0);
    if (table.dim() != 2) raise(PyExc_ValueError, "page_table must be 2-D [B, max_pages]");
    const int64_t B = table.size(0), pages = table.size(1);
    const int* tp = data<int>(table, kI32, {B, pages}, "page_table");
    const int* lens = data<int>(a[3], kI32, {B}, "kv_lens");
    const int* cu = data<int>(a[4], kI32, {B + 1}, "cu_q");
    const int64_t most = given(a[5]) ? PyLong_AsLongLong(a[5]) : T == B ? 1 : T;
    const double scale = given(a[6]) ? PyFloat_AsDouble(a[6]) : 1.0 / std::sqrt(static_cast<double>(c.head_dim));
    if (PyErr_Occurred()) throw Raised{};
    to_int(T, "tokens");
    to_int(q.size(1), "q_heads");
    return {c, q, qs, T, q.size(1), to_int(pages, "max_pages"), to_int(B, "B"), to_int(most, "max_q_len"), tp, lens, cu, scale};
}

// (soft_cap, window, prefix_lens, first, slopes)
fp8act_scores scores_of(PyObject* const* a, const Rows& r) {
    fp8act_scores s = {};
    s.soft_cap = given(a[0]) ? static_cast<float>(PyFloat_AsDouble(a[0])) : 0.0f;
    if (PyErr_Occurred()) throw Raised{};
    s.window = given(a[1]) ? to_count(a[1], "window") : 0;
    s.prefix_lens = optional<int>(a[2], kI32, {r.B}, "prefix_lens");
    s.first = optional<int>(a[3], kI32, {r.T}, "first");
    s.slopes = optional<float>(a[4], kF32, {r.Hq}, "slopes");
    return s;
}

// (q, cache, page_table, kv_lens, cu_q, max_q_len, softmax_scale, out, lse, workspace, stream, soft_cap, window,
//  prefix_lens, first, slopes) -> out
PyObject* kv_attention(PyObject* const* a) {
    const Rows r = rows_of(a);
    const fp8act_scores s = scores_of(a + 11, r);
    cudaStream_t stream = stream_of(a[10]);
    const int64_t D = r.c.head_dim;
    at::Tensor out = output(a[7], kBf16, {r.T, r.Hq, D}, r.q, stream, "out");
    void* op = data(out, kBf16, {r.T, r.Hq, D}, "out");
    float* lse = optional<float>(a[8], kF32, {r.T, r.Hq}, "lse");
    const int hq = static_cast<int>(r.Hq);
    const Workspace w = workspace(a[9], fp8_kv_attention_workspace(r.max_q, hq, &r.c), r.q, stream);
    check("fp8_kv_attention",
          fp8_kv_attention_scored(r.q.data_ptr(), r.q_stride, r.cu, r.lens, r.table, r.pages, r.B, static_cast<int>(r.T), r.max_q,
                                  hq, static_cast<float>(r.scale), &s, &r.c, op, lse, w.p, w.bytes, stream));
    return THPVariable_Wrap(out);
}

// (q, cache, page_table, kv_lens, cu_q, max_q_len, softmax_scale, lse, mass, accumulate, stream, soft_cap, window,
//  prefix_lens, first, slopes, old_lens)
PyObject* kv_attention_mass(PyObject* const* a) {
    const Rows r = rows_of(a);
    const fp8act_scores s = scores_of(a + 11, r);
    const float* lse = data<float>(a[7], kF32, {r.T, r.Hq}, "lse");
    float* mass = data<float>(a[8], kF32, {r.c.num_pages, r.c.kv_heads, r.c.page_size}, "mass");
    const int* old = optional<int>(a[16], kI32, {r.B}, "old_lens");
    const int accumulate = PyObject_IsTrue(a[9]);
    if (accumulate < 0) throw Raised{};
    check("fp8_kv_attention_mass",
          fp8_kv_attention_mass(r.q.data_ptr(), r.q_stride, r.cu, r.lens, r.table, r.pages, r.B, static_cast<int>(r.T), r.max_q,
                                static_cast<int>(r.Hq), static_cast<float>(r.scale), &s, &r.c, lse, mass, accumulate, old,
                                stream_of(a[10])));
    Py_RETURN_NONE;
}

// (cache, mass, page_table, kv_lens, keep, new_table, recent, first, new_lens, kept, stream) -> (new_lens, kept)
PyObject* kv_evict(PyObject* const* a) {
    const fp8act_kv_cache c = cache_of(a[0]);
    const at::Tensor &table = tensor(a[2], "page_table"), &next = tensor(a[5], "new_table");
    float* mass = data<float>(a[1], kF32, {c.num_pages, c.kv_heads, c.page_size}, "mass");
    if (table.dim() != 2 || next.dim() != 2) raise(PyExc_ValueError, "page_table and new_table must be 2-D [B, pages]");
    const int64_t B = table.size(0), pages = table.size(1), fresh_pages = next.size(1);
    const int* tp = data<int>(table, kI32, {B, pages}, "page_table");
    const int* np = data<int>(next, kI32, {B, fresh_pages}, "new_table");
    const int* lens = data<int>(a[3], kI32, {B}, "kv_lens");
    const int* keep = data<int>(a[4], kI32, {B}, "keep");
    const int recent = to_count(a[6], "recent"), first = to_count(a[7], "first");
    cudaStream_t stream = stream_of(a[10]);
    const int64_t places = fresh_pages * c.page_size;
    at::Tensor new_lens = output(a[8], kI32, {B}, table, stream, "new_lens"),
               kept = output(a[9], kI32, {B, c.kv_heads, places}, table, stream, "kept");
    int* lp = data<int>(new_lens, kI32, {B}, "new_lens");
    int* kp = data<int>(kept, kI32, {B, c.kv_heads, places}, "kept");
    check("fp8_kv_evict", fp8_kv_evict(&c, mass, tp, to_int(pages, "max_pages"), lens, keep, np, to_int(fresh_pages, "new_pages"),
                                       to_int(B, "B"), recent, first, lp, kp, stream));
    return tuple<2>({new_lens, kept});
}

// (target_logits, draft_tokens, uniform, noise, temperature, draft_logits, n_draft, accepted, tokens, accept_prob,
//  workspace, stream) -> (accepted, tokens, accept_prob)
PyObject* verify_drafts(PyObject* const* a) {
    const at::Tensor& t = tensor(a[0], "target_logits");
    if (t.dim() != 3) raise(PyExc_ValueError, "target_logits must be [B, k + 1, V]");
    const int64_t B = t.size(0), rows = t.size(1), V = t.size(2), k = rows - 1;
    const auto kind = t.scalar_type();
    const void* tp = data<void>(t, kBf16, kF32, {B, rows, V}, "target_logits");
    const void* dp = optional(a[5], kind, {B, k, V}, "draft_logits");
    const int* x = data<int>(a[1], kI32, {B, k}, "draft_tokens");
    const float* u = data<float>(a[2], kF32, {B, k}, "uniform");
    const float* e = data<float>(a[3], kF32, {B, V}, "noise");
    const float* temp = data<float>(a[4], kF32, {B}, "temperature");
    const int* n = optional<int>(a[6], kI32, {B}, "n_draft");
    cudaStream_t stream = stream_of(a[11]);
    at::Tensor took = output(a[7], kI32, {B}, t, stream, "accepted"),
               tokens = output(a[8], kI32, {B, rows}, t, stream, "tokens"),
               prob = output(a[9], kF32, {B, k}, t, stream, "accept_prob");
    int* ap = data<int>(took, kI32, {B}, "accepted");
    int* op = data<int>(tokens, kI32, {B, rows}, "tokens");
    float* pp = data<float>(prob, kF32, {B, k}, "accept_prob");
    const int b = to_int(B, "B"), kk = to_int(k, "k");
    const Workspace w = workspace(a[10], fp8act_verify_drafts_workspace(b, kk), t, stream);
    check("fp8act_verify_drafts", fp8act_verify_drafts(tp, dp, kind == kF32, x, u, e, temp, n, b, kk, to_int(V, "V"), ap, op,
                                                       pp, w.p, w.bytes, stream));
    return tuple<3>({took, tokens, prob});
}

template <PyObject* (*kFunction)(PyObject* const*), Py_ssize_t kArgs>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) return PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", kArgs, n);
    g_device = -1;
    try {
        return kFunction(args);
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject* set_error(PyObject*, PyObject* f) {
    Py_XSETREF(g_error, Py_NewRef(f));
    Py_RETURN_NONE;
}

template <PyObject* (*kFunction)(PyObject* const*), Py_ssize_t kArgs>
constexpr PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<kFunction, kArgs>));
}

PyMethodDef g_methods[] = {
    {"rmsnorm_quant", fast<rmsnorm_quant, 9>(), METH_FASTCALL, nullptr},
    {"silu_mul_quant", fast<silu_mul_quant, 4>(), METH_FASTCALL, nullptr},
    {"kv_append", fast<kv_append, 5>(), METH_FASTCALL, nullptr},
    {"rope_append", fast<rope_append, 16>(), METH_FASTCALL, nullptr},
    {"kv_attention", fast<kv_attention, 16>(), METH_FASTCALL, nullptr},
    {"kv_attention_mass", fast<kv_attention_mass, 17>(), METH_FASTCALL, nullptr},
    {"kv_evict", fast<kv_evict, 11>(), METH_FASTCALL, nullptr},
    {"verify_drafts", fast<verify_drafts, 12>(), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fp8act", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8act() { return PyModule_Create(&g_module); }
