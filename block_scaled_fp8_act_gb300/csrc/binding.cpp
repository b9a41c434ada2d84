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
               kE4m3 = at::kFloat8_e4m3fn;

// A contiguous CUDA tensor of a known shape and one of two types.
template <class T>
T* data(const at::Tensor& t, at::ScalarType a, at::ScalarType b, at::IntArrayRef shape, const char* name) {
    if (!t.is_cuda() || (t.scalar_type() != a && t.scalar_type() != b))
        raise(PyExc_TypeError, std::string(name) + " must be a CUDA tensor of type " + c10::toString(a) +
                                   (a == b ? "" : std::string(" or ") + c10::toString(b)));
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

// (q, cache, page_table, kv_lens, cu_q, max_q_len, softmax_scale, out, lse, workspace, stream) -> out
PyObject* kv_attention(PyObject* const* a) {
    const fp8act_kv_cache c = cache_of(a[1]);
    const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[2], "page_table");
    const int64_t qs = heads_of(q, -1, c.head_dim, "q"), T = q.size(0), Hq = q.size(1);
    if (table.dim() != 2) raise(PyExc_ValueError, "page_table must be 2-D [B, max_pages]");
    const int64_t B = table.size(0), pages = table.size(1);
    const int* tp = data<int>(table, kI32, {B, pages}, "page_table");
    const int* lens = data<int>(a[3], kI32, {B}, "kv_lens");
    const int* cu = data<int>(a[4], kI32, {B + 1}, "cu_q");
    const int64_t most = given(a[5]) ? PyLong_AsLongLong(a[5]) : T == B ? 1 : T;
    const double scale = given(a[6]) ? PyFloat_AsDouble(a[6]) : 1.0 / std::sqrt(static_cast<double>(c.head_dim));
    if (PyErr_Occurred()) throw Raised{};
    cudaStream_t stream = stream_of(a[10]);
    at::Tensor out = output(a[7], kBf16, {T, Hq, c.head_dim}, q, stream, "out");
    void* op = data(out, kBf16, {T, Hq, c.head_dim}, "out");
    float* lse = optional<float>(a[8], kF32, {T, Hq}, "lse");
    const int max_q = to_int(most, "max_q_len"), hq = to_int(Hq, "q_heads");
    const Workspace w = workspace(a[9], fp8_kv_attention_workspace(max_q, hq, &c), q, stream);
    check("fp8_kv_attention", fp8_kv_attention(q.data_ptr(), qs, cu, lens, tp, to_int(pages, "max_pages"), to_int(B, "B"),
                                               to_int(T, "tokens"), max_q, hq, static_cast<float>(scale), &c, op, lse, w.p,
                                               w.bytes, stream));
    return THPVariable_Wrap(out);
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
    {"kv_attention", fast<kv_attention, 11>(), METH_FASTCALL, nullptr},
    {"verify_drafts", fast<verify_drafts, 12>(), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fp8act", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8act() { return PyModule_Create(&g_module); }
