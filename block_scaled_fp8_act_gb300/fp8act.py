"""Binding of libfp8act.so (argument marshalling only).

The linear layer's functions go through ctypes, the operators between the
layers (fp8_rmsnorm_quant .. verify_drafts) through an extension module that
does the same in C++ (csrc/binding.cpp), since a decode step's calls of them
are shorter on the device than their argument checks are in Python.

Each function takes CUDA torch tensors, checks dtype / device / contiguity,
passes raw device pointers, sizes and the current CUDA stream to the C entry
point of the same name (include/fp8act.h) and raises Fp8ActError on a
non-zero status. All arithmetic runs in the library's CUDA kernels; there is
no fallback: if the library is not built, loading it raises.

The library launches on the current device. The operators between the layers
refuse a tensor of another one (ValueError), whichever argument it is.

With a `stream` that is not torch's current one, what an operator between the
layers makes itself (outputs, a workspace) comes from that stream's memory
pool; the outputs may be read and dropped on the current stream once it has
waited for the other. In a graph captured on a stream that is not the current
one they have to be brought (ValueError).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import re
from typing import NamedTuple

import torch

from . import build as _build

G = 128
_lib = None
_ext = None

STATUS = {0: "FP8ACT_OK", 1: "FP8ACT_ERR_NULL", 2: "FP8ACT_ERR_SHAPE", 3: "FP8ACT_ERR_ALIGN",
          4: "FP8ACT_ERR_LAUNCH", 5: "FP8ACT_ERR_TIMEOUT", 6: "FP8ACT_ERR_DEVICE", 7: "FP8ACT_ERR_CUDA",
          8: "FP8ACT_ERR_INDEX"}


class Fp8ActError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)}: {msg}")
        self.status = status


def header_symbols() -> list[str]:
    """Names of the entry points include/fp8act.h declares."""
    text = open(os.path.join(_build.INCLUDE, "fp8act.h"), encoding="utf-8").read()
    return re.findall(r"FP8ACT_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)


def lib_path() -> str:
    return _build.LIB_PATH


def load(build: bool = False) -> ctypes.CDLL:
    """Load libfp8act.so (compiling it first when build=True)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.build() if build else _build.LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libfp8act.so is not built ({path}); run block_scaled_fp8_act_gb300.build.build()")
    L = ctypes.CDLL(path)
    p, i = ctypes.c_void_p, ctypes.c_int
    L.fp8_act_quant.argtypes = [p, i, i, p, p, p]
    L.fp8_weight_quant.argtypes = [p, i, i, p, p, p]
    L.fp8_block_gemm.argtypes = [p, p, p, p, i, i, i, p, p]
    L.fp8_block_gemm_f32.argtypes = [p, p, p, p, i, i, i, p, p]
    L.fp8_block_gemm_w8a16.argtypes = [p, p, p, i, i, i, p, p]
    L.fp8_block_gemm_w8a16_f32.argtypes = [p, p, p, i, i, i, p, p]
    L.fp8_linear.argtypes = [p, p, p, i, i, i, p, p]
    L.fp8_linear_f32.argtypes = [p, p, p, i, i, i, p, p]
    L.fp8_act_quant_grouped.argtypes = [p, i, p]
    L.fp8_block_gemm_grouped.argtypes = [p, i, p]
    L.fp8_block_gemm_grouped_f32.argtypes = [p, i, p]
    L.fp8act_strerror.argtypes = [i]
    L.fp8act_strerror.restype = ctypes.c_char_p
    L.fp8act_check_status.argtypes = [p]
    L.fp8act_set_wait_limit.argtypes = [ctypes.c_longlong, i]
    L.fp8act_stream_read.argtypes = [p, ctypes.c_size_t, p, p]
    f, i64 = ctypes.c_float, ctypes.c_int64
    L.fp8_rmsnorm_quant.argtypes = [p, p, p, f, f, i, i, p, p, p, p]
    L.fp8_silu_mul_quant.argtypes = [p, i, i, p, p, p]
    L.fp8_kv_append.argtypes = [p, p, p, i, i64, i64, p, p]
    L.fp8_rope_append.argtypes = [p, p, p, i64, i64, i64, p, p, f, f, p, p, p, i, i, i, f, p, i, i, p, p, p]
    L.fp8_kv_attention.argtypes = [p, i64, p, p, p, i, i, i, i, i, f, p, p, p, p, ctypes.c_size_t, p]
    L.fp8_kv_attention_scored.argtypes = [p, i64, p, p, p, i, i, i, i, i, f, p, p, p, p, p, ctypes.c_size_t, p]
    L.fp8_kv_attention_mass.argtypes = [p, i64, p, p, p, i, i, i, i, i, f, p, p, p, p, i, p, p]
    L.fp8_kv_attention_workspace.argtypes = [i, i, p]
    L.fp8_kv_attention_workspace.restype = ctypes.c_size_t
    L.fp8_kv_evict.argtypes = [p, p, p, i, p, p, p, i, i, i, i, p, p, p]
    L.fp8act_verify_drafts.argtypes = [p, p, i, p, p, p, p, p, i, i, i, p, p, p, p, ctypes.c_size_t, p]
    L.fp8act_verify_drafts_workspace.argtypes = [i, i]
    L.fp8act_verify_drafts_workspace.restype = ctypes.c_size_t
    for fn in (L.fp8_rmsnorm_quant, L.fp8_silu_mul_quant, L.fp8_kv_append, L.fp8_rope_append, L.fp8_kv_attention,
               L.fp8_kv_attention_scored, L.fp8_kv_attention_mass, L.fp8_kv_evict,
               L.fp8act_verify_drafts, L.fp8_act_quant, L.fp8_weight_quant, L.fp8_block_gemm, L.fp8_block_gemm_f32,
               L.fp8_block_gemm_w8a16, L.fp8_block_gemm_w8a16_f32,
               L.fp8_act_quant_grouped, L.fp8_block_gemm_grouped, L.fp8_block_gemm_grouped_f32,
               L.fp8_linear, L.fp8_linear_f32,
               L.fp8act_check_status, L.fp8act_set_wait_limit, L.fp8act_version, L.fp8act_stream_read):
        fn.restype = ctypes.c_int
    _lib = L
    return L


def _raise(fn: str, status: int) -> None:
    raise Fp8ActError(fn, status, strerror(status))


def _native():
    """The extension module of the operators between the linear layers."""
    global _ext
    if _ext is None:
        load()
        if not os.path.exists(_build.EXT_PATH):
            raise RuntimeError(f"the binding is not built ({_build.EXT_PATH}); run block_scaled_fp8_act_gb300.build.build()")
        loader = importlib.machinery.ExtensionFileLoader("_fp8act", _build.EXT_PATH)
        ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fp8act", loader))
        loader.exec_module(ext)
        ext.set_error(_raise)
        _ext = ext
    return _ext


def strerror(status: int) -> str:
    return load().fp8act_strerror(int(status)).decode()


def _stream(stream) -> int:
    """The cudaStream_t to launch on, as an integer (None: the current device's current stream)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise Fp8ActError(fn, status, strerror(status))


def _cuda2d(t: torch.Tensor, dtypes, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D tensor")


_CODES = (torch.uint8, torch.float8_e4m3fn)


def fp8_act_quant(x: torch.Tensor, q: torch.Tensor | None = None, sa: torch.Tensor | None = None, stream=None):
    """x bf16 [M, K] -> (q uint8 E4M3 codes [M, K], sa fp32 [M, K/128])."""
    _cuda2d(x, (torch.bfloat16,), "x")
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device) if q is None else q
    sa = torch.empty((M, K // G), dtype=torch.float32, device=x.device) if sa is None else sa
    _cuda2d(q, _CODES, "q")
    _cuda2d(sa, (torch.float32,), "sa")
    if q.shape != (M, K) or sa.shape != (M, K // G):
        raise ValueError("q / sa have the wrong shape")
    _check("fp8_act_quant", load().fp8_act_quant(x.data_ptr(), M, K, q.data_ptr(), sa.data_ptr(), _stream(stream)))
    return q, sa


def fp8_weight_quant(W: torch.Tensor, w: torch.Tensor | None = None, sw: torch.Tensor | None = None, stream=None):
    """W bf16 [N, K] -> (w uint8 E4M3 codes [N, K], sw fp32 [ceil(N/128), K/128])."""
    _cuda2d(W, (torch.bfloat16,), "W")
    N, K = W.shape
    NB = (N + G - 1) // G
    w = torch.empty((N, K), dtype=torch.uint8, device=W.device) if w is None else w
    sw = torch.empty((NB, K // G), dtype=torch.float32, device=W.device) if sw is None else sw
    _cuda2d(w, _CODES, "w")
    _cuda2d(sw, (torch.float32,), "sw")
    if w.shape != (N, K) or sw.shape != (NB, K // G):
        raise ValueError("w / sw have the wrong shape")
    _check("fp8_weight_quant", load().fp8_weight_quant(W.data_ptr(), N, K, w.data_ptr(), sw.data_ptr(),
                                                       _stream(stream)))
    return w, sw


def _gemm(fn_name: str, out_dtype, q, sa, w, sw, out, stream):
    for t, n, d in ((q, "q", _CODES), (sa, "sa", (torch.float32,)), (w, "w", _CODES), (sw, "sw", (torch.float32,))):
        _cuda2d(t, d, n)
    M, K = q.shape
    N = w.shape[0]
    if w.shape[1] != K or sa.shape != (M, K // G) or sw.shape != ((N + G - 1) // G, K // G):
        raise ValueError("inconsistent q / sa / w / sw shapes")
    out = torch.empty((M, N), dtype=out_dtype, device=q.device) if out is None else out
    _cuda2d(out, (out_dtype,), "out")
    if out.shape != (M, N):
        raise ValueError("out has the wrong shape")
    fn = getattr(load(), fn_name)
    _check(fn_name, fn(q.data_ptr(), sa.data_ptr(), w.data_ptr(), sw.data_ptr(), M, N, K, out.data_ptr(),
                       _stream(stream)))
    return out


def fp8_block_gemm(q, sa, w, sw, out=None, stream=None) -> torch.Tensor:
    """bf16 [M, N] = block-scaled q [M, K] x w [N, K]^T."""
    return _gemm("fp8_block_gemm", torch.bfloat16, q, sa, w, sw, out, stream)


def fp8_block_gemm_f32(q, sa, w, sw, out=None, stream=None) -> torch.Tensor:
    """fp32 [M, N] output of the same kernels (no bf16 cast)."""
    return _gemm("fp8_block_gemm_f32", torch.float32, q, sa, w, sw, out, stream)


def fp8_linear(x, w, sw, out=None, stream=None) -> torch.Tensor:
    """bf16 [M, N] = fp8_block_gemm(fp8_act_quant(x), w, sw) in one launch (decode-sized M)."""
    return _gemm_w8a16("fp8_linear", torch.bfloat16, x, w, sw, out, stream)


def fp8_linear_f32(x, w, sw, out=None, stream=None) -> torch.Tensor:
    """fp32 [M, N] output of the fused kernels (no bf16 cast)."""
    return _gemm_w8a16("fp8_linear_f32", torch.float32, x, w, sw, out, stream)


def _gemm_w8a16(fn_name: str, out_dtype, x, w, sw, out, stream):
    _cuda2d(x, (torch.bfloat16,), "x")
    _cuda2d(w, _CODES, "w")
    _cuda2d(sw, (torch.float32,), "sw")
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K or sw.shape != ((N + G - 1) // G, K // G):
        raise ValueError("inconsistent x / w / sw shapes")
    out = torch.empty((M, N), dtype=out_dtype, device=x.device) if out is None else out
    _cuda2d(out, (out_dtype,), "out")
    if out.shape != (M, N):
        raise ValueError("out has the wrong shape")
    fn = getattr(load(), fn_name)
    _check(fn_name, fn(x.data_ptr(), w.data_ptr(), sw.data_ptr(), M, N, K, out.data_ptr(), _stream(stream)))
    return out


def fp8_block_gemm_w8a16(x, w, sw, out=None, stream=None) -> torch.Tensor:
    """bf16 [M, N] = bf16 x [M, K] times block-scaled E4M3 w [N, K]^T (no activation quantisation)."""
    return _gemm_w8a16("fp8_block_gemm_w8a16", torch.bfloat16, x, w, sw, out, stream)


def fp8_block_gemm_w8a16_f32(x, w, sw, out=None, stream=None) -> torch.Tensor:
    """fp32 [M, N] output of the weight-only kernels (no bf16 cast)."""
    return _gemm_w8a16("fp8_block_gemm_w8a16_f32", torch.float32, x, w, sw, out, stream)


class QuantProblem(ctypes.Structure):
    """fp8act_quant_problem of include/fp8act.h."""
    _fields_ = [("x_bf16", ctypes.c_void_p), ("q_e4m3", ctypes.c_void_p), ("sa", ctypes.c_void_p),
                ("M", ctypes.c_int), ("K", ctypes.c_int)]


class GemmProblem(ctypes.Structure):
    """fp8act_gemm_problem of include/fp8act.h."""
    _fields_ = [("q_e4m3", ctypes.c_void_p), ("sa", ctypes.c_void_p), ("w_e4m3", ctypes.c_void_p),
                ("sw", ctypes.c_void_p), ("out", ctypes.c_void_p), ("M", ctypes.c_int), ("N", ctypes.c_int),
                ("K", ctypes.c_int)]


MAX_GROUPED = 16


def fp8_act_quant_grouped(xs, outs=None, stream=None):
    """Quantise several bf16 activations [M_i, K_i] in one launch.

    Returns [(q_i, sa_i)]; `outs` may supply them."""
    if len(xs) > MAX_GROUPED:
        raise ValueError(f"at most {MAX_GROUPED} problems per grouped call")
    res = []
    arr = (QuantProblem * max(1, len(xs)))()
    for i, x in enumerate(xs):
        _cuda2d(x, (torch.bfloat16,), "x")
        M, K = x.shape
        if outs is None:
            q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
            sa = torch.empty((M, K // G), dtype=torch.float32, device=x.device)
        else:
            q, sa = outs[i]
        _cuda2d(q, _CODES, "q")
        _cuda2d(sa, (torch.float32,), "sa")
        if q.shape != (M, K) or sa.shape != (M, K // G):
            raise ValueError("q / sa have the wrong shape")
        arr[i] = QuantProblem(x.data_ptr(), q.data_ptr(), sa.data_ptr(), M, K)
        res.append((q, sa))
    _check("fp8_act_quant_grouped", load().fp8_act_quant_grouped(ctypes.byref(arr), len(xs), _stream(stream)))
    return res


def _gemm_grouped(fn_name: str, out_dtype, problems, outs, stream):
    if len(problems) > MAX_GROUPED:
        raise ValueError(f"at most {MAX_GROUPED} problems per grouped call")
    res = []
    arr = (GemmProblem * max(1, len(problems)))()
    for i, (q, sa, w, sw) in enumerate(problems):
        for t, n, d in ((q, "q", _CODES), (sa, "sa", (torch.float32,)), (w, "w", _CODES),
                        (sw, "sw", (torch.float32,))):
            _cuda2d(t, d, n)
        M, K = q.shape
        N = w.shape[0]
        if w.shape[1] != K or sa.shape != (M, K // G) or sw.shape != ((N + G - 1) // G, K // G):
            raise ValueError("inconsistent q / sa / w / sw shapes")
        out = torch.empty((M, N), dtype=out_dtype, device=q.device) if outs is None else outs[i]
        _cuda2d(out, (out_dtype,), "out")
        if out.shape != (M, N):
            raise ValueError("out has the wrong shape")
        arr[i] = GemmProblem(q.data_ptr(), sa.data_ptr(), w.data_ptr(), sw.data_ptr(), out.data_ptr(), M, N, K)
        res.append(out)
    _check(fn_name, getattr(load(), fn_name)(ctypes.byref(arr), len(problems), _stream(stream)))
    return res


def fp8_block_gemm_grouped(problems, outs=None, stream=None) -> list:
    """Several block GEMMs [(q, sa, w, sw), ...] in one launch; returns the bf16 outputs."""
    return _gemm_grouped("fp8_block_gemm_grouped", torch.bfloat16, problems, outs, stream)


def fp8_block_gemm_grouped_f32(problems, outs=None, stream=None) -> list:
    """fp32 outputs of the grouped kernels (no bf16 cast)."""
    return _gemm_grouped("fp8_block_gemm_grouped_f32", torch.float32, problems, outs, stream)


def fp8_rmsnorm_quant(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0, q=None, sa=None,
                      residual_out=None, stream=None):
    """RMS norm of x (+ residual) with E4M3 codes out, bf16 x, residual [M, K], weight [K].

    Returns (q, sa), or (q, sa, residual_out) with a residual; residual_out = bf16(x + residual)
    may be x or residual. The weight applied is weight + weight_offset."""
    return _native().rmsnorm_quant(x, weight, residual, eps, weight_offset, q, sa, residual_out, stream)


def fp8_silu_mul_quant(gate_up, q=None, sa=None, stream=None):
    """silu(gate) * up of bf16 rows [gate | up] ([M, 2 I]) -> (q E4M3 codes [M, I], sa fp32 [M, I/128])."""
    return _native().silu_mul_quant(gate_up, q, sa, stream)


class KvCache(NamedTuple):
    """The paged E4M3 cache: codes [pages, kv_heads, page_size, head_dim], scales [pages, kv_heads, page_size]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


class KvCacheStruct(ctypes.Structure):
    """fp8act_kv_cache of include/fp8act.h."""
    _fields_ = [("k_e4m3", ctypes.c_void_p), ("v_e4m3", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class ScoresStruct(ctypes.Structure):
    """fp8act_scores of include/fp8act.h."""
    _fields_ = [("soft_cap", ctypes.c_float), ("window", ctypes.c_int), ("prefix_lens", ctypes.c_void_p),
                ("first", ctypes.c_void_p), ("slopes", ctypes.c_void_p)]


def kv_cache(num_pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> KvCache:
    """A cache of zeroed pages."""
    shape = (num_pages, kv_heads, page_size)
    return KvCache(torch.zeros((*shape, head_dim), dtype=torch.uint8, device=device),
                   torch.zeros((*shape, head_dim), dtype=torch.uint8, device=device),
                   torch.ones(shape, device=device), torch.ones(shape, device=device))


def fp8_kv_append(k, v, slots, cache, stream=None) -> None:
    """Quantise bf16 k, v [T, kv_heads, head_dim] into the cache's slots (int64 [T], distinct; negative = skip)."""
    _native().kv_append(k, v, slots, cache, stream)


def fp8_rope_append(q, k, v, positions, inv_freq, slots, cache, q_weight=None, k_weight=None, eps: float = 1e-6,
                    weight_offset: float = 0.0, axes=None, interleaved: bool = False, rope_scale: float = 1.0,
                    q_out=None, stream=None):
    """Head norms, rotary positions and the cache append of new tokens -> q_out bf16 [T, q_heads, head_dim].

    bf16 q [T, q_heads, head_dim], k, v [T, kv_heads, head_dim] (columns of wider rows may be passed);
    q_weight, k_weight [head_dim] (None: no norm). positions int64 [T], or [n, T] with `axes` int32
    [rot / 2] naming the row that turns each pair (None: the first); inv_freq float64 [rot / 2] turns the
    first rot columns, pairs (i, i + rot / 2) or, interleaved, (2i, 2i + 1), by positions * inv_freq, times
    rope_scale. The turned keys and the values go to `slots` (int64 [T], distinct; negative = the cache is
    left alone) of the cache."""
    return _native().rope_append(q, k, v, positions, inv_freq, slots, cache, q_weight, k_weight, eps, weight_offset, axes,
                                 interleaved, rope_scale, q_out, stream)


def kv_attention_workspace(max_q_len: int, q_heads: int, cache) -> int:
    """Bytes of workspace fp8_kv_attention needs."""
    pages, heads, page, dim = cache[0].shape
    c = KvCacheStruct(None, None, None, None, 0, page, heads, dim)
    return int(load().fp8_kv_attention_workspace(max_q_len, q_heads, ctypes.byref(c)))


def fp8_kv_attention(q, cache, page_table, kv_lens, cu_q, max_q_len: int | None = None,
                     softmax_scale: float | None = None, out=None, lse=None, workspace=None, stream=None,
                     soft_cap: float = 0.0, window: int = 0, prefix_lens=None, first=None, slopes=None):
    """bf16 [tokens, q_heads, head_dim] = causal attention of the new tokens q over the cache.

    page_table int32 [B, max_pages], kv_lens int32 [B] (cached tokens, the new ones included),
    cu_q int32 [B + 1] (rows of q per sequence). max_q_len (the most new tokens of a sequence)
    picks the row tile; softmax_scale defaults to head_dim ** -0.5. `lse` (fp32 [tokens, q_heads])
    is filled if given. Rows that no sequence has (past cu_q[B]) are not written. `workspace`: a uint8 tensor of kv_attention_workspace() bytes, kept by the
    caller per stream; without one the binding keeps its own per device and stream.

    Scores: soft_cap > 0 caps them, soft_cap * tanh(x / soft_cap); slopes (fp32 [q_heads]) take
    slopes * distance off. A new token at position i sees position j if j < prefix_lens (int32 [B]), or if
    first <= j <= i (int32 [tokens], not falling over a sequence's) and, with a window, j > i - window. Positions
    are places of the cache: after fp8_kv_evict they are not those that the tokens had."""
    return _native().kv_attention(q, cache, page_table, kv_lens, cu_q, max_q_len, softmax_scale, out, lse, workspace,
                                  stream, soft_cap, window, prefix_lens, first, slopes)


def fp8_kv_attention_mass(q, cache, page_table, kv_lens, cu_q, lse, mass, max_q_len: int | None = None,
                          softmax_scale: float | None = None, accumulate: bool = True, stream=None,
                          soft_cap: float = 0.0, window: int = 0, prefix_lens=None, first=None, slopes=None,
                          old_lens=None) -> None:
    """Adds to mass (fp32 [pages, kv_heads, page_size]) the attention weight that every cached token gets.

    The weights exp(score - lse) of the new tokens q, summed over them and over the query heads of a KV head;
    lse (fp32 [tokens, q_heads]) is what fp8_kv_attention left with the same arguments. The places from
    old_lens (int32 [B]; None: all but the new tokens) on start from zero, all of a sequence's if not
    `accumulate`; pages that no token of q sees and whose weights stay are left alone, whatever the table has
    there. A page that gets weight belongs to one sequence of the call."""
    _native().kv_attention_mass(q, cache, page_table, kv_lens, cu_q, max_q_len, softmax_scale, lse, mass, accumulate, stream,
                                soft_cap, window, prefix_lens, first, slopes, old_lens)


def kv_mass(cache) -> torch.Tensor:
    """Zeroed weights of a cache's tokens, fp32 [pages, kv_heads, page_size]."""
    return torch.zeros_like(cache[2])


def fp8_kv_evict(cache, mass, page_table, kv_lens, keep, new_table, recent: int = 0, first: int = 0, new_lens=None,
                 kept=None, stream=None):
    """Copies the tokens that matter most into other pages -> (new_lens int32 [B], kept int32 [B, kv_heads, places]).

    Of each sequence and KV head min(kv_lens, keep) tokens stay (keep int32 [B]): the last `recent`, the first
    `first`, then those of largest `mass` (fp32 [pages, kv_heads, page_size]; equal ones by position). They go,
    in their order, with their scales and masses to the pages of new_table (int32 [B, new_pages], none of them in
    use); `kept` holds the positions they had, -1 from new_lens on. The old pages are not written. Windows, documents
    and biases over the new pages count places there, not those positions."""
    return _native().kv_evict(cache, mass, page_table, kv_lens, keep, new_table, recent, first, new_lens, kept, stream)


def verify_drafts_workspace(B: int, k: int) -> int:
    """Bytes of workspace verify_drafts needs."""
    return int(load().fp8act_verify_drafts_workspace(B, k))


def verify_drafts(target_logits, draft_tokens, uniform, noise, temperature, draft_logits=None, n_draft=None,
                  accepted=None, tokens=None, accept_prob=None, workspace=None, stream=None):
    """Speculative sampling of drafted tokens -> (accepted int32 [B], tokens int32 [B, k+1], accept_prob fp32 [B, k]).

    target_logits [B, k+1, V] and draft_logits [B, k, V] (None: greedy drafts) bf16 or fp32,
    draft_tokens int32 [B, k], uniform fp32 [B, k], noise fp32 [B, V] (exponential, rate 1),
    temperature fp32 [B] (0 = greedy), n_draft int32 [B] (None: k each). `workspace`: a uint8 tensor
    of verify_drafts_workspace() bytes, kept by the caller per stream; without one the binding
    keeps its own per device and stream."""
    return _native().verify_drafts(target_logits, draft_tokens, uniform, noise, temperature, draft_logits, n_draft,
                                   accepted, tokens, accept_prob, workspace, stream)


def check_status(stream=None) -> int:
    """Synchronise the stream and return the library's device-side status."""
    return int(load().fp8act_check_status(_stream(stream)))


def set_wait_limit(limit_ns: int, withhold_first_load: bool = False) -> None:
    """Test hook of the tcgen05 kernels' failure path (see fp8act_set_wait_limit):
    the wall-time bound of their waits (negative = the 2 s default) and whether
    each CTA skips its first operand copy."""
    _check("fp8act_set_wait_limit", load().fp8act_set_wait_limit(int(limit_ns), 1 if withhold_first_load else 0))


def stream_read(src: torch.Tensor, sink: torch.Tensor, stream=None) -> None:
    """Diagnostic: read every byte of the CUDA tensor `src` once (the weight-stream
    floor), folding it into the int32 CUDA tensor `sink` (see fp8act_stream_read)."""
    if not src.is_cuda or not src.is_contiguous() or not sink.is_cuda or sink.dtype != torch.int32:
        raise TypeError("src must be a contiguous CUDA tensor and sink an int32 CUDA tensor")
    _check("fp8act_stream_read", load().fp8act_stream_read(src.data_ptr(), src.numel() * src.element_size(),
                                                           sink.data_ptr(), _stream(stream)))
