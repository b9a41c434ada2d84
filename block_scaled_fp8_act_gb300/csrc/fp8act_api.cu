// C ABI of libfp8act: argument checks, device checks, dispatch on M.
// The contract of every function is documented in include/fp8act.h.
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/fp8act.h"
#include "kernels.h"

namespace {

constexpr int kMaxDevices = 64;
constexpr int kGroup = 128;
constexpr int kSkinnyMaxM = 16;  // M up to this streams weights through mma.sync; above, tcgen05 kernels
constexpr unsigned long long kDefaultWaitNs = 2000000000ull;  // the tcgen05 kernels' default wait bound (2 s)

// Failure-path test hook (fp8act_set_wait_limit): < 0 = the default bound.
std::atomic<long long> g_wait_limit_ns{-1};
std::atomic<int> g_withhold_first_load{0};

// Per-device facts looked up once: -1 = unknown, 0 = unsupported, else SM count.
std::atomic<int> g_device_sms[kMaxDevices];
std::atomic<bool> g_device_init[kMaxDevices];

// SM count of the current device if it is a compute-capability 10.3 part, 0 otherwise.
int current_device_sms(int* status) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        *status = FP8ACT_ERR_DEVICE;
        return 0;
    }
    if (!g_device_init[dev].load(std::memory_order_acquire)) {
        int major = 0, minor = 0, sms = 0;
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        cudaGetLastError();
        g_device_sms[dev].store((major == 10 && minor == 3) ? sms : 0, std::memory_order_relaxed);
        g_device_init[dev].store(true, std::memory_order_release);
    }
    const int sms = g_device_sms[dev].load(std::memory_order_relaxed);
    *status = sms > 0 ? FP8ACT_OK : FP8ACT_ERR_DEVICE;
    return sms;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int launch_status(cudaError_t e) {
    if (e == cudaSuccess) return FP8ACT_OK;
    return FP8ACT_ERR_LAUNCH;
}

// K: positive multiple of 128; rows*K must fit in int64 and each of M, N, K in int.
int check_k(int K) { return (K <= 0 || K % kGroup) ? FP8ACT_ERR_SHAPE : FP8ACT_OK; }

// The GEMM kernel for M tokens: weight streaming through mma.sync up to 16,
// the swap-AB tcgen05 weight-streaming kernel up to 128, token-tiled tcgen05
// tiles above (prefill).
cudaError_t launch_gemm_any(const uint8_t* q, const float* sa, const uint8_t* w, const float* sw, int M, int N,
                            int K, void* out, bool out_f32, int sms, cudaStream_t s) {
    if (M <= kSkinnyMaxM) return fp8act::launch_gemm_skinny(q, sa, w, sw, M, N, K, out, out_f32, sms, s);
    if (M <= fp8act::kMidMaxM) {
        // cudaErrorNotSupported: the CTA's scale table would not fit (very long K
        // on few tiles); the token-tiled kernel below handles any shape.
        const cudaError_t e = fp8act::launch_gemm_midm(q, sa, w, sw, M, N, K, out, out_f32, sms, s);
        if (e != cudaErrorNotSupported) return e;
    }
    return fp8act::launch_gemm_tc(q, sa, w, sw, M, N, K, out, out_f32, sms, s);
}

int gemm_common(const void* q, const float* sa, const void* w, const float* sw, int M, int N, int K, void* out,
                bool out_f32, void* stream) {
    if (M < 0 || N < 0) return FP8ACT_ERR_SHAPE;
    if (int st = check_k(K)) return st;
    if (M == 0 || N == 0) return FP8ACT_OK;
    if (!q || !sa || !w || !sw || !out) return FP8ACT_ERR_NULL;
    if (!aligned(q, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(sa, 4) || !aligned(sw, 4))
        return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint8_t* q8 = static_cast<const uint8_t*>(q);
    const uint8_t* w8 = static_cast<const uint8_t*>(w);
    return launch_status(launch_gemm_any(q8, sa, w8, sw, M, N, K, out, out_f32, sms, s));
}

constexpr int kMaxGrouped = 16;
constexpr int kTileGroupMaxM = 128;  // one token tile: the grouped tile launch takes these

// The single-call checks of one GEMM problem (no launch); OK for an empty one.
int check_gemm(const fp8act_gemm_problem& p) {
    if (p.M < 0 || p.N < 0) return FP8ACT_ERR_SHAPE;
    if (int st = check_k(p.K)) return st;
    if (p.M == 0 || p.N == 0) return FP8ACT_OK;
    if (!p.q_e4m3 || !p.sa || !p.w_e4m3 || !p.sw || !p.out) return FP8ACT_ERR_NULL;
    if (!aligned(p.q_e4m3, 16) || !aligned(p.w_e4m3, 16) || !aligned(p.out, 16) || !aligned(p.sa, 4) ||
        !aligned(p.sw, 4))
        return FP8ACT_ERR_ALIGN;
    return FP8ACT_OK;
}

int gemm_grouped_common(const fp8act_gemm_problem* problems, int count, bool out_f32, void* stream) {
    if (count < 0 || count > kMaxGrouped) return FP8ACT_ERR_SHAPE;
    if (count == 0) return FP8ACT_OK;
    if (!problems) return FP8ACT_ERR_NULL;
    bool any = false;
    for (int i = 0; i < count; ++i) {
        if (int st = check_gemm(problems[i])) return st;
        any = any || (problems[i].M > 0 && problems[i].N > 0);
    }
    if (!any) return FP8ACT_OK;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    fp8act::GemmProblem skinny[kMaxGrouped];
    int n_skinny = 0;
    for (int i = 0; i < count; ++i) {
        const fp8act_gemm_problem& p = problems[i];
        if (p.M == 0 || p.N == 0 || p.M > kSkinnyMaxM) continue;
        skinny[n_skinny++] = {static_cast<const uint8_t*>(p.q_e4m3), p.sa, static_cast<const uint8_t*>(p.w_e4m3),
                              p.sw, p.out, p.M, p.N, p.K};
    }
    if (int e = launch_status(fp8act::launch_gemm_skinny_grouped(skinny, n_skinny, out_f32, s))) return e;
    auto one = [&](const fp8act::GemmProblem& p) {
        return launch_status(launch_gemm_any(p.q, p.sa, p.w, p.sw, p.M, p.N, p.K, p.out, out_f32, sms, s));
    };
    // Problems of the tile kernel, grouped by width: one token tile each (16 < M
    // <= 128: 128-wide weight tiles, a chunk is worth one launch once its tiles
    // fill the SMs) and several (M > 128: 256-wide tiles, once they fill two
    // waves, the single-problem kernel's own rule for wide tiles). One grouped
    // persistent launch per chunk of up to gemm_tc_grouped_capacity()
    // problems; a chunk with fewer tiles, one launch per problem.
    fp8act::GemmProblem narrow[kMaxGrouped], wide[kMaxGrouped];
    int n_narrow = 0, n_wide = 0;
    for (int i = 0; i < count; ++i) {
        const fp8act_gemm_problem& p = problems[i];
        if (p.M <= kSkinnyMaxM || p.N == 0) continue;
        const fp8act::GemmProblem g = {static_cast<const uint8_t*>(p.q_e4m3), p.sa,
                                       static_cast<const uint8_t*>(p.w_e4m3), p.sw, p.out, p.M, p.N, p.K};
        if (p.M <= kTileGroupMaxM)
            narrow[n_narrow++] = g;
        else
            wide[n_wide++] = g;
    }
    const int cap = fp8act::gemm_tc_grouped_capacity();
    auto run_chunks = [&](const fp8act::GemmProblem* list, int n_list, int bn, int64_t min_tiles) -> int {
        for (int c0 = 0; c0 < n_list; c0 += cap) {
            const int n = n_list - c0 < cap ? n_list - c0 : cap;
            int64_t tiles = 0;
            for (int j = 0; j < n; ++j)
                tiles += static_cast<int64_t>((list[c0 + j].M + 127) / 128) * ((list[c0 + j].N + bn - 1) / bn);
            const cudaError_t g = tiles >= min_tiles
                                      ? fp8act::launch_gemm_tc_grouped(list + c0, n, out_f32, sms, s)
                                      : cudaErrorNotSupported;
            if (g == cudaErrorNotSupported) {  // too few tiles to fill the grid (or too many to list)
                for (int j = 0; j < n; ++j)
                    if (int e = one(list[c0 + j])) return e;
            } else if (int e = launch_status(g)) {
                return e;
            }
        }
        return FP8ACT_OK;
    };
    if (int e = run_chunks(narrow, n_narrow, 128, sms)) return e;
    if (int e = run_chunks(wide, n_wide, 256, 2 * static_cast<int64_t>(sms))) return e;
    return FP8ACT_OK;
}

int linear_common(const void* x, const void* w, const float* sw, int M, int N, int K, void* out, bool out_f32,
                  void* stream) {
    if (M < 0 || N < 0) return FP8ACT_ERR_SHAPE;
    if (int st = check_k(K)) return st;
    if (M == 0 || N == 0) return FP8ACT_OK;
    if (!fp8act::fused_fits(M, K)) return FP8ACT_ERR_SHAPE;
    if (!x || !w || !sw || !out) return FP8ACT_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(sw, 4)) return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    return launch_status(fp8act::launch_linear_fused(x, static_cast<const uint8_t*>(w), sw, M, N, K, out, out_f32,
                                                     sms, static_cast<cudaStream_t>(stream)));
}

int w8a16_common(const void* x, const void* w, const float* sw, int M, int N, int K, void* out, bool out_f32,
                 void* stream) {
    if (M < 0 || N < 0) return FP8ACT_ERR_SHAPE;
    if (int st = check_k(K)) return st;
    if (M == 0 || N == 0) return FP8ACT_OK;
    if (!x || !w || !sw || !out) return FP8ACT_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(sw, 4)) return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    return launch_status(fp8act::launch_gemm_w8a16(x, static_cast<const uint8_t*>(w), sw, M, N, K, out, out_f32, sms,
                                                   static_cast<cudaStream_t>(stream)));
}

constexpr int kNormMaxK = 32768;  // one CTA holds a row: 1024 threads x 4 chunks of 8
constexpr int kMaxQLen = 1 << 20;
constexpr int kMaxVerifyB = 65535;
constexpr int kMaxRopeHeads = 1 << 20, kMaxRopeAxes = 4;

// The cache's own rules; fills the launchers' form of it.
int check_cache(const fp8act_kv_cache* c, fp8act::KvCache* out) {
    if (!c) return FP8ACT_ERR_NULL;
    const int ps = c->page_size;
    if (c->num_pages < 0 || c->kv_heads <= 0 || ps < 16 || ps > 256 || (ps & (ps - 1)) ||
        (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256))
        return FP8ACT_ERR_SHAPE;
    if (c->num_pages > 0) {
        if (!c->k_e4m3 || !c->v_e4m3 || !c->k_scale || !c->v_scale) return FP8ACT_ERR_NULL;
        if (!aligned(c->k_e4m3, 16) || !aligned(c->v_e4m3, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
            return FP8ACT_ERR_ALIGN;
    }
    int log2 = 4;
    while ((1 << log2) < ps) ++log2;
    *out = {static_cast<uint8_t*>(c->k_e4m3), static_cast<uint8_t*>(c->v_e4m3), c->k_scale, c->v_scale,
            c->num_pages, log2, c->kv_heads, c->head_dim};
    return FP8ACT_OK;
}

// What attention over the cache and its weights have in common.
int check_rows(const fp8act::KvCache& c, int64_t q_stride, int max_pages, int batch, int tokens, int max_q_len, int q_heads,
               float softmax_scale) {
    if (batch < 0 || tokens < 0 || max_pages < 0 || max_q_len < 0 || max_q_len > kMaxQLen || q_heads <= 0 ||
        q_heads % c.heads || q_heads / c.heads > 256 || q_stride < static_cast<int64_t>(q_heads) * c.head_dim ||
        static_cast<int64_t>(max_pages) << c.page_log2 > 0x7FFFFF00 ||
        static_cast<int64_t>(tokens) * (q_heads / c.heads) > 0x7FFFFF00)
        return FP8ACT_ERR_SHAPE;
    if (!(softmax_scale > 0.0f) || softmax_scale > 3e38f) return FP8ACT_ERR_SHAPE;
    return FP8ACT_OK;
}

// The caller's score function as the kernels take it.
int check_scores(const fp8act_scores* in, fp8act::Scores* out) {
    *out = {};
    out->unit = 1.0f;
    if (!in) return FP8ACT_OK;
    if (in->window < 0 || !(in->soft_cap == 0.0f || (in->soft_cap >= 1e-30f && in->soft_cap <= 1e30f)))
        return FP8ACT_ERR_SHAPE;
    out->capped = in->soft_cap > 0.0f;
    if (out->capped) out->unit = in->soft_cap * 1.4426950408889634f;
    out->window = in->window;
    out->prefix = in->prefix_lens;
    out->first = in->first;
    out->slopes = in->slopes;
    out->kind = out->capped || in->slopes                             ? fp8act::ScoreKind::kChanged
                : in->window || in->prefix_lens || in->first ? fp8act::ScoreKind::kMasked
                                                              : fp8act::ScoreKind::kPlain;
    return FP8ACT_OK;
}
bool aligned_scores(const fp8act::Scores& s) { return aligned(s.prefix, 4) && aligned(s.first, 4) && aligned(s.slopes, 4); }

}  // namespace

namespace fp8act {
unsigned long long tile_wait_limit_ns() {
    const long long v = g_wait_limit_ns.load(std::memory_order_relaxed);
    return v < 0 ? kDefaultWaitNs : static_cast<unsigned long long>(v);
}
bool tile_withhold_first_load() { return g_withhold_first_load.load(std::memory_order_relaxed) != 0; }
}  // namespace fp8act

extern "C" {

int fp8_act_quant(const void* x_bf16, int M, int K, void* q_e4m3, float* sa, void* stream) {
    if (M < 0) return FP8ACT_ERR_SHAPE;
    if (int st = check_k(K)) return st;
    if (M == 0) return FP8ACT_OK;
    if (!x_bf16 || !q_e4m3 || !sa) return FP8ACT_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(q_e4m3, 16) || !aligned(sa, 4)) return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    return launch_status(fp8act::launch_act_quant(x_bf16, M, K, q_e4m3, sa, sms, static_cast<cudaStream_t>(stream)));
}

int fp8_weight_quant(const void* w_bf16, int N, int K, void* w_e4m3, float* sw, void* stream) {
    if (N < 0) return FP8ACT_ERR_SHAPE;
    if (int st = check_k(K)) return st;
    if (N == 0) return FP8ACT_OK;
    if (!w_bf16 || !w_e4m3 || !sw) return FP8ACT_ERR_NULL;
    if (!aligned(w_bf16, 16) || !aligned(w_e4m3, 16) || !aligned(sw, 4)) return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    current_device_sms(&st);
    if (st) return st;
    return launch_status(fp8act::launch_weight_quant(w_bf16, N, K, w_e4m3, sw, static_cast<cudaStream_t>(stream)));
}

int fp8_block_gemm(const void* q_e4m3, const float* sa, const void* w_e4m3, const float* sw, int M, int N, int K,
                   void* out_bf16, void* stream) {
    return gemm_common(q_e4m3, sa, w_e4m3, sw, M, N, K, out_bf16, false, stream);
}

int fp8_block_gemm_f32(const void* q_e4m3, const float* sa, const void* w_e4m3, const float* sw, int M, int N,
                       int K, float* out_f32, void* stream) {
    return gemm_common(q_e4m3, sa, w_e4m3, sw, M, N, K, out_f32, true, stream);
}

int fp8_block_gemm_w8a16(const void* x_bf16, const void* w_e4m3, const float* sw, int M, int N, int K,
                         void* out_bf16, void* stream) {
    return w8a16_common(x_bf16, w_e4m3, sw, M, N, K, out_bf16, false, stream);
}

int fp8_block_gemm_w8a16_f32(const void* x_bf16, const void* w_e4m3, const float* sw, int M, int N, int K,
                             float* out_f32, void* stream) {
    return w8a16_common(x_bf16, w_e4m3, sw, M, N, K, out_f32, true, stream);
}

int fp8_linear(const void* x_bf16, const void* w_e4m3, const float* sw, int M, int N, int K, void* out_bf16,
               void* stream) {
    return linear_common(x_bf16, w_e4m3, sw, M, N, K, out_bf16, false, stream);
}

int fp8_linear_f32(const void* x_bf16, const void* w_e4m3, const float* sw, int M, int N, int K, float* out_f32,
                   void* stream) {
    return linear_common(x_bf16, w_e4m3, sw, M, N, K, out_f32, true, stream);
}

int fp8_act_quant_grouped(const fp8act_quant_problem* problems, int count, void* stream) {
    if (count < 0 || count > kMaxGrouped) return FP8ACT_ERR_SHAPE;
    if (count == 0) return FP8ACT_OK;
    if (!problems) return FP8ACT_ERR_NULL;
    fp8act::ActQuantProblem probs[kMaxGrouped];
    int n = 0;
    for (int i = 0; i < count; ++i) {
        const fp8act_quant_problem& p = problems[i];
        if (p.M < 0) return FP8ACT_ERR_SHAPE;
        if (int st = check_k(p.K)) return st;
        if (p.M == 0) continue;
        if (!p.x_bf16 || !p.q_e4m3 || !p.sa) return FP8ACT_ERR_NULL;
        if (!aligned(p.x_bf16, 16) || !aligned(p.q_e4m3, 16) || !aligned(p.sa, 4)) return FP8ACT_ERR_ALIGN;
        probs[n++] = {p.x_bf16, p.q_e4m3, p.sa, p.M, p.K};
    }
    if (n == 0) return FP8ACT_OK;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    return launch_status(fp8act::launch_act_quant_grouped(probs, n, sms, static_cast<cudaStream_t>(stream)));
}

int fp8_block_gemm_grouped(const fp8act_gemm_problem* problems, int count, void* stream) {
    return gemm_grouped_common(problems, count, false, stream);
}

int fp8_block_gemm_grouped_f32(const fp8act_gemm_problem* problems, int count, void* stream) {
    return gemm_grouped_common(problems, count, true, stream);
}

int fp8_rmsnorm_quant(const void* x_bf16, const void* residual_bf16, const void* weight_bf16, float eps,
                      float weight_offset, int M, int K, void* q_e4m3, float* sa, void* residual_out_bf16,
                      void* stream) {
    if (M < 0 || K > kNormMaxK) return FP8ACT_ERR_SHAPE;
    if (int st = check_k(K)) return st;
    if (M == 0) return FP8ACT_OK;
    if (!x_bf16 || !weight_bf16 || !q_e4m3 || !sa || !residual_bf16 != !residual_out_bf16) return FP8ACT_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(residual_bf16, 16) || !aligned(weight_bf16, 16) || !aligned(q_e4m3, 16) ||
        !aligned(residual_out_bf16, 16) || !aligned(sa, 4))
        return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    current_device_sms(&st);
    if (st) return st;
    return launch_status(fp8act::launch_rmsnorm_quant(x_bf16, residual_bf16, weight_bf16, eps, weight_offset, M, K,
                                                      q_e4m3, sa, residual_out_bf16, static_cast<cudaStream_t>(stream)));
}

int fp8_silu_mul_quant(const void* gate_up_bf16, int M, int I, void* q_e4m3, float* sa, void* stream) {
    if (M < 0) return FP8ACT_ERR_SHAPE;
    if (int st = check_k(I)) return st;
    if (M == 0) return FP8ACT_OK;
    if (!gate_up_bf16 || !q_e4m3 || !sa) return FP8ACT_ERR_NULL;
    if (!aligned(gate_up_bf16, 16) || !aligned(q_e4m3, 16) || !aligned(sa, 4)) return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    return launch_status(
        fp8act::launch_silu_mul_quant(gate_up_bf16, M, I, q_e4m3, sa, sms, static_cast<cudaStream_t>(stream)));
}

int fp8_kv_append(const void* k_bf16, const void* v_bf16, const int64_t* slots, int T, int64_t k_stride,
                  int64_t v_stride, const fp8act_kv_cache* cache, void* stream) {
    fp8act::KvCache c;
    if (int st = check_cache(cache, &c)) return st;
    const int64_t width = static_cast<int64_t>(c.heads) * c.head_dim;
    if (T < 0 || k_stride < width || v_stride < width) return FP8ACT_ERR_SHAPE;
    if (T > (int64_t{1} << 38) / width) return FP8ACT_ERR_SHAPE;  // keeps the grid within 2^31 CTAs
    if (T == 0) return FP8ACT_OK;
    if (!k_bf16 || !v_bf16 || !slots) return FP8ACT_ERR_NULL;
    if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || !aligned(slots, 8) || k_stride % 8 || v_stride % 8)
        return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    current_device_sms(&st);
    if (st) return st;
    return launch_status(fp8act::launch_kv_append(k_bf16, v_bf16, slots, T, k_stride, v_stride, c,
                                                  static_cast<cudaStream_t>(stream)));
}

int fp8_rope_append(const void* q_bf16, const void* k_bf16, const void* v_bf16, int64_t q_stride, int64_t k_stride,
                    int64_t v_stride, const void* q_weight_bf16, const void* k_weight_bf16, float eps,
                    float weight_offset, const int64_t* positions, const double* inv_freq, const int* axis, int n_axes,
                    int rot_dim, int interleaved, float rope_scale, const int64_t* slots, int T, int q_heads,
                    const fp8act_kv_cache* cache, void* q_out_bf16, void* stream) {
    fp8act::KvCache c;
    if (int st = check_cache(cache, &c)) return st;
    const int64_t width = static_cast<int64_t>(c.heads) * c.head_dim;
    if (T < 0 || q_heads <= 0 || q_heads > kMaxRopeHeads || c.heads > kMaxRopeHeads || n_axes < 1 ||
        n_axes > kMaxRopeAxes || rot_dim < 0 || rot_dim > c.head_dim || rot_dim % 16 || k_stride < width ||
        v_stride < width || q_stride < static_cast<int64_t>(q_heads) * c.head_dim)
        return FP8ACT_ERR_SHAPE;
    if (T == 0) return FP8ACT_OK;
    if (!q_bf16 || !k_bf16 || !v_bf16 || !positions || !slots || !q_out_bf16 || (rot_dim > 0 && !inv_freq))
        return FP8ACT_ERR_NULL;
    if (!aligned(q_bf16, 16) || !aligned(k_bf16, 16) || !aligned(v_bf16, 16) || q_stride % 8 || k_stride % 8 ||
        v_stride % 8 || !aligned(q_weight_bf16, 16) || !aligned(k_weight_bf16, 16) || !aligned(positions, 8) ||
        !aligned(inv_freq, 8) || !aligned(axis, 4) || !aligned(slots, 8) || !aligned(q_out_bf16, 16))
        return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    using bf16 = const uint16_t*;
    const fp8act::RopeProblem p = {static_cast<bf16>(q_bf16), static_cast<bf16>(k_bf16), static_cast<bf16>(v_bf16),
                                   q_stride, k_stride, v_stride, static_cast<bf16>(q_weight_bf16),
                                   static_cast<bf16>(k_weight_bf16), eps, weight_offset, rope_scale, positions,
                                   inv_freq, axis, slots, T, q_heads, rot_dim, n_axes, interleaved != 0, c, q_out_bf16};
    return launch_status(fp8act::launch_rope_append(p, sms, static_cast<cudaStream_t>(stream)));
}

size_t fp8_kv_attention_workspace(int max_q_len, int q_heads, const fp8act_kv_cache* cache) {
    fp8act::KvCache c;
    if (check_cache(cache, &c) || max_q_len < 0 || max_q_len > kMaxQLen || q_heads <= 0 || q_heads % c.heads) return 0;
    return fp8act::kv_attention_workspace(max_q_len, q_heads / c.heads, c.head_dim);
}

int fp8_kv_attention(const void* q_bf16, int64_t q_stride, const int* cu_q, const int* kv_lens, const int* page_table,
                     int max_pages, int batch, int tokens, int max_q_len, int q_heads, float softmax_scale,
                     const fp8act_kv_cache* cache, void* out_bf16, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
    return fp8_kv_attention_scored(q_bf16, q_stride, cu_q, kv_lens, page_table, max_pages, batch, tokens, max_q_len,
                                   q_heads, softmax_scale, nullptr, cache, out_bf16, lse, workspace, workspace_bytes,
                                   stream);
}

int fp8_kv_attention_scored(const void* q_bf16, int64_t q_stride, const int* cu_q, const int* kv_lens,
                            const int* page_table, int max_pages, int batch, int tokens, int max_q_len, int q_heads,
                            float softmax_scale, const fp8act_scores* scores, const fp8act_kv_cache* cache,
                            void* out_bf16, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    fp8act::KvCache c;
    if (int st = check_cache(cache, &c)) return st;
    if (int st = check_rows(c, q_stride, max_pages, batch, tokens, max_q_len, q_heads, softmax_scale)) return st;
    fp8act::Scores s;
    if (int st = check_scores(scores, &s)) return st;
    if (batch == 0 || tokens == 0) return FP8ACT_OK;
    if (c.num_pages == 0) return FP8ACT_ERR_SHAPE;
    if (!q_bf16 || !cu_q || !kv_lens || !out_bf16 || !workspace || (max_pages > 0 && !page_table))
        return FP8ACT_ERR_NULL;
    if (!aligned(q_bf16, 16) || q_stride % 8 || !aligned(out_bf16, 16) || !aligned(workspace, 16) || !aligned(cu_q, 4) ||
        !aligned(kv_lens, 4) || !aligned(page_table, 4) || !aligned(lse, 4) || !aligned_scores(s))
        return FP8ACT_ERR_ALIGN;
    if (workspace_bytes < fp8act::kv_attention_workspace(max_q_len, q_heads / c.heads, c.head_dim))
        return FP8ACT_ERR_SHAPE;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    const fp8act::AttentionProblem p = {q_bf16,    q_stride,  cu_q,          kv_lens, page_table, max_pages,
                                        batch,     tokens,    max_q_len,     q_heads / c.heads,   softmax_scale,
                                        c,         out_bf16,  lse,           workspace,           s};
    return launch_status(fp8act::launch_kv_attention(p, sms, static_cast<cudaStream_t>(stream)));
}

int fp8_kv_attention_mass(const void* q_bf16, int64_t q_stride, const int* cu_q, const int* kv_lens,
                          const int* page_table, int max_pages, int batch, int tokens, int max_q_len, int q_heads,
                          float softmax_scale, const fp8act_scores* scores, const fp8act_kv_cache* cache,
                          const float* lse, float* mass, int accumulate, const int* old_lens, void* stream) {
    fp8act::KvCache c;
    if (int st = check_cache(cache, &c)) return st;
    if (int st = check_rows(c, q_stride, max_pages, batch, tokens, max_q_len, q_heads, softmax_scale)) return st;
    fp8act::Scores s;
    if (int st = check_scores(scores, &s)) return st;
    if (batch == 0) return FP8ACT_OK;
    if (c.num_pages == 0) return FP8ACT_ERR_SHAPE;
    if (!cu_q || !kv_lens || !mass || (tokens > 0 && (!q_bf16 || !lse)) || (max_pages > 0 && !page_table))
        return FP8ACT_ERR_NULL;
    if (!aligned(q_bf16, 16) || q_stride % 8 || !aligned(cu_q, 4) || !aligned(kv_lens, 4) || !aligned(page_table, 4) ||
        !aligned(lse, 4) || !aligned(mass, 16) || !aligned(old_lens, 4) || !aligned_scores(s))
        return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    const fp8act::MassProblem p = {q_bf16, q_stride, cu_q, kv_lens, page_table, max_pages, batch, tokens, max_q_len,
                                   q_heads / c.heads, softmax_scale, c, lse, mass, accumulate != 0, old_lens, s};
    return launch_status(fp8act::launch_kv_mass(p, sms, static_cast<cudaStream_t>(stream)));
}

int fp8_kv_evict(const fp8act_kv_cache* cache, float* mass, const int* page_table, int max_pages, const int* kv_lens,
                 const int* keep, const int* new_table, int new_pages, int batch, int recent, int first, int* new_lens,
                 int* kept, void* stream) {
    fp8act::KvCache c;
    if (int st = check_cache(cache, &c)) return st;
    if (batch < 0 || max_pages < 0 || new_pages < 0 || recent < 0 || first < 0 ||
        static_cast<int64_t>(max_pages) << c.page_log2 > 0x7FFFFF00 ||
        static_cast<int64_t>(new_pages) << c.page_log2 > 0x7FFFFF00)
        return FP8ACT_ERR_SHAPE;
    // (CTAs of a launch: 8 per sequence and head, or one per 64 places)
    const int64_t items = static_cast<int64_t>(batch) * c.heads;
    if (items > 0x7FFFFFFF / 8 || items * ((static_cast<int64_t>(new_pages) << c.page_log2) / 64 + 1) > 0x7FFFFFFF)
        return FP8ACT_ERR_SHAPE;
    if (batch == 0) return FP8ACT_OK;
    if (c.num_pages == 0) return FP8ACT_ERR_SHAPE;
    if (!mass || !kv_lens || !keep || !new_lens || (max_pages > 0 && !page_table) || (new_pages > 0 && (!new_table || !kept)))
        return FP8ACT_ERR_NULL;
    if (new_lens == kv_lens || new_lens == keep) return FP8ACT_ERR_SHAPE;
    if (!aligned(mass, 16) || !aligned(page_table, 4) || !aligned(kv_lens, 4) || !aligned(keep, 4) ||
        !aligned(new_table, 4) || !aligned(new_lens, 4) || !aligned(kept, 4))
        return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    const fp8act::EvictProblem p = {c, mass, page_table, kv_lens, keep, new_table, max_pages, new_pages, batch, recent,
                                    first, new_lens, kept};
    return launch_status(fp8act::launch_kv_evict(p, sms, static_cast<cudaStream_t>(stream)));
}

int fp8act_verify_drafts(const void* target, const void* draft, int logits_f32, const int* draft_tokens,
                         const float* uniform, const float* noise, const float* temperature, const int* n_draft, int B,
                         int k, int V, int* accepted, int* tokens, float* accept_prob, void* workspace,
                         size_t workspace_bytes, void* stream) {
    if (B < 0 || k < 0 || k > fp8act::kMaxDrafts || V <= 0 || V > 0x7FFFFF00 / 16) return FP8ACT_ERR_SHAPE;
    if (B > kMaxVerifyB) return FP8ACT_ERR_SHAPE;
    if (B == 0) return FP8ACT_OK;
    if (!target || !noise || !temperature || !accepted || !tokens || !workspace || (k > 0 && (!draft_tokens || !uniform)))
        return FP8ACT_ERR_NULL;
    if (!aligned(target, 16) || !aligned(draft, 16) || !aligned(draft_tokens, 4) || !aligned(uniform, 4) ||
        !aligned(noise, 4) || !aligned(temperature, 4) || !aligned(n_draft, 4) || !aligned(accepted, 4) ||
        !aligned(tokens, 4) || !aligned(accept_prob, 4) || !aligned(workspace, 16))
        return FP8ACT_ERR_ALIGN;
    if (workspace_bytes < fp8act::verify_drafts_workspace(B, k)) return FP8ACT_ERR_SHAPE;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    const fp8act::VerifyProblem p = {target,  k > 0 ? draft : nullptr, draft_tokens, uniform, noise, temperature,
                                     n_draft, B, k, V, logits_f32 != 0, accepted, tokens, accept_prob, workspace};
    return launch_status(fp8act::launch_verify_drafts(p, sms, static_cast<cudaStream_t>(stream)));
}

size_t fp8act_verify_drafts_workspace(int B, int k) {
    if (B < 0 || B > kMaxVerifyB || k < 0 || k > fp8act::kMaxDrafts) return 0;
    return fp8act::verify_drafts_workspace(B, k);
}

const char* fp8act_strerror(int status) {
    switch (status) {
        case FP8ACT_OK: return "ok";
        case FP8ACT_ERR_NULL: return "a required pointer is NULL";
        case FP8ACT_ERR_SHAPE:
            return "bad shape: M, N must be >= 0 and K a positive multiple of 128 (grouped calls: at most 16 "
                   "problems; fp8_linear: min(8, M) rows of K codes and scales must fit in 200 KiB; the operators "
                   "between the linear layers: see the limits at each)";
        case FP8ACT_ERR_ALIGN: return "misaligned pointer: tensors need 16-byte, scales 4-byte alignment";
        case FP8ACT_ERR_LAUNCH: return "kernel launch failed";
        case FP8ACT_ERR_TIMEOUT: return "a kernel gave up a bounded wait (device-side timeout)";
        case FP8ACT_ERR_DEVICE: return "no current CUDA device of compute capability 10.3 (GB300)";
        case FP8ACT_ERR_CUDA: return "CUDA runtime error";
        case FP8ACT_ERR_INDEX: return "a slot, page, length or token index on the device was out of range";
        default: return "unknown fp8act status";
    }
}

int fp8act_check_status(void* stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return FP8ACT_ERR_CUDA;
    }
    const unsigned int tc = fp8act::read_and_clear_tc_error();
    const unsigned int mid = fp8act::read_and_clear_midm_error();
    const unsigned int rd = fp8act::read_and_clear_read_error();
    const unsigned int index = fp8act::read_and_clear_kv_index_error() | fp8act::read_and_clear_rope_index_error() |
                               fp8act::read_and_clear_attn_index_error() | fp8act::read_and_clear_mass_index_error() |
                               fp8act::read_and_clear_evict_index_error() |
                               fp8act::read_and_clear_verify_index_error();
    const unsigned int at = fp8act::read_and_clear_attn_timeout() | fp8act::read_and_clear_mass_timeout();
    if (tc | mid | rd | at) return FP8ACT_ERR_TIMEOUT;
    return index ? FP8ACT_ERR_INDEX : FP8ACT_OK;
}

int fp8act_set_wait_limit(long long limit_ns, int withhold_first_load) {
    g_wait_limit_ns.store(limit_ns, std::memory_order_relaxed);
    g_withhold_first_load.store(withhold_first_load ? 1 : 0, std::memory_order_relaxed);
    return FP8ACT_OK;
}

int fp8act_stream_read(const void* src, size_t bytes, unsigned int* sink, void* stream) {
    if (bytes == 0) return FP8ACT_OK;
    if (!src || !sink) return FP8ACT_ERR_NULL;
    if (!aligned(src, 16) || !aligned(sink, 4) || bytes % 16) return FP8ACT_ERR_ALIGN;
    int st = FP8ACT_OK;
    const int sms = current_device_sms(&st);
    if (st) return st;
    return launch_status(fp8act::launch_stream_read(src, static_cast<int64_t>(bytes), sink, sms,
                                                    static_cast<cudaStream_t>(stream)));
}

int fp8act_version(void) { return 300; }

}  // extern "C"
