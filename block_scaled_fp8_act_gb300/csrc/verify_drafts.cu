// Verification of drafted tokens against the target model's logits.
//
// Row j of a sequence holds the target's logits after j accepted drafts and
// the draft model's logits that token j was drawn from. With p_j and q_j their
// softmaxes at the sequence's temperature, draft x_j is accepted while
//   u_j < min(1, p_j(x_j) / q_j(x_j)),
// and the token after the accepted ones is drawn from max(p - q, 0) (rejected)
// or from p (all accepted) as argmax_v w_v / e_v with given exponential noise
// e, which draws v with probability w_v / sum w. No cumulative sum is taken,
// so no draw depends on the order of one.
//
// One thread-block cluster per sequence; its CTAs share the vocabulary.
// Pass 1 reads every row once for its maximum and sum (fp32, running rescale;
// a warp per part of a row), the parts meet through distributed shared
// memory, every CTA decides the acceptance alike, and pass 2 reads the one row
// (or pair) drawn from, by then in L2, with the noise.
#include <cfloat>

#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {
namespace {

__device__ unsigned int g_verify_index_error;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = 2 * kMaxDrafts + 1;
constexpr int kMaxParts = 8;
constexpr int kMaxCluster = 16;
constexpr float kNegInf = -__builtin_huge_valf();

// Maximum, sum of exponentials below it, and (for temperature 0) the first index of the maximum.
struct Stat {
    float m, s;
    int at;
};

__device__ __forceinline__ float clean(float v) { return fminf(fmaxf(v, kNegInf), FLT_MAX); }  // NaN counts as masked

template <bool kF32>
struct Row {
    const uint8_t* base;
    int V;
    static constexpr int kBytes = kF32 ? 4 : 2;
    static constexpr int kPer = 16 / kBytes;  // elements per 16-byte vector
    __device__ __forceinline__ float at(int i) const {
        if (kF32) return clean(ld_dep_f32(reinterpret_cast<const float*>(base) + i));
        uint16_t v;
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(base + 2 * static_cast<int64_t>(i)) : "memory");
        return clean(__uint_as_float(static_cast<uint32_t>(v) << 16));
    }
    // Elements before the first 16-byte boundary (rows of an odd vocabulary start anywhere).
    __device__ __forceinline__ int head() const {
        const int h = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / kBytes;
        return h < V ? h : V;
    }
    __device__ __forceinline__ void vec(int i, float (&f)[kPer]) const {
        const uint4 v = ld_dep_v4(base + static_cast<int64_t>(i) * kBytes);
        if constexpr (kF32) {
            f[0] = clean(__uint_as_float(v.x));
            f[1] = clean(__uint_as_float(v.y));
            f[2] = clean(__uint_as_float(v.z));
            f[3] = clean(__uint_as_float(v.w));
        } else {
            unpack_bf16x8(v, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = clean(f[j]);
        }
    }
};

__device__ __forceinline__ float exp_below(float v, float m, float c) { return v > kNegInf ? ex2((v - m) * c) : 0.0f; }

__device__ __forceinline__ void join(Stat& a, const Stat& b, float c) {
    const float m = fmaxf(a.m, b.m);
    const float fa = a.m > kNegInf ? ex2((a.m - m) * c) : 0.0f, fb = b.m > kNegInf ? ex2((b.m - m) * c) : 0.0f;
    if (b.m > a.m || (b.m == a.m && b.at < a.at)) a.at = b.at;
    a.s = a.s * fa + b.s * fb;
    a.m = m;
}

// The best draw so far: largest key, lowest index among equals.
struct Best {
    float key;
    int at;
};
__device__ __forceinline__ void better(Best& a, float key, int at) {
    if (key > a.key || (key == a.key && at < a.at)) {
        a.key = key;
        a.at = at;
    }
}

struct VerifyShared {
    Stat part[kMaxRows * kMaxParts];
    Stat mine[kMaxRows];   // this CTA's share of every row (read by the cluster)
    Stat row[kMaxRows];    // whole rows
    float prob[kMaxDrafts];
    int taken, n;
    Best warp_best[kWarps];
    Best best[2];          // this CTA's best draw (read by the cluster); one slot per pass
    Best all;
};

__device__ __forceinline__ Stat ld_cluster_stat(const Stat* p, uint32_t rank) {
    const uint32_t at = ptx::mapa_shared(ptx::smem_u32(p), rank);
    Stat r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r.m) : "r"(at) : "memory");
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r.s) : "r"(at + 4) : "memory");
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(r.at) : "r"(at + 8) : "memory");
    return r;
}
__device__ __forceinline__ Best ld_cluster_best(const Best* p, uint32_t rank) {
    const uint32_t at = ptx::mapa_shared(ptx::smem_u32(p), rank);
    Best r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r.key) : "r"(at) : "memory");
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(r.at) : "r"(at + 4) : "memory");
    return r;
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyProblem p, int cluster, int parts) {
    using R = Row<kF32>;
    __shared__ VerifyShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / cluster;
    const int rank = static_cast<int>(blockIdx.x) % cluster;
    const int V = p.V, k = p.k;
    const int targets = k + 1, rows = p.draft ? 2 * k + 1 : k + 1;
    const int64_t row_bytes = static_cast<int64_t>(V) * R::kBytes;
    const uint8_t* target = static_cast<const uint8_t*>(p.target) + static_cast<int64_t>(b) * targets * row_bytes;
    const uint8_t* draft =
        p.draft ? static_cast<const uint8_t*>(p.draft) + static_cast<int64_t>(b) * k * row_bytes : nullptr;
    auto row_of = [&](int r) { return R{r < targets ? target + r * row_bytes : draft + (r - targets) * row_bytes, V}; };
    const float* noise = p.noise + static_cast<int64_t>(b) * V;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const float temp = ld_dep_f32(p.temperature + b);
    const bool greedy = !(temp > 0.0f);
    const float c = greedy ? 1.0f : 1.4426950408889634f / temp;
    int n = p.n_draft ? ld_dep_s32(p.n_draft + b) : k;
    if (n < 0 || n > k) {
        if (threadIdx.x == 0) atomicOr(&g_verify_index_error, 1u);
        n = n < 0 ? 0 : k;
    }

    // Pass 1: maximum and sum of this CTA's share of every row.
    const int tasks = rows * parts;
    for (int task = warp; task < tasks; task += kWarps) {
        const int r = task / parts, share = rank * parts + task % parts, shares = cluster * parts;
        const R row = row_of(r);
        const int head = row.head(), vecs = (V - head) / R::kPer, tail = head + vecs * R::kPer;
        const int v0 = static_cast<int>(static_cast<int64_t>(vecs) * share / shares);
        const int v1 = static_cast<int>(static_cast<int64_t>(vecs) * (share + 1) / shares);
        Stat st = {kNegInf, 0.0f, 0x7FFFFFFF};
        auto one = [&](int i) {
            const Stat o = {row.at(i), 1.0f, i};
            if (o.m > kNegInf) join(st, o, c);
        };
        if (share == 0 && lane < head) one(lane);
        for (int v = v0 + lane; v < v1; v += 32) {
            float f[R::kPer];
            const int i = head + v * R::kPer;
            row.vec(i, f);
            float top = f[0];
#pragma unroll
            for (int j = 1; j < R::kPer; ++j) top = fmaxf(top, f[j]);
            if (top > st.m) {
                st.s *= st.m > kNegInf ? ex2((st.m - top) * c) : 0.0f;
                st.m = top;
                st.at = i;
#pragma unroll
                for (int j = R::kPer - 1; j >= 0; --j)
                    if (f[j] == top) st.at = i + j;
            }
#pragma unroll
            for (int j = 0; j < R::kPer; ++j) st.s += exp_below(f[j], st.m, c);
        }
        if (share == shares - 1 && tail + lane < V) one(tail + lane);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            Stat other;
            other.m = __shfl_xor_sync(0xffffffffu, st.m, o);
            other.s = __shfl_xor_sync(0xffffffffu, st.s, o);
            other.at = __shfl_xor_sync(0xffffffffu, st.at, o);
            join(st, other, c);
        }
        if (lane == 0) sh.part[task] = st;
    }
    __syncthreads();
    for (int r = threadIdx.x; r < rows; r += kThreads) {
        Stat st = sh.part[r * parts];
        for (int i = 1; i < parts; ++i) join(st, sh.part[r * parts + i], c);
        sh.mine[r] = st;
    }
    ptx::cluster_sync();
    for (int r = threadIdx.x; r < rows; r += kThreads) {
        Stat st = ld_cluster_stat(&sh.mine[r], 0);
        for (int i = 1; i < cluster; ++i) join(st, ld_cluster_stat(&sh.mine[r], i), c);
        sh.row[r] = st;
    }
    __syncthreads();

    // Acceptance, decided alike in every CTA.
    if (warp == 0) {
        int taken = 0;
        bool open = true;
        for (int j0 = 0; j0 < k; j0 += 32) {
            const int j = j0 + lane;
            bool ok = false;
            if (j < k) {
                const int x = ld_dep_s32(p.draft_tokens + static_cast<int64_t>(b) * k + j);
                const bool there = x >= 0 && x < V;
                if (!there && j < n && rank == 0) atomicOr(&g_verify_index_error, 1u);
                float prob = 0.0f;
                if (there && j < n) {
                    const Stat st = sh.row[j];
                    if (greedy) {
                        prob = st.m > kNegInf && st.at == x ? 1.0f : 0.0f;
                    } else {
                        const float px = st.s > 0.0f ? __fdiv_rn(exp_below(row_of(j).at(x), st.m, c), st.s) : 0.0f;
                        float qx = 1.0f;
                        if (draft) {
                            const Stat sd = sh.row[targets + j];
                            qx = sd.s > 0.0f ? __fdiv_rn(exp_below(row_of(targets + j).at(x), sd.m, c), sd.s) : 0.0f;
                        }
                        prob = qx > 0.0f ? fminf(__fdiv_rn(px, qx), 1.0f) : px > 0.0f ? 1.0f : 0.0f;
                    }
                }
                sh.prob[j] = prob;
                ok = j < n && ld_dep_f32(p.uniform + static_cast<int64_t>(b) * k + j) < prob;
            }
            const uint32_t no = ~__ballot_sync(0xffffffffu, ok);
            if (open) {
                const int run = no ? __ffs(no) - 1 : 32;
                taken += run;
                open = run == 32;
            }
        }
        if (lane == 0) sh.taken = taken;
    }
    __syncthreads();
    const int taken = sh.taken;

    // Pass 2: the draw. `rest` draws from max(p - q, 0), else from p.
    const Stat st = sh.row[taken];
    int token = -1;
    bool rest = taken < n && !greedy;
    if (greedy) {
        if (st.m > kNegInf) token = st.at;
    } else if (st.s > 0.0f) {
        const R row = row_of(taken);
        const int skip = rest && !draft ? ld_dep_s32(p.draft_tokens + static_cast<int64_t>(b) * k + taken) : -1;
        const float inv_p = __fdiv_rn(1.0f, st.s);
        const int i0 = static_cast<int>(static_cast<int64_t>(V) * rank / cluster);
        const int i1 = static_cast<int>(static_cast<int64_t>(V) * (rank + 1) / cluster);
        for (int pass = 0; pass < 2; ++pass) {
            Best best = {0.0f, 0x7FFFFFFF};
            Stat sd = {0.0f, 1.0f, 0};
            float inv_q = 0.0f;
            if (rest && draft) {
                sd = sh.row[targets + taken];
                inv_q = sd.s > 0.0f ? __fdiv_rn(1.0f, sd.s) : 0.0f;
            }
            for (int i = i0 + static_cast<int>(threadIdx.x); i < i1; i += kThreads) {
                float w = exp_below(row.at(i), st.m, c) * inv_p;
                if (rest) {
                    if (draft)
                        w -= exp_below(row_of(targets + taken).at(i), sd.m, c) * inv_q;
                    else if (i == skip)
                        w = 0.0f;
                }
                if (w > 0.0f) better(best, __fdiv_rn(w, ld_dep_f32(noise + i)), i);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                const float key = __shfl_xor_sync(0xffffffffu, best.key, o);
                const int at = __shfl_xor_sync(0xffffffffu, best.at, o);
                better(best, key, at);
            }
            if (lane == 0) sh.warp_best[warp] = best;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int w = 1; w < kWarps; ++w) better(best, sh.warp_best[w].key, sh.warp_best[w].at);
                sh.best[pass] = best;
            }
            ptx::cluster_sync();
            if (threadIdx.x == 0) {
                Best all = ld_cluster_best(&sh.best[pass], 0);
                for (int i = 1; i < cluster; ++i) {
                    const Best o = ld_cluster_best(&sh.best[pass], i);
                    better(all, o.key, o.at);
                }
                sh.all = all;
            }
            __syncthreads();
            if (sh.all.at < V) token = sh.all.at;
            if (token >= 0 || !rest) break;
            rest = false;  // p <= q everywhere to fp32: draw from p
        }
    }
    if (rank == 0) {
        int* out = p.tokens + static_cast<int64_t>(b) * targets;
        for (int j = threadIdx.x; j < targets; j += kThreads)
            out[j] = j < taken ? ld_dep_s32(p.draft_tokens + static_cast<int64_t>(b) * k + j) : j == taken ? token : -1;
        if (p.accept_prob)
            for (int j = threadIdx.x; j < k; j += kThreads) p.accept_prob[static_cast<int64_t>(b) * k + j] = sh.prob[j];
        if (threadIdx.x == 0) p.accepted[b] = taken;
    }
    ptx::cluster_sync();  // no CTA leaves while a peer may still read its shared memory
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyProblem& p, cudaStream_t stream) {
    const int rows = p.draft ? 2 * p.k + 1 : p.k + 1;
    int cluster = kMaxCluster;
    while (cluster > 1 && p.V < 2048 * cluster) cluster /= 2;
    // Parts per row: the count that keeps the CTA's warps busiest.
    int parts = 1;
    for (int i = 2; i <= kMaxParts; ++i)
        if (((rows * i + kWarps - 1) / kWarps) * parts < ((rows * parts + kWarps - 1) / kWarps) * i) parts = i;
    auto kernel = p.f32 ? verify_kernel<true> : verify_kernel<false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(p.B) * cluster), kThreads, 0, stream, cluster, p, cluster,
                            parts);
}

unsigned int read_and_clear_verify_index_error() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_verify_index_error, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_verify_index_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace fp8act
