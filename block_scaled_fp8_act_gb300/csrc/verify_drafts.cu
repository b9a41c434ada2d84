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
// Two launches. The first reads every row once for its maximum and sum (fp32,
// running rescale), rows cut into as many parts as fill the SMs a few times.
// The second, dependent, has a thread-block cluster per sequence: its CTAs
// join the parts and decide the acceptance alike, then share the vocabulary of
// the one row (or pair) drawn from, by then in L2, and meet through
// distributed shared memory for the draw. (One launch with a cluster of 16 per sequence for
// both took 20.5 us for 7 drafts at one sequence, where 16 SMs read 4.6 MB,
// and 53 us for 34 x 2 drafts.)
//
// Measured over 151936 bf16 logits: 27.2 us for 34 sequences of 2 drafts (72 MB read once, 2.7 TB/s; 10.7 us at the
// rate of a copy) and 11.3 us for one sequence of 7 (0.8). What bounds it: in the first kernel, about half of the time,
// neither issue (an exponential, a widening and a maximum per logit: 2.6 of 4 instructions a clock) nor memory (39 %) is
// full, but some SMs have 4 CTAs where others have 3; the second, and a single
// sequence, by the chain of dependent latencies: statistics, acceptance, the row drawn from, the cluster's meeting.
// (With fp32 logits the second spills 164 bytes a thread at 64 registers, which two CTAs per SM leave.)
// Widening and adding in pairs (packed maximum, fp32 pairs) took 0.8 us off the first.
// The second reads nothing before its own wait, which alone makes what earlier kernels wrote visible to it; so that its
// acceptance is still one trip to memory, the first notes the drafted token's logit in the record of a row's first part.
// (Inputs read while the first still ran took 0.7 to 1.1 us less, on the ground that their writers have ended; but
// only the wait orders what they wrote before a read here.)
#include <atomic>

#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {
namespace {

__device__ unsigned int g_verify_index_error;

constexpr int kStatThreads = 256;
constexpr int kStatWarps = kStatThreads / 32;
constexpr int kThreads = 512;  // of the second kernel
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = 2 * kMaxDrafts + 1;
static_assert(kMaxDrafts <= 32, "a lane per draft");
constexpr int kMaxParts = 32;
constexpr int kMaxCluster = 16;
constexpr float kNegInf = -__builtin_huge_valf();

// Maximum, sum of exponentials below it, and (for temperature 0) the first index of the maximum.
struct Stat {
    float m, s;
    int at;
};
// What the first kernel leaves of a part of a row; `drafted`: the row's logit at the token drafted there (in part 0).
struct __align__(16) Part {
    Stat st;
    float drafted;
};
static_assert(sizeof(Part) == 16, "one load");

__device__ __forceinline__ float clean(float v) { return fmaxf(v, kNegInf); }  // NaN counts as masked

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
    __device__ __forceinline__ uint4 raw(int i) const { return ld_dep_v4(base + static_cast<int64_t>(i) * kBytes); }
    // A vector to fp32, NaN as -inf, and its maximum.
    static __device__ __forceinline__ float widen_max(const uint4& v, float (&f)[kPer]) {
        if constexpr (kF32) {
            widen(v, f);
            return fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
        } else {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            const __nv_bfloat162 low = __bfloat162bfloat162(__ushort_as_bfloat16(0xFF80));  // -inf
            __nv_bfloat162 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]), low);
                const uint32_t u = *reinterpret_cast<const uint32_t*>(&x[j]);
                f[2 * j] = bf16_lo(u);
                f[2 * j + 1] = bf16_hi(u);
            }
            const __nv_bfloat162 top = __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3]));
            return fmaxf(__low2float(top), __high2float(top));
        }
    }
    static __device__ __forceinline__ void widen(const uint4& v, float (&f)[kPer]) {
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

// What both kernels know of a sequence.
template <bool kF32>
struct Sequence {
    const uint8_t* target;
    const uint8_t* draft;
    int64_t row_bytes;
    int V, targets, rows;
    float c;  // log2(e) / temperature
    bool greedy;
    __device__ __forceinline__ Sequence(const VerifyProblem& p, int b) : V(p.V), targets(p.k + 1) {
        rows = p.draft ? 2 * p.k + 1 : p.k + 1;
        row_bytes = static_cast<int64_t>(V) * Row<kF32>::kBytes;
        target = static_cast<const uint8_t*>(p.target) + static_cast<int64_t>(b) * targets * row_bytes;
        draft = p.draft ? static_cast<const uint8_t*>(p.draft) + static_cast<int64_t>(b) * p.k * row_bytes : nullptr;
    }
    __device__ __forceinline__ void read_temperature(const VerifyProblem& p, int b) {
        const float temp = ld_dep_f32(p.temperature + b);
        greedy = !(temp > 0.0f);
        // Kept a positive normal number, so that its products with differences of logits, -inf among them, are none of
        // them NaN: at an infinite temperature a masked logit stays masked, at a tiny one the largest keeps its 0.
        c = greedy ? 1.0f : fminf(fmaxf(1.4426950408889634f / temp, 0x1p-126f), 0x1p126f);
    }
    __device__ __forceinline__ Row<kF32> row(int r) const {
        return {r < targets ? target + r * row_bytes : draft + (r - targets) * row_bytes, V};
    }
};

// Maximum and sum of part x of row y of sequence z.
template <bool kF32>
__global__ void __launch_bounds__(kStatThreads) verify_stats_kernel(const VerifyProblem p, Part* parts) {
    using R = Row<kF32>;
    __shared__ Stat part[kStatWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sequence<kF32> q(p, blockIdx.z);
    const R row = q.row(blockIdx.y);
    const int share = blockIdx.x, shares = gridDim.x;
    const int head = row.head(), vecs = (p.V - head) / R::kPer, tail = head + vecs * R::kPer;
    const int v0 = static_cast<int>(static_cast<int64_t>(vecs) * share / shares);
    const int v1 = static_cast<int>(static_cast<int64_t>(vecs) * (share + 1) / shares);
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    q.read_temperature(p, blockIdx.z);
    Stat st = {kNegInf, 0.0f, 0x7FFFFFFF};
    auto one = [&](int i) {
        const Stat o = {row.at(i), 1.0f, i};
        if (o.m > kNegInf) join(st, o, q.c);
    };
    if (share == 0 && static_cast<int>(threadIdx.x) < head) one(threadIdx.x);
    // kAhead vectors are in flight while kAhead are used.
    constexpr int kAhead = 4;
    uint4 raw[kAhead];
    auto request = [&](int v, uint4 (&to)[kAhead]) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (v + kStatThreads * u < v1) to[u] = row.raw(head + (v + kStatThreads * u) * R::kPer);
    };
    const int first = v0 + static_cast<int>(threadIdx.x);
    float2 sum = make_float2(st.s, 0.0f);
    request(first, raw);
    float drafted = kNegInf;
    const int draft_row = static_cast<int>(blockIdx.y) - (static_cast<int>(blockIdx.y) < q.targets ? 0 : q.targets);
    if (share == 0 && threadIdx.x == 0 && draft_row < p.k) {
        const int x = ld_dep_s32(p.draft_tokens + static_cast<int64_t>(blockIdx.z) * p.k + draft_row);
        if (x >= 0 && x < p.V) drafted = row.at(x);
    }
    for (int v = first; v < v1; v += kStatThreads * kAhead) {
        uint4 next[kAhead];
        request(v + kStatThreads * kAhead, next);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (v + kStatThreads * u >= v1) break;
            float f[R::kPer];
            const float top = R::widen_max(raw[u], f);
            if (top > st.m) {
                const float f0 = st.m > kNegInf ? ex2((st.m - top) * q.c) : 0.0f;
                sum = __fmul2_rn(sum, make_float2(f0, f0));
                st.m = top;
                if (q.greedy) {
                    const int i = head + (v + kStatThreads * u) * R::kPer;
#pragma unroll
                    for (int j = R::kPer - 1; j >= 0; --j)
                        if (f[j] == top) st.at = i + j;
                }
            }
            // (the row's values are -inf or finite, and so is st.m, unless all so far were -inf)
            const float m = st.m > kNegInf ? -st.m : 0.0f;
            const float2 m2 = make_float2(m, m), c2 = make_float2(q.c, q.c);
#pragma unroll
            for (int j = 0; j < R::kPer; j += 2) {
                const float2 y = __fmul2_rn(__fadd2_rn(make_float2(f[j], f[j + 1]), m2), c2);
                sum = __fadd2_rn(sum, make_float2(ex2(y.x), ex2(y.y)));
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) raw[u] = next[u];
    }
    st.s = sum.x + sum.y;
    if (share == shares - 1 && tail + static_cast<int>(threadIdx.x) < p.V) one(tail + threadIdx.x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        Stat other;
        other.m = __shfl_xor_sync(0xffffffffu, st.m, o);
        other.s = __shfl_xor_sync(0xffffffffu, st.s, o);
        other.at = __shfl_xor_sync(0xffffffffu, st.at, o);
        join(st, other, q.c);
    }
    if (lane == 0) part[warp] = st;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kStatWarps; ++i) join(st, part[i], q.c);
        parts[(static_cast<int64_t>(blockIdx.z) * q.rows + blockIdx.y) * shares + share] = {st, drafted};
    }
}

struct VerifyShared {
    Stat row[kMaxRows];
    float drafted[kMaxRows];
    float prob[kMaxDrafts];
    int taken, n;
    Best warp_best[kWarps];
    Best best[2];  // this CTA's best draw (read by the cluster); one slot per pass
    Best all;
};

__device__ __forceinline__ Best ld_cluster_best(const Best* p, uint32_t rank) {
    const uint32_t at = ptx::mapa_shared(ptx::smem_u32(p), rank);
    Best r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r.key) : "r"(at) : "memory");
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(r.at) : "r"(at + 4) : "memory");
    return r;
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads, 2) verify_draw_kernel(const VerifyProblem p, const Part* parts, int cluster,
                                                               int shares) {
    using R = Row<kF32>;
    __shared__ VerifyShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / cluster;
    const int rank = static_cast<int>(blockIdx.x) % cluster;
    const int V = p.V, k = p.k;
    Sequence<kF32> q(p, b);
    const int targets = q.targets;
    const float* noise = p.noise + static_cast<int64_t>(b) * V;
    const int i0 = static_cast<int>(static_cast<int64_t>(V) * rank / cluster);
    const int i1 = static_cast<int>(static_cast<int64_t>(V) * (rank + 1) / cluster);
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    q.read_temperature(p, b);
    const float c = q.c;
    const bool greedy = q.greedy;
    const bool draft = p.draft != nullptr;
    auto row_of = [&](int r) { return q.row(r); };
    int n = p.n_draft ? ld_dep_s32(p.n_draft + b) : k;
    // Warp 0's lane j holds draft j and its number, requested together with the row statistics and looked at after them.
    int x = -1;
    float u = 1.0f;
    if (warp == 0 && lane < k) {
        x = ld_dep_s32(p.draft_tokens + static_cast<int64_t>(b) * k + lane);
        u = ld_dep_f32(p.uniform + static_cast<int64_t>(b) * k + lane);
    }
    for (int r = warp; r < q.rows; r += kWarps) {  // a warp per row, a lane per part
        const Part* from = parts + (static_cast<int64_t>(b) * q.rows + r) * shares + lane;
        Stat st = {kNegInf, 0.0f, 0x7FFFFFFF};
        float drafted = kNegInf;
        if (lane < shares) {
            const uint4 v = ld_dep_v4(from);
            st = {__uint_as_float(v.x), __uint_as_float(v.y), static_cast<int>(v.z)};
            drafted = __uint_as_float(v.w);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            Stat other;
            other.m = __shfl_xor_sync(0xffffffffu, st.m, o);
            other.s = __shfl_xor_sync(0xffffffffu, st.s, o);
            other.at = __shfl_xor_sync(0xffffffffu, st.at, o);
            join(st, other, c);
        }
        if (lane == 0) {
            sh.row[r] = st;
            sh.drafted[r] = drafted;
        }
    }
    if (threadIdx.x == 0) {
        if (n < 0 || n > k) atomicOr(&g_verify_index_error, 1u);
        sh.n = min(max(n, 0), k);
    }
    __syncthreads();

    // Acceptance, decided alike in every CTA.
    if (warp == 0) {
        const bool there = x >= 0 && x < V;
        n = sh.n;
        if (!there && lane < n && rank == 0) atomicOr(&g_verify_index_error, 1u);
        float prob = 0.0f;
        if (there && lane < n) {
            const Stat st = sh.row[lane];
            if (greedy) {
                prob = st.m > kNegInf && st.at == x ? 1.0f : 0.0f;
            } else {
                const float px = st.s > 0.0f ? __fdiv_rn(exp_below(sh.drafted[lane], st.m, c), st.s) : 0.0f;
                float qx = 1.0f;
                if (draft) {
                    const Stat sd = sh.row[targets + lane];
                    qx = sd.s > 0.0f ? __fdiv_rn(exp_below(sh.drafted[targets + lane], sd.m, c), sd.s) : 0.0f;
                }
                prob = qx > 0.0f ? fminf(__fdiv_rn(px, qx), 1.0f) : px > 0.0f ? 1.0f : 0.0f;
            }
        }
        if (lane < k) sh.prob[lane] = prob;
        const uint32_t no = ~__ballot_sync(0xffffffffu, lane < n && u < prob);
        if (lane == 0) sh.taken = no ? __ffs(no) - 1 : 32;
    }
    __syncthreads();
    const int taken = sh.taken;

    // Pass 2: the draw. `rest` draws from max(p - q, 0), else from p.
    const Stat st = sh.row[taken];
    int token = -1;
    bool rest = taken < sh.n && !greedy;
    if (greedy) {
        if (st.m > kNegInf) token = st.at;
    } else if (st.s > 0.0f) {
        const R row = row_of(taken);
        const int skip = rest && !draft ? ld_dep_s32(p.draft_tokens + static_cast<int64_t>(b) * k + taken) : -1;
        const float inv_p = __fdiv_rn(1.0f, st.s);
        for (int pass = 0; pass < 2; ++pass) {
            Best best = {0.0f, 0x7FFFFFFF};
            Stat sd = {0.0f, 1.0f, 0};
            float inv_q = 0.0f;
            if (rest && draft) {
                sd = sh.row[targets + taken];
                inv_q = sd.s > 0.0f ? __fdiv_rn(1.0f, sd.s) : 0.0f;
            }
            const R other = rest && draft ? row_of(targets + taken) : row;
            auto consider = [&](float t, float d, float e, int i) {
                float w = exp_below(t, st.m, c) * inv_p;
                if (rest) {
                    if (draft)
                        w -= exp_below(d, sd.m, c) * inv_q;
                    else if (i == skip)
                        w = 0.0f;
                }
                if (w > 0.0f) better(best, __fdividef(w, e), i);
            };
            // Logit rows start on 16-byte boundaries if V is a multiple of 8; the caller's noise may start on any 4-byte one.
            if (V % 8 == 0 && (reinterpret_cast<uintptr_t>(noise) & 15) == 0) {
                const int n8 = V / 8;
                const int v0 = static_cast<int>(static_cast<int64_t>(n8) * rank / cluster);
                const int v1 = static_cast<int>(static_cast<int64_t>(n8) * (rank + 1) / cluster);
                struct Loaded {
                    uint4 n[2], t[8 / R::kPer], d[8 / R::kPer];
                };
                auto request = [&](int v, Loaded& to) {
                    if (v >= v1) return;
                    to.n[0] = ld_dep_v4(noise + v * 8);
                    to.n[1] = ld_dep_v4(noise + v * 8 + 4);
#pragma unroll
                    for (int u = 0; u < 8 / R::kPer; ++u) {
                        to.t[u] = row.raw(v * 8 + u * R::kPer);
                        to.d[u] = other.raw(v * 8 + u * R::kPer);
                    }
                };
                Loaded now, next;
                request(v0 + static_cast<int>(threadIdx.x), now);
                for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += kThreads) {
                    request(v + kThreads, next);
                    const float e[8] = {__uint_as_float(now.n[0].x), __uint_as_float(now.n[0].y), __uint_as_float(now.n[0].z),
                                        __uint_as_float(now.n[0].w), __uint_as_float(now.n[1].x), __uint_as_float(now.n[1].y),
                                        __uint_as_float(now.n[1].z), __uint_as_float(now.n[1].w)};
#pragma unroll
                    for (int u = 0; u < 8 / R::kPer; ++u) {
                        float ft[R::kPer], fd[R::kPer];
                        R::widen(now.t[u], ft);
                        R::widen(now.d[u], fd);
#pragma unroll
                        for (int j = 0; j < R::kPer; ++j) consider(ft[j], fd[j], e[u * R::kPer + j], v * 8 + u * R::kPer + j);
                    }
                    now = next;
                }
            } else {
                constexpr int kAhead = 4;
                for (int i = i0 + static_cast<int>(threadIdx.x); i < i1; i += kAhead * kThreads) {
                    float t[kAhead], d[kAhead], e[kAhead];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const int x = i + u * kThreads < i1 ? i + u * kThreads : i;
                        t[u] = row.at(x);
                        d[u] = other.at(x);
                        e[u] = ld_dep_f32(noise + x);
                    }
#pragma unroll
                    for (int u = 0; u < kAhead; ++u)
                        if (i + u * kThreads < i1) consider(t[u], d[u], e[u], i + u * kThreads);
                }
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) {
                const float key = __shfl_xor_sync(0xffffffffu, best.key, o);
                const int at = __shfl_xor_sync(0xffffffffu, best.at, o);
                better(best, key, at);
            }
            if (lane == 0) sh.warp_best[warp] = best;
            __syncthreads();
            auto reduce = [&](int width) {
                for (int o = width / 2; o >= 1; o >>= 1) {
                    const float key = __shfl_xor_sync(0xffffffffu, best.key, o);
                    const int at = __shfl_xor_sync(0xffffffffu, best.at, o);
                    better(best, key, at);
                }
            };
            if (warp == 0) {
                best = sh.warp_best[lane % kWarps];
                reduce(kWarps);
                if (lane == 0) sh.best[pass] = best;
            }
            ptx::cluster_sync();
            if (warp == 0) {
                best = ld_cluster_best(&sh.best[pass], lane % cluster);
                reduce(cluster);
                if (lane == 0) sh.all = best;
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

size_t verify_drafts_workspace(int B, int k) {
    return static_cast<size_t>(B < 1 ? 1 : B) * (2 * k + 1) * kMaxParts * sizeof(Part);
}

cudaError_t launch_verify_drafts(const VerifyProblem& p, int num_sms, cudaStream_t stream) {
    const int rows = p.draft ? 2 * p.k + 1 : p.k + 1;
    // Parts of a row: as many as run at once with 4 CTAs of the first kernel per SM, of 2048 logits at least. (Rounded
    // up, which leaves a second wave, 34 x 2 drafts over 151936 logits took 27.5 us instead of 26.8 and fp32 ones over
    // 248320 58.4 instead of 51.5; parts for 5 or 6 CTAs per SM are within 3 % either way.)
    int shares = static_cast<int>(4 * static_cast<int64_t>(num_sms) / (static_cast<int64_t>(p.B) * rows));
    if (shares < 1) shares = 1;
    if (shares > kMaxParts) shares = kMaxParts;
    while (shares > 1 && p.V < 2048 * shares) --shares;
    // CTAs of a sequence in the second: as many as stay within two per SM, of 2048 logits at least.
    int cluster = kMaxCluster;
    while (cluster > 1 && (p.V < 2048 * cluster || static_cast<int64_t>(p.B) * cluster > 2 * num_sms)) cluster /= 2;
    Part* parts = static_cast<Part*>(p.workspace);
    auto draw = p.f32 ? verify_draw_kernel<true> : verify_draw_kernel<false>;
    static std::atomic<bool> configured[2][64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (!configured[p.f32][dev & 63].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(draw, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        configured[p.f32][dev & 63].store(true, std::memory_order_relaxed);
    }
    const cudaError_t e = launch_dependent(p.f32 ? verify_stats_kernel<true> : verify_stats_kernel<false>, dim3(shares, rows, p.B),
                         kStatThreads, 0, stream, 1, p, parts);
    if (e != cudaSuccess) return e;
    return launch_dependent(draw, dim3(static_cast<unsigned>(p.B) * cluster), kThreads, 0, stream, cluster, p, parts,
                            cluster, shares);
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
