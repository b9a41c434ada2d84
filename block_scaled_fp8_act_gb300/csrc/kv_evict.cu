// Eviction from the paged cache: per sequence and KV head the `keep` tokens of
// the largest accumulated weight, in their order, copied into other pages.
//
// Select. A weight's bits become a whole number of the same order, the kept
// class above it: the last `recent` and the first `first` tokens are the largest
// number, NaN counts as -infinity. The keep-th largest number T is found 11, 10
// and 11 bits at a time from counts in shared memory, then the tokens above T
// and the first of those equal to it are listed by a running count; a thread has
// 16 in a row as bits of a word and goes through those that stay. A (sequence,
// head) has a cluster of up to 8 CTAs, each with a run of tokens whose numbers
// stay in shared memory: the weights are read once. The CTAs join their counts
// through distributed shared memory, so nothing goes through global memory but
// the list: in the first and the last round, where few bins hold something, each
// adds its own to every other's (0.8 us; reading all bins of all CTAs 2.4), in the
// second, where most of them do, they read each other's. How many tokens of a CTA
// lie above T and at it is known from its own counts.
//
// What bounds it: the trips of a selection. 131072 tokens x 4 heads to 8192, 19.9
// us with a copy of 4: start 2.5, weights and first counts 3, the three exchanges
// 2, 2.2 and 1.4, sums of the bins 1.6, the other rounds' counts 2.1, the list 1.7
// (3.4 with a test and a store for each token). Clusters of 16 CTAs took 2 us more.
//
// Copy. A CTA takes 64 places of the list: one thread each looks up where a
// token is and where it goes, then the codes move 16 bytes a thread, all of a
// thread's loads before its stores. 34 sequences up to 16384 -> 4096: 34.9 us with
// the selection, 5.1 TB/s.
#include <atomic>
#include <type_traits>

#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {
namespace {

__device__ unsigned int g_evict_index_error;

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kMostKeys = 36864;  // that a CTA holds in shared memory; more are read again
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint2 ld_shared_cluster_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

// What a sequence comes to: its cached tokens, how many stay, and how many of those by their place.
struct Budget {
    int len, count, recent, first;
};
__device__ __forceinline__ Budget budget_of(const EvictProblem& p, int b, bool report) {
    const int64_t most = p.table_stride << p.cache.page_log2, room = p.new_stride << p.cache.page_log2;
    const int len = ld_dep_s32(p.kv_lens + b), keep = ld_dep_s32(p.keep + b);
    if (report && (len < 0 || len > most || keep < 0 || keep > room)) atomicOr(&g_evict_index_error, 1u);
    Budget g;
    g.len = len < 0 ? 0 : static_cast<int>(len > most ? most : len);
    const int k = keep < 0 ? 0 : static_cast<int>(keep > room ? room : keep);
    g.count = min(g.len, k);
    g.recent = min(p.recent, g.count);
    g.first = min(p.first, g.count - g.recent);
    return g;
}

__device__ __forceinline__ void red_shared_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// The order of weights as that of whole numbers; NaN as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t ordered(float w) {
    uint32_t u = __float_as_uint(w);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) u = 0xFF800000u;
    if (u == 0x80000000u) u = 0;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sums over the CTA's threads, and the sum of all.
__device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t (&warps)[33], uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    __syncthreads();  // (the sums of a scan before have been read)
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const uint32_t w = warps[lane];
        uint32_t s = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        warps[lane] = s - w;
        if (lane == 31) warps[32] = s;
    }
    __syncthreads();
    total = warps[32];
    return warps[warp] + incl - v;
}

__global__ void __launch_bounds__(kThreads) kv_evict_select_kernel(const __grid_constant__ EvictProblem p, int ctas, uint32_t held) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ __align__(8) uint32_t hist[3][kBins];  // this CTA's counts of a round
    __shared__ __align__(8) uint32_t all[3][kBins];   // the cluster's (only there with more CTAs than one)
    __shared__ uint32_t warps[33], found[2];
    __shared__ __align__(8) uint2 mine;  // tokens above the threshold and equal to it
    const int item = blockIdx.x / ctas, rank = blockIdx.x - item * ctas;
    const int b = item / p.cache.heads, h = item - b * p.cache.heads;
    for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&hist[0][0])[i] = (&all[0][0])[i] = 0;
    if (threadIdx.x == 0) mine = make_uint2(0, 0);
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const Budget g = budget_of(p, b, h == 0 && rank == 0 && threadIdx.x == 0);
    const int64_t room = p.new_stride << p.cache.page_log2;
    int* const kept = p.kept + item * room;
    if (h == 0 && rank == 0 && threadIdx.x == 0) p.new_lens[b] = g.count;
    const int64_t me = static_cast<int64_t>(rank) * kThreads + threadIdx.x, threads = static_cast<int64_t>(ctas) * kThreads;
    for (int64_t i = g.count + me; i < room; i += threads) kept[i] = -1;
    if (g.count == g.len || g.count == 0) {  // (the whole cluster)
        for (int64_t i = me; i < g.count; i += threads) kept[i] = static_cast<int>(i);
        return;
    }
    // (the other CTAs' counts are zero before any is added to; waited for after the weights have been asked for)
    if (ctas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    // This CTA's tokens: [begin, end), begin a multiple of 4.
    const int64_t run = ((static_cast<int64_t>(g.len) + ctas - 1) / ctas + 3) & ~int64_t{3};
    const int64_t begin64 = rank * run;
    const int begin = static_cast<int>(begin64 < g.len ? begin64 : g.len);
    // (unsigned, so that a step past the longest run does not wrap)
    const uint32_t n = static_cast<uint32_t>(begin64 + run < g.len ? run : g.len - begin);
    const int* table = p.page_table + static_cast<int64_t>(b) * p.table_stride;
    auto read = [&](uint32_t i) -> uint4 {  // the numbers of tokens begin + i .. + 3; 0, below every weight's, past the last
        const int pos = begin + static_cast<int>(i), page = ld_dep_s32(table + (pos >> p.cache.page_log2));
        uint4 w = make_uint4(0x7FFFFFFFu, 0x7FFFFFFFu, 0x7FFFFFFFu, 0x7FFFFFFFu);
        if (page >= 0 && page < p.cache.num_pages)
            w = ld_dep_v4(p.mass + ((static_cast<int64_t>(page) * p.cache.heads + h) << p.cache.page_log2) +
                          (pos & ((1 << p.cache.page_log2) - 1)));
        else
            atomicOr(&g_evict_index_error, 1u);
        uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = ordered(__uint_as_float(u[j]));
        if (pos + 4 > g.len - g.recent || pos < g.first) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (pos + j >= g.len - g.recent || pos + j < g.first) u[j] = pos + j < g.len ? 0xFFFFFFFFu : 0;
        }
        if (i + 4 > n) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j >= n) u[j] = 0;
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    };
    // Where four tokens' numbers are held: in an order in which both those of neighbouring threads and every fourth of them
    // (a thread's of 16 in a row) lie in different banks.
    auto at_keys = [&](uint32_t i) { return reinterpret_cast<uint4*>(keys) + (i >> 2 ^ (i >> 4 & 7)); };
    auto again = [&](uint32_t i) { return i < held ? *at_keys(i) : read(i); };
    auto each = [&](const uint4& k, auto f) {
        f(k.x);
        f(k.y);
        f(k.z);
        f(k.w);
    };
    __syncthreads();

    uint32_t want = g.count, prefix = 0;  // the want-th largest of those whose upper bits are `prefix`
    uint32_t above_here = 0, equal_here = 0;  // this CTA's tokens above those and among them, in this thread's bins
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 11 : 0, top = pass == 0 ? 32 : pass == 1 ? 21 : 11;
        const uint32_t mask = pass == 1 ? 1023u : 2047u;
        uint32_t* const count = hist[pass];
        if (pass == 0) {
#pragma unroll 4
            for (uint32_t i = threadIdx.x * 4; i < n; i += kThreads * 4) {
                const uint4 k = read(i);
                if (i < held) *at_keys(i) = k;
                each(k, [&](uint32_t u) { atomicAdd(count + (u >> 21), 1u); });
            }
        } else {
            const uint32_t least = prefix << top, span = 1u << top;
            for (uint32_t i = threadIdx.x * 4; i < n; i += kThreads * 4) {
                const uint4 k = again(i);
                // (in the last round most warps have none)
                if (min(min(k.x - least, k.y - least), min(k.z - least, k.w - least)) < span)
                    each(k, [&](uint32_t u) {
                        if (u - least < span) atomicAdd(count + (u >> shift & mask), 1u);
                    });
            }
        }
        __syncthreads();
        // Counts from the largest bin down, two a thread.
        const int bin = kBins - 2 - 2 * static_cast<int>(threadIdx.x);
        const uint32_t own_lo = count[bin], own_hi = count[bin + 1];
        uint32_t lo = own_lo, hi = own_hi;
        if (ctas > 1) {
            if (pass == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            if (pass != 1) {
                const uint32_t at = ptx::smem_u32(all[pass] + bin);
                for (int r = 0; r < ctas; ++r) {
                    const uint32_t to = ptx::mapa_shared(at, r);
                    if (lo) red_shared_cluster_u32(to, lo);
                    if (hi) red_shared_cluster_u32(to + 4, hi);
                }
                ptx::cluster_sync();
                lo = all[pass][bin];
                hi = all[pass][bin + 1];
            } else {
                ptx::cluster_sync();
                const uint32_t at = ptx::smem_u32(count + bin);
                uint2 v[kMaxCluster];
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r)
                    v[r] = r < ctas && bin < 1024 ? ld_shared_cluster_v2(ptx::mapa_shared(at, r)) : make_uint2(0, 0);
                lo = hi = 0;
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) {
                    lo += v[r].x;
                    hi += v[r].y;
                }
            }
        }
        uint32_t total;
        const uint32_t above = scan(lo + hi, warps, total);
        if (above < want && want <= above + lo + hi) {
            const bool upper = want <= above + hi;
            found[0] = bin + (upper ? 1 : 0);
            found[1] = want - above - (upper ? 0 : hi);
        }
        __syncthreads();
        const int at = static_cast<int>(found[0]);
        above_here += (bin > at ? own_lo : 0) + (bin + 1 > at ? own_hi : 0);
        equal_here = bin == at ? own_lo : bin + 1 == at ? own_hi : 0;
        prefix = prefix << (pass == 1 ? 10 : 11) | found[0];
        want = found[1];
    }
    const uint32_t threshold = prefix;  // `want` of those equal to it stay

    // Tokens above the threshold and equal to it in the CTAs before this one.
    uint32_t base_above = 0, base_equal = 0;
    if (ctas > 1) {
        const uint32_t above = __reduce_add_sync(0xffffffffu, above_here), equal = __reduce_add_sync(0xffffffffu, equal_here);
        if ((threadIdx.x & 31) == 0) {
            atomicAdd(&mine.x, above);
            atomicAdd(&mine.y, equal);
        }
        ptx::cluster_sync();
        const uint32_t at = ptx::smem_u32(&mine);
        for (int r = 0; r < rank; ++r) {
            const uint2 v = ld_shared_cluster_v2(ptx::mapa_shared(at, r));
            base_above += v.x;
            base_equal += v.y;
        }
    }
    // Every thread lists kRun tokens in a row at a time (counts of a round fit 16 bits), 4 where that is enough.
    auto list = [&](auto run) {
        constexpr int kRun = decltype(run)::value;
        for (uint32_t i0 = 0; i0 < n; i0 += kThreads * kRun) {
            const uint32_t i = i0 + threadIdx.x * kRun;
            uint32_t above = 0, equal = 0;  // a bit a token
#pragma unroll
            for (int j = 0; j < kRun / 4; ++j) {
                const uint4 k = i + 4 * j < n ? again(i + 4 * j) : make_uint4(0, 0, 0, 0);
                uint32_t bit = 1u << 4 * j;
                each(k, [&](uint32_t u) {
                    above |= u > threshold ? bit : 0;
                    equal |= u == threshold ? bit : 0;
                    bit <<= 1;
                });
            }
            uint32_t total;
            const uint32_t before = scan(__popc(above) | __popc(equal) << 16, warps, total);
            const uint32_t equals = base_equal + (before >> 16);  // in front of this thread's
            uint32_t stay = above;
            for (uint32_t left = equals < want ? want - equals : 0; equal && left; --left, equal &= equal - 1) stay |= equal & -equal;
            int* to = kept + base_above + (before & 0xFFFFu) + min(equals, want);
            for (; stay; stay &= stay - 1) *to++ = begin + static_cast<int>(i) + __ffs(stay) - 1;
            base_above += total & 0xFFFFu;
            base_equal += total >> 16;
        }
    };
    if (n <= 4 * kThreads)
        list(std::integral_constant<int, 4>{});
    else
        list(std::integral_constant<int, 16>{});
    if (ctas > 1) ptx::cluster_sync();  // no CTA leaves while another reads its counts
}

constexpr int kCopyTokens = 64, kCopyThreads = 256;

template <int kD>
__global__ void __launch_bounds__(kCopyThreads) kv_evict_copy_kernel(const __grid_constant__ EvictProblem p, int chunks) {
    __shared__ int64_t from[kCopyTokens], to[kCopyTokens];
    const int64_t item = blockIdx.x / static_cast<unsigned>(chunks);
    const int chunk = blockIdx.x % static_cast<unsigned>(chunks);
    const int b = static_cast<int>(item / p.cache.heads), h = static_cast<int>(item % p.cache.heads);
    const KvCache& c = p.cache;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t at = static_cast<int64_t>(chunk) * kCopyTokens;
    const Budget g = budget_of(p, b, false);
    if (at >= g.count) return;
    const int n = static_cast<int>(min(static_cast<int64_t>(kCopyTokens), g.count - at));
    if (threadIdx.x < kCopyTokens) {
        int64_t src = -1, dst = -1;
        if (static_cast<int>(threadIdx.x) < n) {
            const int in_page = (1 << c.page_log2) - 1, i = static_cast<int>(at) + threadIdx.x;
            const int pos = ld_dep_s32(p.kept + ((item * p.new_stride) << c.page_log2) + i);
            const int a = ld_dep_s32(p.page_table + b * p.table_stride + (pos >> c.page_log2));
            const int z = ld_dep_s32(p.new_table + b * p.new_stride + (i >> c.page_log2));
            if (a >= 0 && a < c.num_pages && z >= 0 && z < c.num_pages) {
                src = ((static_cast<int64_t>(a) * c.heads + h) << c.page_log2) + (pos & in_page);
                dst = ((static_cast<int64_t>(z) * c.heads + h) << c.page_log2) + (i & in_page);
            } else {
                atomicOr(&g_evict_index_error, 1u);
            }
        }
        from[threadIdx.x] = src;
        to[threadIdx.x] = dst;
    }
    __syncthreads();
    constexpr int kC = kD / 16, kSteps = kCopyTokens * kC / kCopyThreads;  // 16-byte chunks of a vector; a thread's
    const int col = threadIdx.x % kC, row = threadIdx.x / kC;
    const uint4 *k = reinterpret_cast<const uint4*>(c.k) + col, *v = reinterpret_cast<const uint4*>(c.v) + col;
    uint4 x[kSteps], y[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int64_t src = from[row + i * (kCopyThreads / kC)];
        if (src >= 0) {
            x[i] = ld_dep_stream_v4(k + src * kC);
            y[i] = ld_dep_stream_v4(v + src * kC);
        }
    }
    float s0 = 0.0f;
    const int which = threadIdx.x / kCopyTokens;  // key scales, value scales, weights
    float* const words = which == 0 ? c.k_scale : which == 1 ? c.v_scale : p.mass;
    const int64_t src = from[threadIdx.x % kCopyTokens], dst = to[threadIdx.x % kCopyTokens];
    if (which < 3 && src >= 0) s0 = ld_dep_f32(words + src);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int64_t z = to[row + i * (kCopyThreads / kC)];
        if (z >= 0) {
            reinterpret_cast<uint4*>(c.k)[z * kC + col] = x[i];
            reinterpret_cast<uint4*>(c.v)[z * kC + col] = y[i];
        }
    }
    if (which < 3 && dst >= 0) words[dst] = s0;
}

}  // namespace

cudaError_t launch_kv_evict(const EvictProblem& p, int num_sms, cudaStream_t stream) {
    const int items = p.batch * p.cache.heads;
    const int64_t most = p.table_stride << p.cache.page_log2;
    // A cluster while the SMs are not full and a CTA has work for every thread. (us, with clusters and without, 4 heads of one
    // sequence: 131072 tokens 25.4 and 99.2, 32768 15.9 and 21.6, 16384 13.0 and 14.0, 12000 12.6 and 12.4, 6000 11.7 and 10.3: the
    // exchanges pay from about 12000 tokens on.)
    int ctas = 1;
    while (ctas < kMaxCluster && 2 * ctas * static_cast<int64_t>(items) <= num_sms && most > ctas * int64_t{4 * kThreads}) ctas *= 2;
    const int64_t run = ((most + ctas - 1) / ctas + 3) & ~int64_t{3};
    const uint32_t held = static_cast<uint32_t>(run < kMostKeys ? (run + 31) / 32 * 32 : kMostKeys);  // (whole sets of banks)
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (!configured[dev & 63].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(kv_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * 4);
        if (e != cudaSuccess) return e;
        configured[dev & 63].store(true, std::memory_order_relaxed);
    }
    cudaError_t e = launch_dependent(kv_evict_select_kernel, dim3(items * ctas), kThreads, held * 4, stream, ctas, p, ctas, held);
    if (e != cudaSuccess) return e;
    const int64_t chunks = ((p.new_stride << p.cache.page_log2) + kCopyTokens - 1) / kCopyTokens;
    if (chunks == 0) return cudaSuccess;
    auto copy = p.cache.head_dim == 64 ? kv_evict_copy_kernel<64> : p.cache.head_dim == 128 ? kv_evict_copy_kernel<128> : kv_evict_copy_kernel<256>;
    return launch_dependent(copy, dim3(static_cast<unsigned>(items * chunks)), kCopyThreads, 0, stream, 1, p, static_cast<int>(chunks));
}

unsigned int read_and_clear_evict_index_error() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_evict_index_error, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_evict_index_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace fp8act
