// The weights of cached tokens (kv_mass.cu) for many rows at head size 128, on
// the 5th-generation tensor cores.
//
// S^T = K Q^T with the cached codes as they are: a tile of 128 tokens is the
// MMA's rows, all query rows (up to 256 at a time, as two E4M3 parts each) its
// columns. A token is then a lane of tensor memory and belongs to one thread,
// which goes along its columns: exp(s * k_scale * qs - lse), with qs and lse
// read two rows at a time by all lanes alike, into one running sum. Nothing is
// exchanged between threads, and the codes go from memory to the tensor cores
// untouched.
//
// Two accumulators take turns, each with a warpgroup: the tensor cores fill one
// while the other is read. A token's key scale, its place and the weight that it
// had are fetched a tile ahead by the thread that needs them.
//
// What bounds it: the chain of a tile's sums, 3600 clocks for 128 tokens x 192
// rows, two in flight beside 840 of MMAs: 131072 tokens x 4 heads, 32 new tokens
// of 6 heads, 48.8 us (528
// TFLOP/s, a score counted once; without exponentials 41.6, without the rows'
// values from shared memory 41.8). Measured and slower: two warpgroups an
// accumulator 49.7, four accumulators of 128 rows 51.6, the rows' values in three
// quarters of the bytes (a power of two as bf16 beside the log-sum-exp) 51.8 for
// the instructions that widen them, 8 columns at a time with 16 in flight 55.2.
// A cap takes it to 87.2 us, a bias by distance to 119: with either the kernel
// spills, 628 bytes of stores and 732 of loads a thread at 168 registers (56 and 40
// without), since 32 scores, the next 32 and the rows' values are live across the
// cap, and a bias reads a row's slope and place for every score beside them. In a
// window of 4096 of the 131072: 12.1 us, capped 14.1.
//
// Every wait is bounded as in kv_attention_tc.cu.
#include <atomic>

#include "host_util.h"
#include "kv_attention.cuh"
#include "tc_ptx.cuh"

namespace fp8act {

__device__ unsigned int g_mass_timeout;

namespace {

constexpr int kTok = 128;
constexpr int kD = 128;
constexpr int kRows = 256;      // rows at a time
constexpr int kThreads = 384;   // warps 0 keys, 1 MMA; 4..7 and 8..11 sums
constexpr int kStages = 6;      // key tiles in flight
constexpr int kTileBytes = kTok * kD;
constexpr int kItemCost = 4;    // units that an item counts beside its own, for its queries
using Work = Units<kTok, kItemCost, List::kMass>;

constexpr int kQ = 0;  // high parts, low parts
constexpr int kK = kQ + 2 * kRows * kD;
constexpr int kRowScores = kK + kStages * kTileBytes;
constexpr int kPairs = kRowScores + kRows * 16;           // of two rows: qs, qs, -lse, -lse (log2)
constexpr int kBytes = kPairs + kRows * 8 + 1024;         // (the base is rounded up to 1024)

struct Extra {
    unsigned long long wait_ns;  // bound of every wait
    int withhold;                // test hook: the CTA's first key tile is never requested
};

template <bool kChanged>
__global__ void __launch_bounds__(kThreads, 1) kv_mass_tc_kernel(const __grid_constant__ AttnArgs a,
                                                                 const __grid_constant__ CUtensorMap k_map, const Extra x) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - ptx::smem_u32(smem_raw));
    __shared__ Work::Scratch scratch;
    __shared__ __align__(8) uint64_t bars[2 * kStages + 2 * 2 + 4];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const uint32_t k_full = ptx::smem_u32(bars), k_empty = k_full + 8 * kStages;
    const uint32_t s_full = k_empty + 8 * kStages, s_empty = s_full + 16;  // [accumulator]
    const uint32_t q_full = s_empty + 16, rows_done = q_full + 8, mma_done = rows_done + 8, drain = mma_done + 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(k_full + 8 * i, 1);
            ptx::mbar_init(k_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(s_full + 8 * i, 1);
            ptx::mbar_init(s_empty + 8 * i, 4);
        }
        ptx::mbar_init(q_full, 8);
        ptx::mbar_init(rows_done, 8);
        ptx::mbar_init(mma_done, 1);
        ptx::mbar_init(drain, 1);
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 2) {
        tc::tmem_alloc(ptx::smem_u32(&s_tmem), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;

    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    Item it;
    int64_t per, u, u_end;
    const bool any = Work::first_item(a, 2, scratch, it, per, u, u_end);

    // A bounded wait by the whole warp; false once any wait of the CTA has run out.
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        // (the timer is far from the SM and is read only after a while)
        bool ok = ptx::mbar_try_wait(bar, parity);
        uint64_t start = 0;
        for (uint32_t n = 1; !ok; ++n) {
            ok = ptx::mbar_try_wait(bar, parity);
            if (!ok && n % 64 == 0) {
                const uint64_t now = ptx::globaltimer_ns();
                if (start == 0) start = now;
                if (s_abort || now - start > x.wait_ns) break;
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(&g_mass_timeout, 1u);
        }
        return ok;
    };

    // What every role knows of a job: some rows of an item and this CTA's tiles, [t0, t1) of the item's list. The rows see
    // the a_n ones from t0 on (the prefix's, where the list leaves out none) and the n - a_n ones from b0 on, which is
    // counted in the sequence.
    struct Job {
        int row0, nrows, columns;
        int t0, t1, a_n, b0, n;
        int lo, limit;   // no row needs a mask in [lo, limit), but for the prefix
        int from;        // no row sees anything before it, but for the prefix
        __device__ int tile(int i) const { return i < a_n ? t0 + i : b0 + i - a_n; }
    };
    int row0 = 0;
    auto job_of = [&]() {
        Job j;
        const int64_t item_end = it.first + it.tiles;
        const int rows_total = it.nq * a.group, weight = mass_weight(rows_total);
        auto tile_of = [&](int64_t unit) {
            return static_cast<int>((max(unit - it.first - kItemCost, int64_t{0}) + weight - 1) / weight);
        };
        j.t0 = tile_of(u);
        j.t1 = tile_of(item_end < u_end ? item_end : u_end);
        j.row0 = row0;
        j.nrows = min(rows_total - row0, kRows);
        j.columns = (j.nrows + 31) / 32 * 32;
        j.a_n = j.n = j.b0 = j.lo = j.limit = j.from = 0;
        if (j.nrows > 0) {
            const TileReach r = tile_reach<kTok>(a, it, row0, j.nrows);
            j.lo = r.lo;
            j.limit = r.limit;
            j.from = first_seen(a.scores, it.q0, it.len, it.nq, row0 / a.group);
            const int prefix = r.tiles.prefix_tiles;
            j.a_n = max(min(j.t1, prefix) - j.t0, 0);
            j.b0 = max(max(j.t0, prefix) + it.skip, prefix + r.tiles.skip);
            j.n = j.a_n + max(min(j.t1 + it.skip, r.tiles.end + r.tiles.skip) - j.b0, 0);
        }
        return j;
    };
    uint32_t seq = 0;  // tiles of the jobs before
    auto next = [&](const Job& j) -> bool {
        seq += j.n;
        row0 += kRows;
        if (row0 < it.nq * a.group) return true;
        row0 = 0;
        u = it.first + it.tiles;
        if (u >= u_end) return false;
        Work::next_item(a, it);
        return true;
    };
    const int* table = nullptr;
    // The page of a position of the item as the table has it (0 past its end), and whether there is one. Apart, so that a
    // page is not waited for where it is asked for.
    auto page_of = [&](int pos) { return pos < it.len ? ld_dep_s32(table + (pos >> a.c.page_log2)) : 0; };
    auto is_page = [&](int pos, int page) {
        if (pos >= it.len) return false;
        const bool ok = page >= 0 && page < a.c.num_pages;
        if (!ok) atomicOr(a.index_error, 1u);
        return ok;
    };
    auto place_of = [&](int page, int pos) {
        return ((static_cast<int64_t>(page) * a.c.heads + it.h) << a.c.page_log2) + (pos & ((1 << a.c.page_log2) - 1));
    };

    if (!any) {
        // nothing to do: only tensor memory to free
    } else if (warp == 0) {
        // ------------------------------------------------------------ copies
        const int box = min(1 << a.c.page_log2, kTok);
        bool ok = true;
        uint32_t n = 0;  // tiles requested
        while (ok) {
            const Job j = job_of();
            table = a.table + it.b * a.table_stride;
            // Lane i < 128 / box: copy i of the tile, if it holds a token; its page is looked up a tile ahead.
            auto look_up = [&](int i) { return i < j.n && lane < kTok / box ? page_of(j.tile(i) * kTok + lane * box) : 0; };
            int ahead = look_up(0);
            for (int i = 0; i < j.n; ++i, ++n) {
                const int page = ahead;
                ahead = look_up(i + 1);
                const uint32_t round = n / kStages, stage = n - round * kStages, bar = k_full + 8 * stage;
                if (round > 0 && !(ok = wait(k_empty + 8 * stage, (round - 1) & 1))) break;
                const int pos = j.tile(i) * kTok + lane * box;
                const bool copy = lane < kTok / box && (pos < it.prefix || pos + box > j.from) && is_page(pos, page);
                const uint32_t copies = __ballot_sync(0xffffffffu, copy);
                const bool withheld = x.withhold && n == 0;
                if (lane == 0 && !withheld) ptx::mbar_arrive_expect_tx(bar, __popc(copies) * box * kD);
                __syncwarp();
                if (copy && !withheld)
                    load_tokens(base + kK + stage * kTileBytes + lane * box * kD, &k_map, bar, static_cast<int>(place_of(page, pos)));
            }
            if (!ok || !next(j)) break;
        }
        // Every copy must have landed before the CTA leaves (its consumer has usually seen it).
        for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i)
            if (!(x.withhold && i == 0) && !ptx::mbar_wait(k_full + 8 * (i % kStages), (i / kStages) & 1) && lane == 0)
                atomicOr(&g_mass_timeout, 2u);
    } else if (warp == 1) {
        // --------------------------------------------------------------- MMA
        bool ok = true;
        uint32_t jobs = 0;
        while (ok) {
            const Job j = job_of();
            if (!(ok = wait(q_full, jobs & 1))) break;
            tc::fence_after_sync();
            const uint32_t idesc = tc::idesc_e4m3_f32(kTok, j.columns);
            for (int i = 0; i < j.n; ++i) {
                const uint32_t n = seq + i, stage = n % kStages, acc = n & 1;
                if (!(ok = wait(k_full + 8 * stage, (n / kStages) & 1))) break;
                if (n >= 2 && !(ok = wait(s_empty + 8 * acc, ((n >> 1) - 1) & 1))) break;
                tc::fence_after_sync();
                const uint64_t k_desc = tc::desc_kmajor_sw128(base + kK + stage * kTileBytes);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const uint64_t q_desc = tc::desc_kmajor_sw128(base + kQ + part * kRows * kD);
#pragma unroll
                    for (int k = 0; k < kD / 32; ++k)  // (a descriptor counts 16 bytes)
                        tc::mma_e4m3_ss(tmem + acc * 256, k_desc + 2 * k, q_desc + 2 * k, idesc, part + k > 0 ? 1u : 0u);
                }
                tc::commit_elected(s_full + 8 * acc);
                tc::commit_elected(k_empty + 8 * stage);
            }
            if (!ok) break;
            tc::commit_elected(mma_done);
            ++jobs;
            if (!next(j)) break;
        }
        // No MMA may still run when tensor memory is freed or the CTA leaves.
        tc::commit_elected(drain);
        if (!ptx::mbar_wait(drain, 0)) atomicOr(&g_mass_timeout, 4u);
        __syncwarp();
    } else if (warp >= 4) {
        // -------------------------------------------------------------- sums
        const int acc = (warp - 4) >> 2, quad = warp & 3;
        const uint32_t t_s = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * 256;
        const int mine = quad * 32 + lane;  // this thread's token of a tile
        RowScore* const row_scores = reinterpret_cast<RowScore*>(smem + kRowScores);
        float* const pairs = reinterpret_cast<float*>(smem + kPairs);
        uint32_t jobs = 0;
        bool ok = true;
        while (ok) {
            const Job j = job_of();
            table = a.table + it.b * a.table_stride;
            const int kept_end = old_end(a, it.b, it.len, it.nq);
            // The place of this thread's token of tile t, what it has so far and its key scale. There is none for a token that no
            // row sees and that keeps its weight, whose page may be another sequence's by now.
            const int touched_from = j.row0 > 0 ? j.from : j.nrows > 0 ? min(j.from, kept_end) : kept_end;
            auto fetch = [&](int t, int page, int64_t& place, float& have, float& ks) {
                const int pos = t * kTok + mine;
                place = (pos < it.prefix || pos >= touched_from) && is_page(pos, page) ? place_of(page, pos) : -1;
                const bool adds = j.row0 > 0 || pos < kept_end;
                have = adds && place >= 0 ? ld_dep_f32(a.mass + place) : 0.0f;
                ks = place >= 0 ? ld_dep_f32(a.c.k_scale + place) : 0.0f;
            };
            auto look_up = [&](int i) { return i < j.n ? page_of(j.tile(i) * kTok + mine) : 0; };
            // The accumulator's tiles are every other one; the first one's values are on their way while the queries are staged,
            // once the rows before are done with theirs.
            const int first = (static_cast<uint32_t>(acc) - seq) & 1;
            int64_t place = -1;
            float have = 0.0f, ks = 0.0f;
            const int page = look_up(first);
            int page_ahead = look_up(first + 2);
            const int r0 = (warp - 4) * 32;
            const int r = j.row0 + r0 + lane;  // this lane's row of the sequence's
            const int qi = r / a.group, hg = r - qi * a.group;
            float lse = kNegInf;
            if (r0 + lane < j.nrows)
                lse = ld_dep_f32(a.lse + static_cast<int64_t>(it.q0 + qi) * (a.c.heads * a.group) + it.h * a.group + hg);

            // Queries: rows 32 (warp - 4) .. + 31 of the job, once the job before is done with its own.
            if (jobs > 0 && !(ok = wait(rows_done, (jobs - 1) & 1))) break;
            if (jobs > 0 && !(ok = wait(mma_done, (jobs - 1) & 1))) break;
            if (first < j.n) fetch(j.tile(first), page, place, have, ks);
            if (r0 < j.columns) {
                stage_query_parts(smem + kQ + r0 * kD, kRows * kD, a.q,
                                  (it.q0 + qi) * a.q_stride + static_cast<int64_t>(it.h * a.group + hg) * kD, j.nrows - r0,
                                  [&](int row, float step) { row_scores[r0 + row].qs = row_scale(step, a.scale_log2); });
                __syncwarp();  // (the rows' scales were written by other lanes)
                const float qs = row_scores[r0 + lane].qs;
                RowScore info = row_score(a.scores, it.q0, it.len, it.nq, a.group, it.h, r, a.index_error);
                info.qs = qs;
                float less = kNegInf;  // a row that is not one, or sees nothing, adds nothing
                if (lse != kNegInf) less = lse * -1.4426950408889634f;
                if (r0 + lane >= j.nrows) info.lo = info.limit = 0;
                row_scores[r0 + lane] = info;
                float* const pair = pairs + (r0 + lane) / 2 * 4 + (lane & 1);
                pair[0] = qs;
                pair[2] = less;
                fence_async_proxy();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(q_full);
            if (!(ok = wait(q_full, jobs & 1))) break;

            // Tiles that no row sees get nothing; those that start from zero are zero.
            if (j.row0 == 0 && j.n < j.t1 - j.t0)
                for (int v = j.t0 + acc; v < j.t1; v += 2) {
                    const int t = v * kTok < it.prefix ? v : v + it.skip;
                    if (v < j.t0 + j.a_n || (t >= j.b0 && t < j.b0 + j.n - j.a_n) || (t + 1) * kTok <= kept_end) continue;
                    int64_t at;
                    float old, unused;
                    fetch(t, page_of(t * kTok + mine), at, old, unused);
                    if (at >= 0) a.mass[at] = old;
                }

            for (int i = first; i < j.n; i += 2) {
                const uint32_t n = seq + i;
                const int64_t to = place;
                const float old = have, k = ks;
                const int pos0 = j.tile(i) * kTok, pos = pos0 + mine;
                if (i + 2 < j.n) fetch(j.tile(i + 2), page_ahead, place, have, ks);
                page_ahead = look_up(i + 4);
                if (!(ok = wait(s_full + 8 * acc, n >> 1 & 1))) break;
                tc::fence_after_sync();
                const bool edge = on_edge(pos0, kTok, it.prefix, j.lo, j.limit);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                const float2 k2 = make_float2(k, k);
                auto add = [&](const uint32_t (&s)[32], const float4 (&row)[16], int c) {  // columns c .. c + 31
                    float2 y[16];
#pragma unroll
                    for (int w = 0; w < 16; ++w) {
                        y[w] = __fmul2_rn(make_float2(__uint_as_float(s[2 * w]), __uint_as_float(s[2 * w + 1])), k2);
                        y[w] = kChanged ? __fmul2_rn(y[w], make_float2(row[w].x, row[w].y))
                                       : __ffma2_rn(y[w], make_float2(row[w].x, row[w].y), make_float2(row[w].z, row[w].w));
                    }
                    if constexpr (kChanged) {
                        if (a.scores.capped)
                            cap_scores<16>([&](int w) { return y[w]; }, [&](int w, const float2& z) { y[w] = z; });
                        if (a.scores.slopes) {
                            // (distances from the sequence's end, which are small whole numbers where they matter)
                            const float from = static_cast<float>(pos - it.len);
#pragma unroll
                            for (int w = 0; w < 16; ++w) {
                                const RowScore r0 = row_scores[c + 2 * w], r1 = row_scores[c + 2 * w + 1];
                                y[w].x = fmaf(-r0.slope, fabsf(static_cast<float>(r0.limit - 1 - it.len) - from), y[w].x);
                                y[w].y = fmaf(-r1.slope, fabsf(static_cast<float>(r1.limit - 1 - it.len) - from), y[w].y);
                            }
                        }
#pragma unroll
                        for (int w = 0; w < 16; ++w) y[w] = __ffma2_rn(y[w], make_float2(a.scores.unit, a.scores.unit), make_float2(row[w].z, row[w].w));
                    }
                    if (edge) {
#pragma unroll
                        for (int w = 0; w < 32; ++w) {
                            const RowScore r = row_scores[c + w];
                            float& z = w & 1 ? y[w >> 1].y : y[w >> 1].x;
                            if (pos >= it.prefix && (pos < r.lo || pos >= r.limit)) z = kNegInf;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < 16; ++w) sum[w & 1] = __fadd2_rn(sum[w & 1], make_float2(ex2(y[w].x), ex2(y[w].y)));
                };
                // The rows' values of 32 columns are asked for together, and the scores of the next 32.
                float4 row[16];
                auto rows_from = [&](int c) {
#pragma unroll
                    for (int w = 0; w < 16; ++w) row[w] = lds_v4(ptx::smem_u32(pairs) + (c + 2 * w) * 8);
                };
                uint32_t s0[32], s1[32];
                tc::ld_32x32b_x32(t_s, s0);
#pragma unroll 1
                for (int c = 0; c < j.columns; c += 64) {
                    rows_from(c);
                    tc::wait_ld(s0);
                    if (c + 32 < j.columns) tc::ld_32x32b_x32(t_s + c + 32, s1);
                    add(s0, row, c);
                    if (c + 32 >= j.columns) break;
                    rows_from(c + 32);
                    tc::wait_ld(s1);
                    if (c + 64 < j.columns) tc::ld_32x32b_x32(t_s + c + 64, s0);
                    add(s1, row, c + 32);
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(s_empty + 8 * acc);
                if (to >= 0) a.mass[to] = old + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(rows_done);
            ++jobs;
            if (!next(j)) break;
        }
    }

    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 2) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <bool kChanged>
cudaError_t launch(const AttnArgs& a, int num_sms, cudaStream_t stream) {
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaGetDevice(&dev);
    auto kernel = kv_mass_tc_kernel<kChanged>;
    if (!configured[dev & 63].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
        if (e != cudaSuccess) return e;
        configured[dev & 63].store(true, std::memory_order_relaxed);
    }
    // The cache as rows of one token and head; a copy is a page's tokens, 128 at most.
    const uint64_t tokens = static_cast<uint64_t>(a.c.num_pages) * a.c.heads << a.c.page_log2;
    const uint32_t box = 1u << a.c.page_log2 < kTok ? 1u << a.c.page_log2 : kTok;
    CUtensorMap k_map;
    if (!encode_tmap_2d_u8(&k_map, a.c.k, kD, tokens, kD, kD, box, true)) return cudaErrorInvalidValue;
    const Extra x = {tile_wait_limit_ns(), tile_withhold_first_load() ? 1 : 0};
    return launch_dependent(kernel, dim3(num_sms), kThreads, kBytes, stream, 1, a, k_map, x);
}

}  // namespace

cudaError_t launch_mass_tc(const AttnArgs& a, int num_sms, cudaStream_t stream) {
    return a.scores.kind == ScoreKind::kChanged ? launch<true>(a, num_sms, stream) : launch<false>(a, num_sms, stream);
}

unsigned int read_and_clear_mass_timeout() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_mass_timeout, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_mass_timeout, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace fp8act
