// The attention weight that every cached token gets: with the scores x of
// kv_attention.cu and the log-sum-exp that the attention left of each row,
//   mass[j] (+)= sum over the rows of a KV head of exp(x[r, j] - lse[r]).
//
// The scores are computed again, f16 MMAs of S^T = K Q^T as there, and no
// maximum is needed: the log-sum-exp bounds every exponent by 0. A row of the
// accumulator is a cached token, so its sum over the query rows stays in the
// lane that has it, and a token's codes stay in registers, widened once, while
// all the rows go by in shared memory.
//
// Work split. A unit is 32 cached tokens of a KV head with all the sequence's
// rows; a warp takes whole units, so that no sum is joined and the order is
// fixed. The units of all sequences and heads form one list, shared evenly by the
// CTAs, weighted by their rows; tiles that no row sees and whose tokens keep their
// weights are not in it. A warp has its own ring of key tiles in
// flight. Rows come 256 at a time (128 for D = 256); with more, a token's sum
// goes through its place in memory between them.
//
// What bounds it with few rows: the trips at a warp's start, lengths to page
// table to keys. 34 sequences of one token to 16384, 6 heads on each of 4: 17.4
// us on the device, 2.3 TB/s (6.0 us at a copy's rate); all of 16384 56.8, 5.5 TB/s.
// In a window a sequence's other tokens cost nothing: of 4096 20.4 us.
#include <atomic>

#include "kv_attention.cuh"

namespace fp8act {
namespace {

__device__ unsigned int g_mass_index_error;

constexpr int kTile = 32;
// Rows from which on head size 128 takes the tcgen05 kernel, which is then faster throughout (us, here and there: 36 rows of
// one sequence of 131072 26.5 and 25.0, of one of 4096 11.1 and 9.0, of 34 ragged ones to 16384 70.1 and 54.1). With fewer it
// goes by the lengths: 24 rows 21.3 and 22.1, 9.5 and 8.4, 55.9 and 48.5, of 8 sequences of 2048 9.9 and 10.3.
constexpr int kWideRows = 33;
constexpr int kItemCost = 8;  // units that an item counts beside its own, for its start
using Work = Units<kTile, kItemCost, List::kMass>;

// Many rows: one CTA per SM whose warps share the rows in shared memory, as many as the registers allow that a tile's
// widened codes take (half of kD a thread). Few rows (kFew): CTAs of one warp, several per SM, so that a short sequence
// costs one warp its start and not a CTA; 34 sequences of one token to 16384: 51.0 us with whole CTAs, 21.2 with 8 of
// one warp an SM, 18.0 with 16.
template <int kD, bool kFew>
struct Mass {
    static constexpr int kWarps = kFew ? 1 : kD == 64 ? 16 : kD == 128 ? 12 : 8;
    static constexpr int kCtas = !kFew ? 1 : kD == 256 ? 8 : 16;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRows = kFew ? 16 : kD == 256 ? 128 : 256;
    static constexpr int kStageBytes = kTile * kD + kTile * 4;  // keys, key scales
    static constexpr int kRowBytes = kD * 2 + 16 + 8;           // queries, RowScore, (qs, -lse)
    static constexpr int kRoom = 226 * 1024 / kCtas - 1024 * (kCtas > 1 ? 1 : 0);
    static int stages(int rows) {
        const int fit = (kRoom - rows * kRowBytes) / (kWarps * kStageBytes);
        return fit < 8 ? fit : 8;
    }
    static_assert((kRoom - kRows * kRowBytes) / (kWarps * kStageBytes) >= 2, "a tile in flight beside the one being read");
};

// (Plain scores have an instance of their own, without the masks' tests of what a row sees: 34 single tokens over 16384
// 56.8 us, and 60.2 with them.)
template <int kD, bool kFew, ScoreKind kKind>
__global__ void __launch_bounds__(Mass<kD, kFew>::kThreads, Mass<kD, kFew>::kCtas)
    kv_mass_kernel(const __grid_constant__ AttnArgs a, int stages) {
    using M = Mass<kD, kFew>;
    constexpr int kKS = kD / 32;
    constexpr bool kScored = kKind != ScoreKind::kPlain, kChanged = kKind == ScoreKind::kChanged;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Work::Scratch scratch;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, qd = lane & 3;
    const int og = order<kD>(g);  // the token of a block of 8 that is the lane's MMA row
    uint8_t* const queries = smem;
    RowScore* const row_scores = reinterpret_cast<RowScore*>(smem + a.rows * kD * 2);
    float2* const row_mass = reinterpret_cast<float2*>(row_scores + a.rows);  // (qs, -lse) in log2
    uint8_t* const ring = smem + a.rows * M::kRowBytes + warp * stages * M::kStageBytes;

    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    Item it;
    int64_t per, u, u_end;
    if (!Work::first_item(a, kFew ? 4 : M::kWarps, scratch, it, per, u, u_end)) return;
    while (true) {
        const int64_t item_end = it.first + it.tiles;
        const int rows_total = it.nq * a.group, weight = mass_weight(rows_total);
        // Tile t of the item is this CTA's if its first unit is.
        auto tile_of = [&](int64_t unit) {
            return static_cast<int>((max(unit - it.first - kItemCost, int64_t{0}) + weight - 1) / weight);
        };
        const int t0 = tile_of(u), t1 = tile_of(item_end < u_end ? item_end : u_end);
        const int* table = a.table + it.b * a.table_stride;
        const int in_page = (1 << a.c.page_log2) - 1;
        const int kept_end = old_end(a, it.b, it.len, it.nq);
        const int prefix = kScored ? it.prefix : 0;
        auto position = [&](int t) { return t * kTile + (t * kTile < prefix ? 0 : it.skip * kTile); };

        int row0 = 0;
        do {
            const int nrows = min(rows_total - row0, a.rows), blocks = (nrows + 7) / 8;
            int lo_first = 0, lo_last = 0, limit_first = 0, limit_last = 0;
            if (nrows > 0) {
                const int q_first = row0 / a.group, q_last = (row0 + nrows - 1) / a.group;
                limit_first = it.len - it.nq + q_first + 1;
                limit_last = it.len - it.nq + q_last + 1;
                if constexpr (kScored) {
                    lo_first = first_seen(a.scores, it.q0, it.len, it.nq, q_first);
                    lo_last = first_seen(a.scores, it.q0, it.len, it.nq, q_last);
                }
            }
            // Whether some row may see a token of the tile at pos.
            auto seen = [&](int pos) { return pos < prefix || (pos < limit_last && pos + kTile > lo_first); };
            // Whether one of n tokens from pos on may be touched: not those that no row sees and that keep their weight, whose
            // pages may be another sequence's by now.
            const int touched_from = row0 > 0 ? lo_first : nrows > 0 ? min(lo_first, kept_end) : kept_end;
            auto touched = [&](int pos, int n) { return pos < prefix || pos + n > touched_from; };
            // The warp's tiles are t0 + warp, + kWarps, ... Pages of its next 16, one per 16 tokens and lane.
            auto look_up = [&](int t) -> int {
                t += (lane >> 1) * M::kWarps;
                const int pos = position(t) + (lane & 1) * 16;
                if (t >= t1 || pos >= it.len || !touched(pos, 16)) return -1;
                const int p = ld_dep_s32(table + (pos >> a.c.page_log2));
                if (p >= 0 && p < a.c.num_pages) return p;
                atomicOr(a.index_error, 1u);
                return -1;
            };
            const int first_pages = look_up(t0 + warp);
            int pages = first_pages, asked = 0;
            auto place_of = [&](int pos, int page) -> int64_t {
                return page >= 0 && pos < it.len && touched(pos, 1)
                           ? ((static_cast<int64_t>(page) * a.c.heads + it.h) << a.c.page_log2) + (pos & in_page)
                           : -1;
            };
            auto request = [&](int t, int stage) {
                if (t < t1) {
                    const int p0 = __shfl_sync(0xffffffffu, pages, 2 * asked), p1 = __shfl_sync(0xffffffffu, pages, 2 * asked + 1);
                    const int pos0 = position(t);
                    if (seen(pos0)) {
                        const uint32_t dst = ptx::smem_u32(ring) + stage * M::kStageBytes;
                        constexpr int kC = kD / 16, kStep = 32 / kC, kSteps = 32 / kStep;  // chunks per token, tokens per instruction
                        const int c = lane % kC, r0 = lane / kC;
                        const int64_t row_a = ((static_cast<int64_t>(p0) * a.c.heads + it.h) << a.c.page_log2) + (pos0 & in_page);
                        const int64_t row_b =
                            ((static_cast<int64_t>(p1) * a.c.heads + it.h) << a.c.page_log2) + ((pos0 + 16) & in_page) - 16;
                        const int end_a = p0 >= 0 ? it.len - pos0 : 0, end_b = p1 >= 0 ? it.len - pos0 : 0;  // tokens there are
                        const uint32_t scales = dst + kTile * kD + lane * 4;
                        if (min(end_a, end_b) >= kTile) {
                            const uint8_t *ka = a.c.k + (row_a + r0) * kD + c * 16, *kb = a.c.k + (row_b + r0) * kD + c * 16;
#pragma unroll
                            for (int j = 0; j < kSteps; ++j)
                                cp_async16(dst + stage_offset<kD>(j * kStep + r0, c), (j * kStep < 16 ? ka : kb) + j * kStep * kD, true);
                            cp_async4(scales, a.c.k_scale + (lane < 16 ? row_a : row_b) + lane, true);
                        } else {
#pragma unroll 1
                            for (int j = 0; j < kSteps; ++j) {
                                const int row = j * kStep + r0;
                                const bool first = j * kStep < 16, in = row < (first ? end_a : end_b);
                                cp_async16(dst + stage_offset<kD>(row, c), a.c.k + (in ? ((first ? row_a : row_b) + row) * kD + c * 16 : 0), in);
                            }
                            const bool in = lane < (lane < 16 ? end_a : end_b);
                            cp_async4(scales, a.c.k_scale + (in ? (lane < 16 ? row_a : row_b) + lane : 0), in);
                        }
                    }
                    if (++asked == 16) {
                        asked = 0;
                        pages = look_up(t + M::kWarps);
                    }
                }
                cp_async_commit();
            };
            // (the number of stages is not known to the compiler, the number of groups in flight has to be)
            auto wait_for_tile = [&]() {
                switch (stages) {
                    case 2: cp_async_wait<0>(); break;
                    case 3: cp_async_wait<1>(); break;
                    case 4: cp_async_wait<2>(); break;
                    case 5: cp_async_wait<3>(); break;
                    case 6: cp_async_wait<4>(); break;
                    case 7: cp_async_wait<5>(); break;
                    default: cp_async_wait<6>(); break;
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int i = 0; i < stages - 1; ++i) request(t0 + warp + i * M::kWarps, i);

            stage_queries<kD, M::kThreads>(
                queries, blocks * 8,
                [&](int r, int c) {
                    if (r >= nrows) return make_uint4(0, 0, 0, 0);
                    const int qi = (row0 + r) / a.group, hg = (row0 + r) - qi * a.group;
                    return ld_dep_v4(a.q + (it.q0 + qi) * a.q_stride + (it.h * a.group + hg) * kD + c * 8);
                },
                [&](int r, float step) { row_scores[r].qs = row_mass[r].x = row_scale(step, a.scale_log2); });
            for (int r = threadIdx.x; r < blocks * 8; r += M::kThreads) {  // (a thread per row)
                RowScore info = row_score(a.scores, it.q0, it.len, it.nq, a.group, it.h, row0 + r, a.index_error);
                float less = kNegInf;  // a row that is not one, or sees nothing, adds nothing
                if (r < nrows) {
                    const int qi = (row0 + r) / a.group, hg = (row0 + r) - qi * a.group;
                    const float lse = ld_dep_f32(a.lse + static_cast<int64_t>(it.q0 + qi) * (a.c.heads * a.group) + it.h * a.group + hg);
                    if (lse != kNegInf) less = lse * -1.4426950408889634f;
                } else {
                    info.lo = info.limit = 0;
                }
                row_scores[r].lo = info.lo;
                row_scores[r].limit = info.limit;
                row_scores[r].slope = info.slope;
                row_mass[r].y = less;
            }
            __syncthreads();

            // Where the weight of the token is that is this lane's in the end, and what it has so far: a tile ahead.
            int used = 0, held = first_pages;
            const int my_token = qd * 8 + og;
            int64_t mine = -1;
            float have = 0.0f;
            auto look_ahead = [&](int t) {
                if (t >= t1) return;
                const int pos = position(t) + my_token;
                mine = place_of(pos, __shfl_sync(0xffffffffu, held, 2 * used + (my_token >> 4)));
                if (++used == 16) {
                    used = 0;
                    held = look_up(t + M::kWarps);
                }
                const bool adds = row0 > 0 || pos < kept_end;
                have = adds && mine >= 0 ? ld_dep_f32(a.mass + mine) : 0.0f;
            };
            look_ahead(t0 + warp);
            int stage = 0;
#pragma unroll 1
            for (int t = t0 + warp; t < t1; t += M::kWarps) {
                const int64_t to = mine;
                const float old = have;
                look_ahead(t + M::kWarps);
                wait_for_tile();
                const uint8_t* kt = ring + stage * M::kStageBytes;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                const int pos0 = position(t);
                if (seen(pos0)) {
                    // The tile's codes as A fragments: af[k-step][16 tokens][4].
                    uint32_t af[kD / 16][2][4];
                    float ks[4];
                    const float* sk = reinterpret_cast<const float*>(kt + kTile * kD);
#pragma unroll
                    for (int x = 0; x < 4; ++x) ks[x] = sk[x * 8 + og];
#pragma unroll
                    for (int w = 0; w < kD / 64; ++w)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint4 v = *reinterpret_cast<const uint4*>(kt + stage_offset<kD>(x * 16 + y * 8 + og, w * 4 + qd));
                                const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    af[w * 4 + z][x][y] = e4m3x2_lo_to_f16x2(words[z]);
                                    af[w * 4 + z][x][y + 2] = e4m3x2_hi_to_f16x2(words[z]);
                                }
                            }
                    __syncwarp();  // the stage is read
                    request(t + (stages - 1) * M::kWarps, stage == 0 ? stages - 1 : stage - 1);
                    const bool edge = on_edge(pos0, kTile, prefix, lo_last, limit_first);
                    const uint4* qf = reinterpret_cast<const uint4*>(queries) + lane;
                    auto rows_of = [&](auto masks, int i) {
                        float s[2][4] = {};
#pragma unroll
                        for (int k = 0; k < kKS; ++k) {
                            const uint4 b = qf[(i * kKS + k) * 32];
#pragma unroll
                            for (int x = 0; x < 2; ++x) mma_f16(s[x], af[2 * k][x], b.x, b.y);
#pragma unroll
                            for (int x = 0; x < 2; ++x) mma_f16(s[x], af[2 * k + 1][x], b.z, b.w);
                        }
                        const float4 row = *reinterpret_cast<const float4*>(row_mass + i * 8 + qd * 2);
                        const RowScore* const info = row_scores + i * 8 + qd * 2;
                        // y[2 j + e]: token j * 8 + og, row 2 qd + e
                        float y[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            y[j] = s[j >> 2][j & 3] * ks[j >> 1];
                            const float qs = j & 1 ? row.z : row.x, less = j & 1 ? row.w : row.y;
                            y[j] = kChanged ? y[j] * qs : fmaf(y[j], qs, less);
                        }
                        if constexpr (kChanged) {
                            if (a.scores.capped)
                                cap_scores<4>(
                                    [&](int j) { return make_float2(y[2 * j], y[2 * j + 1]); },
                                    [&](int j, const float2& z) {
                                        y[2 * j] = z.x;
                                        y[2 * j + 1] = z.y;
                                    });
                            if (a.scores.slopes) {
                                const float slope[2] = {info[0].slope, info[1].slope};
                                const float far[2] = {static_cast<float>(info[0].limit - 1 - pos0 - og), static_cast<float>(info[1].limit - 1 - pos0 - og)};
#pragma unroll
                                for (int j = 0; j < 8; ++j) y[j] = fmaf(-slope[j & 1], fabsf(far[j & 1] - (j >> 1) * 8), y[j]);
                            }
#pragma unroll
                            for (int j = 0; j < 8; ++j) y[j] = fmaf(y[j], a.scores.unit, j & 1 ? row.w : row.y);
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float p = ex2(y[j]);
                            if constexpr (decltype(masks)::value) {
                                const int pos = pos0 + (j >> 1) * 8 + og;
                                if (pos >= prefix && (pos < info[j & 1].lo || pos >= info[j & 1].limit)) p = 0.0f;
                            }
                            sum[j >> 1] += p;
                        }
                    };
                    if (edge) {
#pragma unroll 1
                        for (int i = 0; i < blocks; ++i) rows_of(std::true_type{}, i);
                    } else {
#pragma unroll 2
                        for (int i = 0; i < blocks; ++i) rows_of(std::false_type{}, i);
                    }
                } else {
                    __syncwarp();
                    request(t + (stages - 1) * M::kWarps, stage == 0 ? stages - 1 : stage - 1);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
                    sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
                }
                const float total = qd == 0 ? sum[0] : qd == 1 ? sum[1] : qd == 2 ? sum[2] : sum[3];
                if (to >= 0) a.mass[to] = old + total;
                stage = stage + 1 == stages ? 0 : stage + 1;
            }
            cp_async_wait<0>();
            row0 += a.rows;
            __syncthreads();  // the queries and the rings are free
        } while (row0 < rows_total);
        if (item_end >= u_end) break;
        u = item_end;
        Work::next_item(a, it);
    }
}

template <int kD, bool kFew, ScoreKind kKind>
cudaError_t launch(AttnArgs& a, int64_t rows, int num_sms, cudaStream_t stream) {
    using M = Mass<kD, kFew>;
    a.rows = rows >= M::kRows ? M::kRows : rows < 8 ? 8 : static_cast<int>((rows + 7) / 8 * 8);
    const int stages = M::stages(a.rows);
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaGetDevice(&dev);
    auto kernel = kv_mass_kernel<kD, kFew, kKind>;
    if (!configured[dev & 63].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, M::kRoom);
        if (e != cudaSuccess) return e;
        configured[dev & 63].store(true, std::memory_order_relaxed);
    }
    const size_t bytes = a.rows * M::kRowBytes + static_cast<size_t>(M::kWarps) * stages * M::kStageBytes;
    return launch_dependent(kernel, dim3(num_sms * M::kCtas), M::kThreads, bytes, stream, 1, a, stages);
}

template <int kD, ScoreKind kKind>
cudaError_t launch_rows(AttnArgs& a, int max_q_len, int num_sms, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(max_q_len) * a.group;
    if (kD == 128 && rows >= kWideRows) {
        a.rows = kWideRows;  // (any: an item has all rows)
        return launch_mass_tc(a, num_sms, stream);
    }
    // CTAs of one warp for as many rows as one pass of them takes (us, with them and with whole CTAs, D = 128: 12 rows of 34
    // ragged sequences to 16384 40.8 and 50.0, of one of 131072 21.4 and 18.6; 18 rows, two passes, 69.2 and 56.2, 33.7 and 21.5).
    return rows <= Mass<kD, true>::kRows ? launch<kD, true, kKind>(a, rows, num_sms, stream)
                                         : launch<kD, false, kKind>(a, rows, num_sms, stream);
}

template <int kD>
cudaError_t launch_kind(AttnArgs& a, int max_q_len, int num_sms, cudaStream_t stream) {
    switch (a.scores.kind) {
        case ScoreKind::kPlain: return launch_rows<kD, ScoreKind::kPlain>(a, max_q_len, num_sms, stream);
        case ScoreKind::kMasked: return launch_rows<kD, ScoreKind::kMasked>(a, max_q_len, num_sms, stream);
        default: return launch_rows<kD, ScoreKind::kChanged>(a, max_q_len, num_sms, stream);
    }
}

}  // namespace

cudaError_t launch_kv_mass(const MassProblem& p, int num_sms, cudaStream_t stream) {
    AttnArgs a = {};
    a.q = static_cast<const uint16_t*>(p.q);
    a.q_stride = p.q_stride;
    a.cu_q = p.cu_q;
    a.kv_lens = p.kv_lens;
    a.table = p.page_table;
    a.table_stride = p.table_stride;
    a.batch = p.batch;
    a.tokens = p.tokens;
    a.group = p.group;
    a.rows = 1;
    void* error = nullptr;
    const cudaError_t found = cudaGetSymbolAddress(&error, g_mass_index_error);
    if (found != cudaSuccess) return found;
    a.index_error = static_cast<unsigned int*>(error);
    a.scale_log2 = p.softmax_scale * 1.4426950408889634f / p.scores.unit;
    a.c = p.cache;
    a.lse = const_cast<float*>(p.lse);
    a.scores = p.scores;
    a.mass = p.mass;
    a.accumulate = p.accumulate;
    a.old_lens = p.old_lens;
    switch (p.cache.head_dim) {
        case 64: return launch_kind<64>(a, p.max_q_len, num_sms, stream);
        case 128: return launch_kind<128>(a, p.max_q_len, num_sms, stream);
        default: return launch_kind<256>(a, p.max_q_len, num_sms, stream);
    }
}

unsigned int read_and_clear_mass_index_error() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_mass_index_error, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_mass_index_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace fp8act
