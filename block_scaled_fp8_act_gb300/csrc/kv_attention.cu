// Attention of new tokens over the paged E4M3 cache (decode, draft verify,
// prompt chunks), grouped query heads, causal from the end of the sequence.
//
// For a sequence with L cached tokens, n of them new, new token i sees the
// positions <= L - n + i. With codes k, v and one scale per token and head,
//   S[r, j] = softmax_scale * s_k[j] * (q_r . k_j),   P = softmax(S),
//   O[r]    = sum_j P[r, j] s_v[j] v_j.
//
// Arithmetic. Codes widen exactly to f16 (cvt.rn.f16x2.e4m3x2), so both
// products run as f16 MMAs with fp32 accumulation. (The warp-level E4M3 MMA is
// built from f16 ones with conversions and fp32 additions by the compiler:
// queries as pairs of E4M3 rows took 106 us where f16 took 83, at 8 tokens
// over 131072.) Both are transposed, S^T = K Q^T and O^T = V^T W^T, so that the
// cached tokens and the output columns are the MMA's 16 rows and the query rows
// its 8 columns: a decode step of 6 or 8 heads fills them. A query row is
// scaled by a power of two so that its largest value is in [1, 2): bf16 then
// fits f16 exactly down to 2^-17 of the largest value, and below that to
// within 2^-25 of it. The weights W = p * s_v are rounded to f16 (11 bits; bf16
// would give 8) after scaling by 2^6 / R, R the power of two below the largest
// s_v so far: p s_v keeps its 11 bits down to 2^-20 R, and below that is within
// 2^-31 R. The running maximum moves only when a score passes it by 8 (in
// log2), so that the accumulators are seldom rescaled; a weight then stays
// below 2^15. Maxima, sums, and both accumulations are fp32.
//
// Work split. A row tile is up to 192 rows of (new token, query head of one KV
// head); a unit is one row tile x 32 cached tokens. The units of all
// sequences, KV heads and row tiles form one list, which the CTAs, up to two
// per SM, share evenly: no host knowledge of the lengths is needed and a ragged batch
// balances itself. An item (sequence, head, row tile) counts kItemCost units
// more than it has, about what its start and end cost, so that short ones
// spread out. In a CTA, groups of warps take an item's units in turn, each with
// its own ring of cached tokens and its own running softmax; a group's warps
// share a ring and split the rows. The groups join in shared memory. An item
// that crosses CTAs leaves fp32 parts in the workspace, which a second kernel,
// launched dependently, adds in unit order: results do not depend on timing.
//
// What bounds it, by rows of a tile (D = 128): with up to 8 (one token) the
// cache's bytes, 31 us for 131072 tokens x 4 heads (0.81 of a copy's rate while
// it streams); with 24 (34 sequences x 3 tokens, ragged up to 16384: 33 us, 0.38)
// and 48 (8 tokens over 131072: 59 us, 0.35) the latency of a unit's chain, keys
// to scores to weights to output, with 8 and 12 warps an SM to hide it: their
// accumulators fill the registers. A single token over 4096 tokens takes 9.0
// us, the chain of the two kernels.
#include <atomic>
#include <type_traits>

#include "kv_attention.cuh"

namespace fp8act {
namespace {

__device__ unsigned int g_attn_index_error;

constexpr int kTile = 32;  // cached tokens per unit
constexpr int kLeastUnits = 8;  // least share of a CTA
constexpr int kItemCost = 20;   // units that an item counts beside its own
using Work = Units<kTile, kItemCost>;

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit values held as an MMA fragment.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// A stage holds the cached codes as 128-byte lines, as the cache does (a token
// is half a line, a line or two); chunk c of a line sits at c ^ (line % 8).
// Byte offset of 16-byte chunk c of
// token `row`:
template <int kD>
__device__ __forceinline__ uint32_t stage_offset(int row, int c) {
    const int line = kD == 64 ? row >> 1 : kD == 128 ? row : row * 2 + (c >> 3);
    const int chunk = kD == 64 ? ((row & 1) << 2) | c : c & 7;
    return line * 128 + ((chunk ^ (line & 7)) << 4);
}

// The MMA's rows are the cached tokens of a block of 8 in an order of our own:
// row i is token order<kD>(i). The 8 lanes of a shared-memory phase read 4
// chunks of 2 neighbouring rows; the order gives those two tokens swizzles
// that differ in bit 2, so that they read distinct banks.
template <int kD>
__device__ __forceinline__ int order(int i) {
    if (kD == 64) return i;
    if (kD == 128) return (i >> 1) | ((i & 1) << 2);
    return ((i >> 1) & 1) | ((i & 1) << 1) | (i & 4);
}

// kWR warps of a group split the row tile, kRW groups of 8 rows each; kG groups in a CTA; kCtas CTAs per SM (two
// where a group is one warp: one streams while the other starts or ends an item, 38 us instead of 46 for 34 ragged
// sequences x 3 tokens; but one for D = 256, whose stages are twice as large: one token over 32768 with 8 heads on 4
// 30.2 us instead of 42.2, two tokens of 8 ragged sequences 23.1 instead of 32.8).
template <int kD, int kWR, int kRW, int kG, int kCtas_>
struct Attn {
    static constexpr int kCtas = kCtas_;
    static constexpr int kWarpRows = kRW * 8;
    static constexpr int kRows = kWR * kWarpRows;
    static constexpr int kWarps = kWR * kG;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kStageBytes = 2 * kTile * kD + 2 * kTile * 4;  // keys, values, key scales, value scales
    static constexpr int kQ = 0;
    static constexpr int kML = kQ + kRows * kD * 2;
    static constexpr int kQScale = kML + kG * kRows * 8;
    static constexpr int kRing = (kQScale + kRows * 4 + 127) / 128 * 128;
    static constexpr int kFit = (226 * 1024 / kCtas - 1024 * (kCtas - 1) - kRing) / kG / kStageBytes;
    static constexpr int kStages = kFit < 8 ? kFit : kFit < 16 && kG > 1 ? 8 : kFit < 16 ? kFit : 16;
    static constexpr int kRingBytes = kStages * kStageBytes;
    static constexpr int kOStride = kD + 4;  // floats of a row of a group's result, which replaces its ring at the end
    static_assert(kStages >= 2 && kRows * kOStride * 4 <= kRingBytes, "a stage in flight, and room for the result");
    static constexpr int kBytes = kRing + kG * kRingBytes;
};

// One finished row: lane's kD / 32 columns of sum p s_v v, the row's maximum (log2) and sum of p.
template <int kD>
__device__ __forceinline__ void write_row(const AttnArgs& a, int q0, int h, int row, int lane, float m, float sum,
                                          const float (&o)[kD / 32]) {
    const int qi = row / a.group, hg = row - qi * a.group;
    const int64_t at = static_cast<int64_t>(q0 + qi) * (a.c.heads * a.group) + h * a.group + hg;
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int x = 0; x < kD / 32; x += 2) a.out[(at * kD + lane * (kD / 32) + x) >> 1] = pack_bf16x2(o[x] * f, o[x + 1] * f);
    if (a.lse && lane == 0) a.lse[at] = sum == 0.0f ? kNegInf : (m + log2f(sum)) * 0.6931471805599453f;
}

template <int kD, int kWR, int kRW, int kG, int kCtas>
__global__ void __launch_bounds__(Attn<kD, kWR, kRW, kG, kCtas>::kThreads, kCtas)
    kv_attention_kernel(const __grid_constant__ AttnArgs a) {
    using S = Attn<kD, kWR, kRW, kG, kCtas>;
    constexpr int kRows = S::kRows, kStages = S::kStages;
    constexpr int kKS = kD / 32;  // pairs of k-steps of the score product
    constexpr int kDT = kD / 16;  // 16-row tiles of the transposed output
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Work::Scratch scratch;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, qd = lane & 3;
    const int og = order<kD>(g);                  // the token of a block of 8 that is the lane's MMA row
    const int vg = kD == 64 ? g : order<128>(g);  // the chunk of output columns that is the lane's (the same reason)
    const int group = warp / kWR, wr = warp % kWR;
    uint8_t* const ring = smem + S::kRing + group * S::kRingBytes;
    float* qscale = reinterpret_cast<float*>(smem + S::kQScale);
    float2* ml = reinterpret_cast<float2*>(smem + S::kML);
    auto group_sync = [&]() {
        if constexpr (kWR == 1)
            __syncwarp();
        else
            ptx::named_bar_sync(1 + group, kWR * 32);
    };

    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    Item it;
    int64_t per, u, u_end;
    if (!Work::first_item(a, kLeastUnits, scratch, it, per, u, u_end)) return;
    const int64_t u_begin = u;

    while (true) {
        const int t0 = static_cast<int>(u - it.first);
        const int64_t item_end = it.first + it.tiles;
        const int t1 = static_cast<int>((item_end < u_end ? item_end : u_end) - it.first);
        const int rows_total = it.nq * a.group;
        const int row0 = it.rt * kRows;
        const int nrows = rows_total - row0 < kRows ? rows_total - row0 : kRows;
        // This CTA's tiles [f0, f1): units past the item's cost, as far as some row of the tile sees.
        const int seen = max(it.len - it.nq + (row0 + nrows - 1) / a.group + 1, 0);
        const int f0 = max(t0 - kItemCost, 0), f1 = min((seen + kTile - 1) / kTile, t1 - kItemCost);

        // The group's tiles are f0 + group, + kG, ... Pages of its next 16, one per 16 tokens and lane.
        const int* table = a.table + it.b * a.table_stride;
        auto look_up = [&](int t) -> int {
            t += (lane >> 1) * kG;
            const int pos = t * kTile + (lane & 1) * 16;
            if (t >= f1 || pos >= it.len) return -1;
            const int p = ld_dep_s32(table + (pos >> a.c.page_log2));
            if (p >= 0 && p < a.c.num_pages) return p;
            atomicOr(a.index_error, 1u);
            return -1;
        };
        int pages = look_up(f0 + group), asked = 0;
        // Request the group's next tile, t, into `stage`: the group's warps share the 16-byte chunks.
        auto request = [&](int t, int stage) {
            if (t < f1) {
                const int p0 = __shfl_sync(0xffffffffu, pages, 2 * asked), p1 = __shfl_sync(0xffffffffu, pages, 2 * asked + 1);
                const uint32_t dst = ptx::smem_u32(ring) + stage * S::kStageBytes;
                constexpr int kC = kD / 16, kStep = 32 / kC;  // chunks per token, tokens per instruction
                const int c = lane % kC, r0 = lane / kC;
                const int pos0 = t * kTile, in_page = (1 << a.c.page_log2) - 1;
                const int64_t row_a = ((static_cast<int64_t>(p0) * a.c.heads + it.h) << a.c.page_log2) + (pos0 & in_page);
                const int64_t row_b =
                    ((static_cast<int64_t>(p1) * a.c.heads + it.h) << a.c.page_log2) + ((pos0 + 16) & in_page) - 16;
                const int end_a = p0 >= 0 ? it.len - pos0 : 0, end_b = p1 >= 0 ? it.len - pos0 : 0;  // tokens there are
                constexpr int kSteps = 32 / kStep;
                const uint32_t scales = dst + 2 * kTile * kD + lane * 4;
                if (min(end_a, end_b) >= kTile) {
                    // A whole tile, almost always: addresses are a base per page and constant offsets.
                    const int64_t at_a = (row_a + r0) * kD + c * 16, at_b = (row_b + r0) * kD + c * 16;
                    const uint8_t *ka = a.c.k + at_a, *kb = a.c.k + at_b, *va = a.c.v + at_a, *vb = a.c.v + at_b;
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) {
                        if (kWR > 1 && j % kWR != wr) continue;
                        const uint32_t off = dst + stage_offset<kD>(j * kStep + r0, c);
                        cp_async16(off, (j * kStep < 16 ? ka : kb) + j * kStep * kD, true);
                        cp_async16(off + kTile * kD, (j * kStep < 16 ? va : vb) + j * kStep * kD, true);
                    }
                    if (wr == 0) {
                        const int64_t at = (lane < 16 ? row_a : row_b) + lane;
                        cp_async4(scales, a.c.k_scale + at, true);
                        cp_async4(scales + kTile * 4, a.c.v_scale + at, true);
                    }
                } else {
#pragma unroll 1
                    for (int j = 0; j < kSteps; ++j) {
                        if (kWR > 1 && j % kWR != wr) continue;
                        const int row = j * kStep + r0;
                        const bool first = j * kStep < 16;
                        const bool in = row < (first ? end_a : end_b);
                        const int64_t at = in ? ((first ? row_a : row_b) + row) * kD + c * 16 : 0;
                        const uint32_t off = dst + stage_offset<kD>(row, c);
                        cp_async16(off, a.c.k + at, in);
                        cp_async16(off + kTile * kD, a.c.v + at, in);
                    }
                    if (wr == 0) {
                        const bool in = lane < (lane < 16 ? end_a : end_b);
                        const int64_t at = in ? (lane < 16 ? row_a : row_b) + lane : 0;
                        cp_async4(scales, a.c.k_scale + at, in);
                        cp_async4(scales + kTile * 4, a.c.v_scale + at, in);
                    }
                }
                if (++asked == 16) {
                    asked = 0;
                    pages = look_up(t + kG);
                }
            }
            cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) request(f0 + group + i * kG, i);

        // Queries: power-of-two scaled f16 in fragment order.
        {
            constexpr int kLanes = kD / 8;
            static_assert(kLanes <= 32 && kRows % (32 / kLanes) == 0, "whole warps of rows");
            const int c = threadIdx.x % kLanes;
            for (int r = threadIdx.x / kLanes; r < kRows; r += S::kWarps * 32 / kLanes) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (r < nrows) {
                    const int qi = (row0 + r) / a.group, hg = (row0 + r) - qi * a.group;
                    x = ld_dep_v4(a.q + (it.q0 + qi) * a.q_stride + (it.h * a.group + hg) * kD + c * 8);
                }
                // (a warp's rows are all below kRows or none is, so that the whole warp is here)
                uint32_t top = top_bits(x);
#pragma unroll
                for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                // (a zero row's exponent is as good as any)
                const uint32_t e = top == 0 ? 127 : min(max(top >> 7, 1u), 253u);
                const float up = __uint_as_float((254 - e) << 23);  // 2^(127 - e)
                if (c == 0) qscale[r] = fmaxf(__uint_as_float(e << 23) * a.scale_log2, 0x1p-126f);
                float f[8];
                unpack_bf16x8(x, f);
                uint32_t h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __half2 v = __floats2half2_rn(f[2 * j] * up, f[2 * j + 1] * up);
                    h[j] = *reinterpret_cast<const uint32_t*>(&v);
                }
                // d = 8c .. 8c + 7: two k-steps of lane (r & 7, (c % 8) / 2)
                const int ks = (c / 8) * 2 + (c & 1);
                reinterpret_cast<uint4*>(smem + S::kQ)[((r >> 3) * kKS + ks) * 32 + (r & 7) * 4 + (c % 8) / 2] =
                    make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
        __syncthreads();

        float acc[kDT][kRW][4];
        // mq: the reference of rows 2q, 2q + 1 of each 8 in log2, -inf before the first score; l: sum of p
        constexpr float kSlack = 8.0f;
        float mq[kRW][2], l[kRW][2], qs[kRW][2], r_ref = 0x1p-100f;
        int limit[kRW][2];  // first position that the row does not see
#pragma unroll
        for (int i = 0; i < kRW; ++i) {
#pragma unroll
            for (int j = 0; j < kDT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][i][e] = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = wr * S::kWarpRows + i * 8 + qd * 2 + e;
                mq[i][e] = kNegInf;
                l[i][e] = 0.0f;
                qs[i][e] = qscale[r];
                limit[i][e] = it.len - it.nq + (row0 + r) / a.group + 1;
            }
        }
        const int all_see = it.len - it.nq + row0 / a.group + 1;  // positions below it need no mask
        const uint4* qf = reinterpret_cast<const uint4*>(smem + S::kQ) + wr * kRW * kKS * 32 + lane;

        int stage = 0;
        for (int t = f0 + group; t < f1; t += kG) {
            cp_async_wait<kStages - 2>();
            group_sync();  // the tile is there, and the stage before it is free
            request(t + (kStages - 1) * kG, stage == 0 ? kStages - 1 : stage - 1);
            const uint8_t* kt = ring + stage * S::kStageBytes;
            const uint8_t* vt = kt + kTile * kD;
            const float* sk = reinterpret_cast<const float*>(kt + 2 * kTile * kD);
            const float* sv = sk + kTile;

            // S^T of 2 x 16 tokens: s[x][i] rows are tokens 16x + g, + 8, columns query rows 2q, 2q + 1.
            float s[2][kRW][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int i = 0; i < kRW; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[x][i][e] = 0.0f;
#pragma unroll
            for (int w = 0; w < kD / 64; ++w) {
                uint4 ka[2][2];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        ka[x][y] = *reinterpret_cast<const uint4*>(kt + stage_offset<kD>(x * 16 + y * 8 + og, w * 4 + qd));
#pragma unroll
                for (int z = 0; z < 4; z += 2) {  // 4 codes of a chunk are a k-step
                    uint32_t af[2][2][4];
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t v0 = z == 0 ? ka[x][y].x : ka[x][y].z, v1 = z == 0 ? ka[x][y].y : ka[x][y].w;
                            af[0][x][y] = e4m3x2_lo_to_f16x2(v0);
                            af[0][x][y + 2] = e4m3x2_hi_to_f16x2(v0);
                            af[1][x][y] = e4m3x2_lo_to_f16x2(v1);
                            af[1][x][y + 2] = e4m3x2_hi_to_f16x2(v1);
                        }
                    uint4 b[kRW];
#pragma unroll
                    for (int i = 0; i < kRW; ++i) b[i] = qf[(i * kKS + w * 2 + (z >> 1)) * 32];
#pragma unroll
                    for (int i = 0; i < kRW; ++i) {
                        mma_f16(s[0][i], af[0][0], b[i].x, b[i].y);
                        mma_f16(s[1][i], af[0][1], b[i].x, b[i].y);
                    }
#pragma unroll
                    for (int i = 0; i < kRW; ++i) {
                        mma_f16(s[0][i], af[1][0], b[i].z, b[i].w);
                        mma_f16(s[1][i], af[1][1], b[i].z, b[i].w);
                    }
                }
            }
            // The tile's largest value scale as a power of two (a NaN scale marks a poisoned token).
            const uint32_t rb = __reduce_max_sync(0xffffffffu, scale_exponent(sv[lane]));
            float ks[4], vs[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                ks[x] = sk[x * 8 + og];
                vs[x] = sv[x * 8 + og];
            }
            // Key scales and mask; exponents relative to the rows' references. A tile that every row sees whole needs
            // no mask.
            const bool edge = t * kTile + kTile > all_see;
            bool passed = __uint_as_float(rb) > r_ref;
            auto masked = [&](int i, int x, int e) { return edge && t * kTile + x * 8 + og >= limit[i][e]; };
#pragma unroll
            for (int i = 0; i < kRW; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) s[x >> 1][i][(x & 1) * 2 + e] *= ks[x];
            if (edge) {
#pragma unroll
                for (int i = 0; i < kRW; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (masked(i, x, e)) s[x >> 1][i][(x & 1) * 2 + e] = kNegInf;
            }
#pragma unroll
            for (int i = 0; i < kRW; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float top = fmaxf(fmaxf(s[0][i][e], s[0][i][e + 2]), fmaxf(s[1][i][e], s[1][i][e + 2]));
                    passed = passed || fmaf(top, qs[i][e], -mq[i][e]) > kSlack;
                }
            // A reference moves only when a score passes it by 2^8, so this is rare past the first tiles; without it
            // no maximum is shared between lanes and nothing is rescaled.
            if (__any_sync(0xffffffffu, passed)) {
                const float r_new = fmaxf(__uint_as_float(rb), r_ref);
                const float r_step = r_new == r_ref ? 1.0f : __fdividef(r_ref, r_new);
                r_ref = r_new;
#pragma unroll
                for (int i = 0; i < kRW; ++i) {
                    float beta[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(fmaxf(s[0][i][e], s[0][i][e + 2]), fmaxf(s[1][i][e], s[1][i][e + 2]));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        const float next = fmaf(top, qs[i][e], -mq[i][e]) > kSlack ? top * qs[i][e] : mq[i][e];
                        const float alpha = next == mq[i][e] ? 1.0f : ex2(mq[i][e] - next);
                        mq[i][e] = next;
                        beta[e] = alpha * r_step;
                        l[i][e] *= alpha;
                    }
#pragma unroll
                    for (int j = 0; j < kDT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][i][e] *= beta[e & 1];
                }
            }
            // Weights p * s_v as the B operand, and sums.
            const float r_inv = __fdividef(0x1p6f, r_ref);
#pragma unroll
            for (int x = 0; x < 4; ++x) vs[x] *= r_inv;
            uint32_t wb[2][kRW][2];
            auto weigh = [&](auto masks) {
#pragma unroll
                for (int i = 0; i < kRW; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float p[2], w[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            p[e] = ex2(fmaf(s[x >> 1][i][(x & 1) * 2 + e], qs[i][e], -mq[i][e]));
                            w[e] = p[e] * vs[x];
                            // a masked weight is zero whatever its row's reference and its scale hold
                            if (decltype(masks)::value && masked(i, x, e)) p[e] = w[e] = 0.0f;
                            l[i][e] += p[e];
                        }
                        const __half2 h = __floats2half2_rn(w[0], w[1]);
                        wb[x >> 1][i][x & 1] = movmatrix(*reinterpret_cast<const uint32_t*>(&h));
                    }
            };
            if (edge)
                weigh(std::true_type{});
            else
                weigh(std::false_type{});
            // O^T += V^T W^T. Lane (g, q) reads the tokens of MMA columns 2q, 2q + 1, 2q + 8, 2q + 9 of each 16;
            // its bytes 2j and 2j + 1 are rows g and g + 8 of output tile j.
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                constexpr int kParts = kD == 256 ? 2 : 1, kWords = kD == 64 ? 2 : 4;
#pragma unroll
                for (int h = 0; h < kParts; ++h) {
                    uint32_t vw[4][kWords];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int row = x * 16 + (y >> 1) * 8 + order<kD>(qd * 2 + (y & 1));
                        if constexpr (kD == 64) {
                            const uint2 v = *reinterpret_cast<const uint2*>(vt + stage_offset<kD>(row, g >> 1) + (g & 1) * 8);
                            vw[y][0] = v.x;
                            vw[y][1] = v.y;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4*>(vt + stage_offset<kD>(row, h * 8 + vg));
                            vw[y][0] = v.x;
                            vw[y][1] = v.y;
                            vw[y][2] = v.z;
                            vw[y][3] = v.w;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 2 * kWords; ++j) {
                        const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
                        const uint32_t lo = __byte_perm(vw[0][j >> 1], vw[1][j >> 1], sel);
                        const uint32_t hi = __byte_perm(vw[2][j >> 1], vw[3][j >> 1], sel);
                        const uint32_t va[4] = {e4m3x2_lo_to_f16x2(lo), e4m3x2_hi_to_f16x2(lo), e4m3x2_lo_to_f16x2(hi),
                                                e4m3x2_hi_to_f16x2(hi)};
#pragma unroll
                        for (int i = 0; i < kRW; ++i) mma_f16(acc[h * 8 + j][i], va, wb[x][i][0], wb[x][i][1]);
                    }
                }
            }
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
        cp_async_wait<0>();
        group_sync();

        // The group's result, in place of its ring: o = sum p s_v v and, per row, its maximum (log2) and sum of p.
#pragma unroll
        for (int i = 0; i < kRW; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], 4);
                l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], 8);
                l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], 16);
            }
        const float r_out = r_ref * 0x1p-6f;
        // Column of output tile j's row g (row g + 8 is the next one).
        constexpr int kRun = kD == 64 ? 8 : 16;  // consecutive columns of a lane
        auto column = [&](int j) { return (j / (kRun / 2)) * 128 + vg * kRun + (j % (kRun / 2)) * 2; };
#pragma unroll
        for (int i = 0; i < kRW; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = wr * S::kWarpRows + i * 8 + qd * 2 + e;
                float* o = reinterpret_cast<float*>(ring) + r * S::kOStride;
#pragma unroll
                for (int j = 0; j < kDT; j += 2)
                    *reinterpret_cast<float4*>(o + column(j)) =
                        make_float4(acc[j][i][e] * r_out, acc[j][i][e + 2] * r_out, acc[j + 1][i][e] * r_out,
                                    acc[j + 1][i][e + 2] * r_out);
                if (g == 0) ml[group * kRows + r] = make_float2(mq[i][e], l[i][e]);
            }
        __syncthreads();

        const bool whole = t0 == 0 && t1 == it.tiles;
        const int slot = 2 * blockIdx.x + (it.first > u_begin ? 1 : 0);
        constexpr int kV = kD / 32;  // columns per lane
        for (int r = warp; r < nrows; r += S::kWarps) {
            float mm = kNegInf, sum = 0.0f, o[kV];
#pragma unroll
            for (int j = 0; j < kG; ++j) mm = fmaxf(mm, ml[j * kRows + r].x);
            const float m_use = mm == kNegInf ? 0.0f : mm;
#pragma unroll
            for (int x = 0; x < kV; ++x) o[x] = 0.0f;
#pragma unroll
            for (int j = 0; j < kG; ++j) {
                const float2 t = ml[j * kRows + r];
                const float f = ex2(t.x - m_use);
                sum = fmaf(t.y, f, sum);
                const float* src =
                    reinterpret_cast<const float*>(smem + S::kRing + j * S::kRingBytes) + r * S::kOStride + lane * kV;
#pragma unroll
                for (int x = 0; x < kV; ++x) o[x] = fmaf(src[x], f, o[x]);
            }
            if (whole) {
                write_row<kD>(a, it.q0, it.h, row0 + r, lane, mm, sum, o);
            } else {
                float* po = a.part_o + (static_cast<int64_t>(slot) * kRows + r) * kD + lane * kV;
#pragma unroll
                for (int x = 0; x < kV; x += 2) *reinterpret_cast<float2*>(po + x) = make_float2(o[x], o[x + 1]);
                if (lane == 0)
                    *reinterpret_cast<float2*>(a.part_ml + (static_cast<int64_t>(slot) * kRows + r) * 2) =
                        make_float2(mm, sum);
            }
        }
        if (!whole && t0 == 0 && threadIdx.x == 0) {  // it starts here and goes on in the next CTA
            write_split(a, it, per, slot, row0, nrows);
        }
        if (item_end >= u_end) break;
        // Next item.
        __syncthreads();
        u = item_end;
        Work::next_item(a, it);
    }
}

// Adds the parts of the items that cross CTAs: CTA (c, y) takes some rows of
// the item that starts in CTA c of the first kernel, kSplit of its 8 warps per
// row. Latency is all it is: the item's record is one load, then every lane
// fetches the maximum and sum of one of the warp's parts while the rows of 8 or
// 16 parts are on their way. A long context of few rows has tens of parts, which
// 4 warps a row take in one or two such trips (one token over 131072: 34.0 us with
// 1 warp a row, 30.9 with 4); many rows have enough warps as it is.
constexpr int kJoinWarps = 8;

// With the wide row tiles of the tcgen05 kernel there are thousands of rows of
// a few parts, and more warps per SM (kWide: 4 parts ahead in 64 registers) hide
// more than longer trips do: 512 tokens over 16384 117.5 us in all instead of
// 123.4, 2048 over 4096 131.6 instead of 143.4; with narrow tiles it costs 0.6 us.
template <int kD, int kSplit, bool kWide>
__global__ void __launch_bounds__(kJoinWarps * 32, kWide ? 4 : 1) kv_attention_join_kernel(const __grid_constant__ AttnArgs a, int listed) {
    constexpr int kV = kD / 32, kAhead = kWide ? 4 : 128 / kV / 2, kRows = kJoinWarps / kSplit;
    __shared__ float2 part_ml[kJoinWarps];
    __shared__ float part_o[kSplit > 1 ? kJoinWarps : 1][kSplit > 1 ? kD : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slice = warp % kSplit;
    const int r = blockIdx.y * kRows + warp / kSplit;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    int c = blockIdx.x;
    if (kSplit > 1 && listed) {  // the x-th record that holds an item
        uint32_t held[kMaxAttnGrid / 32];
#pragma unroll
        for (int i = 0; i < kMaxAttnGrid / 32; ++i)
            held[i] = i * 32 + lane < listed ? ld_dep_s32(&a.split[i * 32 + lane].parts) : 0;
        c = -1;
        int before = blockIdx.x;
#pragma unroll
        for (int i = 0; i < kMaxAttnGrid / 32; ++i) {
            const uint32_t bits = __ballot_sync(0xffffffffu, held[i] != 0);
            const uint32_t hit = __ballot_sync(0xffffffffu, held[i] != 0 && __popc(bits & ((1u << lane) - 1)) == before);
            if (hit) c = i * 32 + __ffs(hit) - 1;
            before -= __popc(bits);
        }
        if (c < 0) return;  // (the whole CTA)
    }
    const uint4 s0 = ld_dep_v4(a.split + c), s1 = ld_dep_v4(reinterpret_cast<const uint4*>(a.split + c) + 1);
    const int parts = static_cast<int>(s0.x), second = static_cast<int>(s0.y), nrows = static_cast<int>(s1.y);
    if (parts == 0 || static_cast<int>(blockIdx.y) * kRows >= nrows) return;  // (the whole CTA)
    const int mine_n = r < nrows ? (parts - slice + kSplit - 1) / kSplit : 0;  // parts slice, slice + kSplit, ...
    auto slot_of = [&](int j) {
        const int i = slice + j * kSplit;
        return static_cast<int64_t>(2 * (c + i) + (i == 0 ? second : 0)) * a.rows + r;
    };
    const float2* pml = reinterpret_cast<const float2*>(a.part_ml);
    float mm = kNegInf, sum = 0.0f, o[kV];
#pragma unroll
    for (int x = 0; x < kV; ++x) o[x] = 0.0f;
    for (int base = 0; base < mine_n; base += 32) {  // 32 parts: the lanes hold their maxima and sums
        const int here = min(mine_n - base, 32);
        const float2 mine = lane < here ? __ldcg(pml + slot_of(base + lane)) : make_float2(kNegInf, 0.0f);
        float f = 0.0f;
        for (int i0 = 0; i0 < here; i0 += kAhead) {
            float2 v[kAhead][kV / 2];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (i0 + j >= here) break;
                const float2* src = reinterpret_cast<const float2*>(a.part_o + slot_of(base + i0 + j) * kD) + lane * (kV / 2);
#pragma unroll
                for (int x = 0; x < kV / 2; ++x) v[j][x] = __ldcg(src + x);
            }
            if (i0 == 0) {
                float top = mine.x;
#pragma unroll
                for (int w = 16; w >= 1; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                const float m_new = fmaxf(mm, top), m_use = m_new == kNegInf ? 0.0f : m_new;
                const float back = ex2(mm - m_use);
                f = ex2(mine.x - m_use);
                float add = mine.y * f;
#pragma unroll
                for (int w = 16; w >= 1; w >>= 1) add += __shfl_xor_sync(0xffffffffu, add, w);
                sum = fmaf(sum, back, add);
#pragma unroll
                for (int x = 0; x < kV; ++x) o[x] *= back;
                mm = m_new;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float w = __shfl_sync(0xffffffffu, f, (i0 + j) & 31);
                if (i0 + j < here)
#pragma unroll
                    for (int x = 0; x < kV / 2; ++x) {
                        o[2 * x] = fmaf(v[j][x].x, w, o[2 * x]);
                        o[2 * x + 1] = fmaf(v[j][x].y, w, o[2 * x + 1]);
                    }
            }
        }
    }
    if constexpr (kSplit > 1) {
        if (lane == 0) part_ml[warp] = make_float2(mm, sum);
#pragma unroll
        for (int x = 0; x < kV; ++x) part_o[warp][lane * kV + x] = o[x];
        __syncthreads();
        if (slice != 0) return;
#pragma unroll
        for (int w = 1; w < kSplit; ++w) mm = fmaxf(mm, part_ml[warp + w].x);
        const float use = mm == kNegInf ? 0.0f : mm;
        sum = 0.0f;
#pragma unroll
        for (int x = 0; x < kV; ++x) o[x] = 0.0f;
#pragma unroll
        for (int w = 0; w < kSplit; ++w) {
            const float f = ex2(part_ml[warp + w].x - use);
            sum = fmaf(part_ml[warp + w].y, f, sum);
#pragma unroll
            for (int x = 0; x < kV; ++x) o[x] = fmaf(part_o[warp + w][lane * kV + x], f, o[x]);
        }
    }
    if (r < nrows)
        write_row<kD>(a, static_cast<int>(s0.z), static_cast<int>(s0.w), static_cast<int>(s1.x) + r, lane, mm, sum, o);
}

template <int kD, int kWR, int kRW, int kG, int kCtas>
cudaError_t launch_attention(const AttnArgs& a, int num_sms, int& grid, cudaStream_t stream) {
    using S = Attn<kD, kWR, kRW, kG, kCtas>;
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaGetDevice(&dev);
    auto kernel = kv_attention_kernel<kD, kWR, kRW, kG, kCtas>;
    if (!configured[dev & 63].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
        if (e != cudaSuccess) return e;
        configured[dev & 63].store(true, std::memory_order_relaxed);
    }
    grid = kCtas * num_sms;
    return launch_dependent(kernel, dim3(grid), S::kThreads, S::kBytes, stream, 1, a);
}

// Row tiles: the smallest that holds a sequence's rows, else the largest. The
// registers of a thread go by the CTA's warps (255 up to 8 warps, 168 up to
// 12), and a warp needs 32 accumulators for every 8 rows x 128 columns. From
// kWideRows rows on, head size 128 takes the tcgen05 kernel's row tiles of any
// multiple of 8 up to 128, or 256.
constexpr int kWideRows = 49;
int rows_of(int max_q_len, int group, int head_dim) {
    const int64_t rows = static_cast<int64_t>(max_q_len) * group;
    if (head_dim == 128 && rows >= kWideRows) return rows > 128 ? 256 : static_cast<int>((rows + 7) / 8 * 8);
    const int wide[] = {8, 16, 24, 48, 96, 192}, narrow[] = {8, 16, 32, 64};
    if (head_dim == 256) {
        for (int r : narrow)
            if (rows <= r) return r;
        return 64;
    }
    for (int r : wide)
        if (rows <= r) return r;
    return 192;
}

// Launches the kernel for the row tile; `grid` is its CTAs.
template <int kD>
cudaError_t launch_rows(const AttnArgs& a, int num_sms, int& grid, cudaStream_t stream);

template <>
cudaError_t launch_rows<64>(const AttnArgs& a, int num_sms, int& grid, cudaStream_t stream) {
    switch (a.rows) {
        case 8: return launch_attention<64, 1, 1, 6, 2>(a, num_sms, grid, stream);
        case 16: return launch_attention<64, 1, 2, 6, 2>(a, num_sms, grid, stream);
        case 24: return launch_attention<64, 1, 3, 6, 2>(a, num_sms, grid, stream);
        case 48: return launch_attention<64, 2, 3, 4, 1>(a, num_sms, grid, stream);
        case 96: return launch_attention<64, 4, 3, 2, 1>(a, num_sms, grid, stream);
        default: return launch_attention<64, 8, 3, 1, 1>(a, num_sms, grid, stream);
    }
}

template <>
cudaError_t launch_rows<128>(const AttnArgs& a, int num_sms, int& grid, cudaStream_t stream) {
    switch (a.rows) {
        case 8: return launch_attention<128, 1, 1, 6, 2>(a, num_sms, grid, stream);
        case 16: return launch_attention<128, 1, 2, 6, 2>(a, num_sms, grid, stream);
        case 24: return launch_attention<128, 1, 3, 4, 2>(a, num_sms, grid, stream);
        case 48: return launch_attention<128, 2, 3, 4, 1>(a, num_sms, grid, stream);
        default: grid = num_sms; return launch_attention_tc(a, num_sms, stream);
    }
}

template <>
cudaError_t launch_rows<256>(const AttnArgs& a, int num_sms, int& grid, cudaStream_t stream) {
    switch (a.rows) {
        case 8: return launch_attention<256, 1, 1, 6, 1>(a, num_sms, grid, stream);
        case 16: return launch_attention<256, 2, 1, 4, 1>(a, num_sms, grid, stream);
        case 32: return launch_attention<256, 2, 2, 4, 1>(a, num_sms, grid, stream);
        default: return launch_attention<256, 4, 2, 2, 1>(a, num_sms, grid, stream);
    }
}

template <int kD>
cudaError_t launch_both(const AttnArgs& a, int max_q_len, int num_sms, cudaStream_t stream) {
    if (num_sms > kMaxAttnGrid / 2) num_sms = kMaxAttnGrid / 2;
    int grid = 0;
    const cudaError_t e = launch_rows<kD>(a, num_sms, grid, stream);
    if (e != cudaSuccess) return e;
    const int64_t items = static_cast<int64_t>(a.batch) * a.c.heads * ((static_cast<int64_t>(max_q_len) * a.group + a.rows - 1) / a.rows);
    // 4 warps a row while the items are few, so that each has many parts: (us, 1 and 4 warps) one token over 4096 10.1 and
    // 8.9, over 131072 34.0 and 30.6, 8 over 131072 61.9 and 58.9, one of 12 heads on 1 39.7 and 22.2; but 8 sequences
    // x 8 tokens 28.1 and 31.4. Up to 16 rows a CTA looks at each record, most of which hold no item; with more rows
    // the CTAs, one per item there can be, find theirs in the list, which costs 1 us and saves the empty CTAs 2 to 3.
    const bool many = items * (a.rows <= 16 ? 4 : 8) <= grid, listed = many && a.rows > 16;
    const int rows = many ? kJoinWarps / 4 : kJoinWarps;
    // (a sequence may have more tokens than max_q_len says: room for every row tile that the tokens can make)
    const int64_t most = a.c.heads * ((static_cast<int64_t>(a.tokens) * a.group + static_cast<int64_t>(a.batch) * (a.rows - 1)) / a.rows);
    const dim3 join(listed && most < grid ? static_cast<int>(most) : grid, (a.rows + rows - 1) / rows);
    auto kernel = many               ? kv_attention_join_kernel<kD, 4, false>
                  : a.rows >= kWideRows ? kv_attention_join_kernel<kD, 1, true>
                                     : kv_attention_join_kernel<kD, 1, false>;
    return launch_dependent(kernel, join, kJoinWarps * 32, 0, stream, 1, a, listed ? grid : 0);
}

}  // namespace

size_t kv_attention_workspace(int max_q_len, int group, int head_dim) {
    const size_t rows = rows_of(max_q_len, group, head_dim);
    return kMaxAttnGrid * sizeof(SplitItem) + 2 * static_cast<size_t>(kMaxAttnGrid) * rows * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv_attention(const AttentionProblem& p, int num_sms, cudaStream_t stream) {
    const int rows = rows_of(p.max_q_len, p.group, p.cache.head_dim);
    const size_t slots = 2 * static_cast<size_t>(kMaxAttnGrid) * rows;
    AttnArgs a;
    a.q = static_cast<const uint16_t*>(p.q);
    a.q_stride = p.q_stride;
    a.cu_q = p.cu_q;
    a.kv_lens = p.kv_lens;
    a.table = p.page_table;
    a.table_stride = p.table_stride;
    a.batch = p.batch;
    a.tokens = p.tokens;
    a.group = p.group;
    a.rows = rows;
    void* error = nullptr;
    const cudaError_t found = cudaGetSymbolAddress(&error, g_attn_index_error);
    if (found != cudaSuccess) return found;
    a.index_error = static_cast<unsigned int*>(error);
    a.scale_log2 = p.softmax_scale * 1.4426950408889634f;
    a.c = p.cache;
    a.out = static_cast<uint32_t*>(p.out);
    a.lse = p.lse;
    a.split = static_cast<SplitItem*>(p.workspace);
    a.part_ml = reinterpret_cast<float*>(a.split + kMaxAttnGrid);
    a.part_o = a.part_ml + slots * 2;
    switch (p.cache.head_dim) {
        case 64: return launch_both<64>(a, p.max_q_len, num_sms, stream);
        case 128: return launch_both<128>(a, p.max_q_len, num_sms, stream);
        default: return launch_both<256>(a, p.max_q_len, num_sms, stream);
    }
}

unsigned int read_and_clear_attn_index_error() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_index_error, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_attn_index_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace fp8act
