// Attention of new tokens over the paged E4M3 cache (decode, draft verify,
// prompt chunks), grouped query heads, causal from the end of the sequence.
//
// For a sequence with L cached tokens, n of them new, new token i sees the
// positions <= L - n + i. With codes k, v and one scale per token and head,
//   S[r, j] = softmax_scale * s_k[j] * (q_r . k_j),   P = softmax(S),
//   O[r]    = sum_j P[r, j] s_v[j] v_j.
//
// Arithmetic. Codes widen exactly to f16 (cvt.rn.f16x2.e4m3x2), so both
// products run as f16 MMAs with fp32 accumulation. A query row is scaled by a
// power of two so that its largest value is in [1, 2): bf16 then fits f16
// exactly down to 2^-17 of the largest value, and below that to within 2^-25
// of it. The value product's weights p * s_v are rounded to f16 (11 bits; bf16
// would give 8) after scaling by 2^14 / R, R the power of two below the
// largest s_v so far: they keep full precision down to 2^-28 of the largest
// weight. Maxima, sums, and both accumulations are fp32.
//
// Work split. A row tile is kMT * 16 rows of (new token, query head of one KV
// head); a unit is one row tile x 64 cached tokens. The units of all
// sequences, KV heads and row tiles form one list, which the CTAs of a fixed
// grid share evenly: no host knowledge of the lengths is needed and a ragged
// batch balances itself. A CTA whose range ends inside a (sequence, head, row
// tile) item leaves an fp32 partial in the workspace; the last CTA to arrive
// at the item adds the parts in a fixed order, so results do not depend on
// timing.
#include <cuda_fp16.h>

#include <atomic>

#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {
namespace {

__device__ unsigned int g_attn_index_error;

constexpr int kTile = 64;     // cached tokens per unit
constexpr int kThreads = 128;
constexpr float kNegInf = -__builtin_huge_valf();

struct AttnArgs {
    const uint16_t* q;
    int64_t q_stride;
    const int* cu_q;
    const int* kv_lens;
    const int* table;
    int64_t table_stride;
    int batch, tokens, group;
    float scale_log2;
    KvCache c;
    uint32_t* out;   // bf16 [tokens, heads * group, D]
    float* lse;      // [tokens, heads * group] or null
    float* part_o;   // [2 * grid][rows][D]
    float* part_ml;  // [2 * grid][rows][2]
    int* counters;   // [grid]
    int min_units;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

// Two E4M3 codes (low 16 bits of `codes`) to f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(r) : "r"(codes));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(r) : "r"(codes));
    return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldmatrix_x4(uint32_t addr) {
    uint4 v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Byte offset of 16-byte chunk c of cached token `row` in a stage. The chunk
// index is permuted by the token so that both the key fragments (8 tokens x 4
// chunks) and the value fragments (tokens 2q + const, the same chunk) read
// distinct banks.
template <int kD>
__device__ __forceinline__ uint32_t stage_offset(int row, int c) {
    const int swz = kD == 64 ? (row >> 1) & 3 : ((row & 1) << 2) ^ (((row >> 1) & 3) << 1);
    return row * kD + ((c ^ swz) << 4);
}

template <int kD, int kMT>
struct AttnSmem {
    static constexpr int kRows = kMT * 16;
    static constexpr int kStages = kD == 256 ? 2 : 3;
    static constexpr int kStageBytes = 2 * kTile * kD + 2 * kTile * 4;  // keys, values, key scales, value scales
    static constexpr int kPStride = kTile + 8;                          // halves; 144 bytes: ldmatrix without conflicts
    static constexpr int kQ = kStages * kStageBytes;
    static constexpr int kP = kQ + kRows * kD * 2;
    static constexpr int kRed = kP + kRows * kPStride * 2;
    static constexpr int kQScale = kRed + 4 * kRows * 4;
    static constexpr int kBytes = kQScale + kRows * 4;
};

// One (sequence, KV head, row tile) and where it lies in the unit list.
struct Item {
    int b, h, rt;      // sequence, KV head, row tile
    int nq, q0, len;   // new tokens, first one's row in q, cached tokens
    int rts, tiles;    // row tiles and units per row tile of this sequence
    int64_t first;     // index of the item's first unit
};

__device__ __forceinline__ void load_sequence(const AttnArgs& a, int rows, int b, Item& it) {
    const int q0 = ld_dep_s32(a.cu_q + b), q1 = ld_dep_s32(a.cu_q + b + 1);
    int len = ld_dep_s32(a.kv_lens + b);
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.tokens;
    it.q0 = q0;
    it.nq = ok ? q1 - q0 : 0;
    const int64_t most = a.table_stride << a.c.page_log2;
    if (!ok || len < 0 || len > most) {
        atomicOr(&g_attn_index_error, 1u);
        len = len < 0 ? 0 : static_cast<int>(len > most ? most : len);
    }
    it.len = len;
    it.rts = (it.nq * a.group + rows - 1) / rows;
    it.tiles = (len + kTile - 1) / kTile;
    if (it.tiles == 0) it.tiles = 1;  // an empty sequence still writes its rows
}

template <int kD, int kMT>
__global__ void __launch_bounds__(kThreads) kv_attention_kernel(const __grid_constant__ AttnArgs a) {
    using S = AttnSmem<kD, kMT>;
    constexpr int kRows = S::kRows;
    constexpr int kKS = kD / 16;   // k-steps of the score product
    constexpr int kNT = kD / 32;   // 8-column tiles of the output per warp
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_total;
    __shared__ int s_b;
    __shared__ int64_t s_first;
    __shared__ int s_last;
    const uint32_t sbase = ptx::smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, qd = lane & 3;
    float* red = reinterpret_cast<float*>(smem + S::kRed);
    float* qscale = reinterpret_cast<float*>(smem + S::kQScale);

    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    // Total units, and the sequence that holds this CTA's first one.
    if (warp == 0) {
        int64_t total = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
            int64_t u = 0;
            if (b0 + lane < a.batch) {
                Item it;
                load_sequence(a, kRows, b0 + lane, it);
                u = static_cast<int64_t>(a.c.heads) * it.rts * it.tiles;
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
            total += u;
        }
        int64_t per = (total + gridDim.x - 1) / gridDim.x;
        if (per < a.min_units) per = a.min_units;
        const int64_t u0 = per * blockIdx.x;
        int64_t base = 0;
        if (lane == 0) s_b = a.batch;
        for (int b0 = 0; b0 < a.batch && u0 < total; b0 += 32) {
            int64_t u = 0;
            if (b0 + lane < a.batch) {
                Item it;
                load_sequence(a, kRows, b0 + lane, it);
                u = static_cast<int64_t>(a.c.heads) * it.rts * it.tiles;
            }
            int64_t incl = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const int64_t lo = base + incl - u;
            if (u0 >= lo && u0 < lo + u) {
                s_b = b0 + lane;
                s_first = lo;
            }
            base = __shfl_sync(0xffffffffu, base + incl, 31);
            if (base > u0) break;
        }
        if (lane == 0) s_total = total;
    }
    __syncthreads();
    const int64_t total = s_total;
    int64_t per = (total + gridDim.x - 1) / gridDim.x;
    if (per < a.min_units) per = a.min_units;
    int64_t u = per * blockIdx.x;
    const int64_t u_end = u + per < total ? u + per : total;
    if (u >= u_end) return;
    const int64_t u_begin = u;

    Item it;
    it.b = s_b;
    load_sequence(a, kRows, it.b, it);
    {
        const int64_t rel = (u - s_first) / it.tiles;
        it.h = static_cast<int>(rel / it.rts);
        it.rt = static_cast<int>(rel % it.rts);
        it.first = s_first + rel * it.tiles;
    }

    while (true) {
        const int t0 = static_cast<int>(u - it.first);
        const int64_t item_end = it.first + it.tiles;
        const int t1 = static_cast<int>((item_end < u_end ? item_end : u_end) - it.first);
        const int rows_total = it.nq * a.group;
        const int row0 = it.rt * kRows;
        const int nrows = rows_total - row0 < kRows ? rows_total - row0 : kRows;
        // Tokens that some row of the tile sees; the units past them are empty.
        const int last_q = (row0 + nrows - 1) / a.group;
        int seen = it.len - it.nq + last_q + 1;
        if (seen < 0) seen = 0;
        const int t_stop = (seen + kTile - 1) / kTile < t1 ? (seen + kTile - 1) / kTile : t1;

        // Queries: power-of-two scaled f16 in fragment order.
        __syncthreads();
        {
            constexpr int kLanes = kD / 8;
            const int c = tid % kLanes;
            for (int r = tid / kLanes; r < kRows; r += kThreads / kLanes) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (r < nrows) {
                    const int qi = (row0 + r) / a.group, hg = (row0 + r) - qi * a.group;
                    x = ld_dep_v4(a.q + (it.q0 + qi) * a.q_stride + (it.h * a.group + hg) * kD + c * 8);
                }
                uint32_t top = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                        __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
                top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
                for (int o = (kLanes < 32 ? kLanes : 32) / 2; o >= 1; o >>= 1)
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                uint32_t e = top >> 7;
                if (e > 253) e = 253;
                const float up = __uint_as_float((254 - e) << 23);  // 2^(127 - e)
                if (c == 0) qscale[r] = __uint_as_float(e << 23) * a.scale_log2;
                float f[8];
                unpack_bf16x8(x, f);
                const int i = c / 8, qq = (c % 8) / 2, w0 = (c & 1) * 2;
                const int l = (r & 7) * 4 + qq, reg = (r & 15) >= 8 ? 1 : 0;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const __half2 hh = __floats2half2_rn(f[2 * p] * up, f[2 * p + 1] * up);
                    const int ks = i * 4 + w0 + (p >> 1);
                    const int at = (((r >> 4) * kKS + ks) * 32 + l) * 4 + reg + (p & 1) * 2;
                    reinterpret_cast<uint32_t*>(smem + S::kQ)[at] = *reinterpret_cast<const uint32_t*>(&hh);
                }
            }
        }
        const int64_t page_bytes = static_cast<int64_t>(kD) << a.c.page_log2;
        const int* table = a.table + it.b * a.table_stride;
        // Pages of the next tile to request: one per 16 cached tokens.
        int page[4];
        auto look_up = [&](int t) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int pos = t * kTile + j * 16;
                page[j] = -1;
                if (t < t_stop && pos < it.len) {
                    const int p = ld_dep_s32(table + (pos >> a.c.page_log2));
                    if (p >= 0 && p < a.c.num_pages)
                        page[j] = p;
                    else if (tid == 0)
                        atomicOr(&g_attn_index_error, 1u);
                }
            }
        };
        auto request = [&](int t, int stage) {
            if (t < t_stop) {
                const uint32_t dst = sbase + stage * S::kStageBytes;
                constexpr int kC = kD / 16;
                const int c = tid % kC;
#pragma unroll
                for (int i = 0; i < kTile * kC / kThreads; ++i) {
                    const int row = tid / kC + i * (kThreads / kC);
                    const int pos = t * kTile + row;
                    const int p = kThreads / kC > 16 ? (tid / kC < 16 ? page[2 * i] : page[2 * i + 1]) : page[i * (kThreads / kC) / 16];
                    const bool in = p >= 0 && pos < it.len;
                    const int64_t at = in ? (static_cast<int64_t>(p) * a.c.heads + it.h) * page_bytes +
                                                (pos & ((1 << a.c.page_log2) - 1)) * kD + c * 16
                                          : 0;
                    const uint32_t off = stage_offset<kD>(row, c);
                    cp_async16(dst + off, a.c.k + at, in);
                    cp_async16(dst + kTile * kD + off, a.c.v + at, in);
                }
                const int row = tid & 63, pos = t * kTile + row;
                const int p = row < 32 ? (row < 16 ? page[0] : page[1]) : (row < 48 ? page[2] : page[3]);
                const bool in = p >= 0 && pos < it.len;
                const int64_t at = in ? ((static_cast<int64_t>(p) * a.c.heads + it.h) << a.c.page_log2) +
                                            (pos & ((1 << a.c.page_log2) - 1))
                                      : 0;
                cp_async4(dst + 2 * kTile * kD + tid * 4, (tid < 64 ? a.c.k_scale : a.c.v_scale) + at, in);
            }
            cp_async_commit();
        };

        float acc[kMT][kNT][4];
        float m[kMT][2], l[kMT][2], r_ref = 0x1p-100f;
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
#pragma unroll
            for (int j = 0; j < kNT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
            m[i][0] = m[i][1] = kNegInf;
            l[i][0] = l[i][1] = 0.0f;
        }
        int limit[kMT][2];  // first position that the row does not see
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = row0 + i * 16 + g + e * 8;
                limit[i][e] = it.len - it.nq + r / a.group + 1;
            }

#pragma unroll
        for (int s = 0; s < S::kStages - 1; ++s) {
            look_up(t0 + s);
            request(t0 + s, s);
        }
        look_up(t0 + S::kStages - 1);
        int stage = 0;
        for (int t = t0; t < t_stop; ++t) {
            cp_async_wait<S::kStages - 2>();
            __syncthreads();
            {
                const int next = stage + S::kStages - 1;
                request(t + S::kStages - 1, next >= S::kStages ? next - S::kStages : next);
                look_up(t + S::kStages);
            }
            const uint8_t* kt = smem + stage * S::kStageBytes;
            const uint8_t* vt = kt + kTile * kD;
            const float* sk = reinterpret_cast<const float*>(kt + 2 * kTile * kD);
            const float* sv = sk + kTile;

            // Scores of this warp's 16 tokens.
            float s[kMT][2][4];
#pragma unroll
            for (int i = 0; i < kMT; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][j][e] = 0.0f;
#pragma unroll
            for (int i = 0; i < kD / 64; ++i) {
                uint4 kw[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    kw[j] = *reinterpret_cast<const uint4*>(kt + stage_offset<kD>(warp * 16 + j * 8 + g, i * 4 + qd));
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t b[2][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t v = w == 0 ? kw[j].x : w == 1 ? kw[j].y : w == 2 ? kw[j].z : kw[j].w;
                        b[j][0] = e4m3x2_to_f16x2(v);
                        b[j][1] = e4m3x2_hi_to_f16x2(v);
                    }
#pragma unroll
                    for (int mt = 0; mt < kMT; ++mt) {
                        const uint4 qa = reinterpret_cast<const uint4*>(smem + S::kQ)[(mt * kKS + i * 4 + w) * 32 + lane];
                        mma_f16(s[mt][0], qa, b[0][0], b[0][1]);
                        mma_f16(s[mt][1], qa, b[1][0], b[1][1]);
                    }
                }
            }
            // Scale, mask, and the tile's maximum per row.
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = warp * 16 + j * 8 + qd * 2;
                const float2 ks = *reinterpret_cast<const float2*>(sk + col);
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float qs = qscale[mt * 16 + g + (e >> 1) * 8];
                        const float v = s[mt][j][e] * ((e & 1) ? ks.y : ks.x) * qs;
                        s[mt][j][e] = t * kTile + col + (e & 1) < limit[mt][e >> 1] ? v : kNegInf;
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(fmaxf(s[mt][0][2 * e], s[mt][0][2 * e + 1]), fmaxf(s[mt][1][2 * e], s[mt][1][2 * e + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    if (qd == 0) red[warp * kRows + mt * 16 + g + e * 8] = x;
                }
            // The largest value scale of the tile, as a power of two.
            float r_new = fmaxf(sv[lane], sv[lane + 32]);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) r_new = fmaxf(r_new, __shfl_xor_sync(0xffffffffu, r_new, o));
            r_new = fmaxf(__uint_as_float(__float_as_uint(r_new) & 0x7F800000u), r_ref);
            const float r_inv = 0x1p14f / r_new;
            const float r_step = r_ref / r_new;
            r_ref = r_new;
            __syncthreads();
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = mt * 16 + g + e * 8;
                    const float x = fmaxf(fmaxf(red[r], red[kRows + r]), fmaxf(red[2 * kRows + r], red[3 * kRows + r]));
                    const float m_new = fmaxf(m[mt][e], x);
                    const float m_use = m_new == kNegInf ? 0.0f : m_new;
                    const float alpha = ex2(m[mt][e] - m_use);
                    m[mt][e] = m_new;
                    const float beta = alpha * r_step;
#pragma unroll
                    for (int j = 0; j < kNT; ++j) {
                        acc[mt][j][2 * e] *= beta;
                        acc[mt][j][2 * e + 1] *= beta;
                    }
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int col = warp * 16 + j * 8 + qd * 2;
                        const float2 vs = *reinterpret_cast<const float2*>(sv + col);
                        const float s0 = s[mt][j][2 * e], s1 = s[mt][j][2 * e + 1];
                        const float p0 = ex2(s0 - m_use), p1 = ex2(s1 - m_use);
                        sum += p0 + p1;
                        // a masked weight is zero whatever its scale holds
                        const __half2 w = __floats2half2_rn(s0 == kNegInf ? 0.0f : p0 * (vs.x * r_inv),
                                                            s1 == kNegInf ? 0.0f : p1 * (vs.y * r_inv));
                        *reinterpret_cast<__half2*>(smem + S::kP + (r * S::kPStride + col) * 2) = w;
                    }
                    l[mt][e] = l[mt][e] * alpha + sum;
                }
            __syncthreads();
            // Output columns [warp * D/4, ...) += weights x values.
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks) {
                uint32_t vw[4][kNT / 4 ? kNT / 4 : 1];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = ks * 16 + qd * 2 + (x & 1) + (x >> 1) * 8;
                    const int d = warp * (kD / 4) + g * kNT;
                    const uint8_t* p = vt + stage_offset<kD>(row, d >> 4) + (d & 15);
                    if constexpr (kNT == 2) {
                        vw[x][0] = *reinterpret_cast<const uint16_t*>(p);
                    } else if constexpr (kNT == 4) {
                        vw[x][0] = *reinterpret_cast<const uint32_t*>(p);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(p);
                        vw[x][0] = v.x;
                        vw[x][1] = v.y;
                    }
                }
                uint32_t b[kNT][2];
#pragma unroll
                for (int n = 0; n < kNT; n += 2) {
                    const int wi = n / 4;
                    const uint32_t sel = (n & 2) ? 0x7362u : 0x5140u;
                    const uint32_t lo = __byte_perm(vw[0][wi], vw[1][wi], sel);
                    const uint32_t hi = __byte_perm(vw[2][wi], vw[3][wi], sel);
                    b[n][0] = e4m3x2_to_f16x2(lo);
                    b[n][1] = e4m3x2_to_f16x2(hi);
                    b[n + 1][0] = e4m3x2_hi_to_f16x2(lo);
                    b[n + 1][1] = e4m3x2_hi_to_f16x2(hi);
                }
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
                    const uint4 pa = ldmatrix_x4(sbase + S::kP +
                                                 ((mt * 16 + (lane & 15)) * S::kPStride + ks * 16 + (lane >> 4) * 8) * 2);
#pragma unroll
                    for (int n = 0; n < kNT; ++n) mma_f16(acc[mt][n], pa, b[n][0], b[n][1]);
                }
            }
            stage = stage + 1 == S::kStages ? 0 : stage + 1;
        }
        cp_async_wait<0>();
        // Row sums over the four warps' tokens.
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = l[mt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (qd == 0) red[warp * kRows + mt * 16 + g + e * 8] = x;
            }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == it.tiles;
        const float r_out = r_ref * 0x1p-14f;
        const int slot = 2 * blockIdx.x + (it.first > u_begin ? 1 : 0);
        const int hq = a.c.heads * a.group;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = mt * 16 + g + e * 8;
                if (r >= nrows) continue;
                const float sum = (red[r] + red[kRows + r]) + (red[2 * kRows + r] + red[3 * kRows + r]);
                if (whole) {
                    const int qi = (row0 + r) / a.group, hg = (row0 + r) - qi * a.group;
                    const int64_t orow = static_cast<int64_t>(it.q0 + qi) * hq + it.h * a.group + hg;
                    const float f = sum == 0.0f ? 0.0f : r_out / sum;
#pragma unroll
                    for (int n = 0; n < kNT; n += 2) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int d = warp * (kD / 4) + (2 * qd + x) * kNT + n;
                            a.out[(orow * kD + d) >> 1] =
                                pack_bf16x2(acc[mt][n][2 * e + x] * f, acc[mt][n + 1][2 * e + x] * f);
                        }
                    }
                    if (a.lse && warp == 0 && qd == 0)
                        a.lse[orow] = sum == 0.0f ? kNegInf : (m[mt][e] + log2f(sum)) * 0.6931471805599453f;
                } else {
                    float* po = a.part_o + (static_cast<int64_t>(slot) * kRows + r) * kD;
#pragma unroll
                    for (int n = 0; n < kNT; n += 2)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            *reinterpret_cast<float2*>(po + warp * (kD / 4) + (2 * qd + x) * kNT + n) =
                                make_float2(acc[mt][n][2 * e + x] * r_out, acc[mt][n + 1][2 * e + x] * r_out);
                    if (warp == 0 && qd == 0)
                        *reinterpret_cast<float2*>(a.part_ml + (static_cast<int64_t>(slot) * kRows + r) * 2) =
                            make_float2(m[mt][e], sum);
                }
            }
        if (!whole) {
            // The last CTA to arrive at the item joins its parts, in unit order.
            const int c0 = static_cast<int>(it.first / per), c1 = static_cast<int>((item_end - 1) / per);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const int n = atomicAdd(a.counters + c0, 1);
                s_last = n == c1 - c0;
                if (s_last) a.counters[c0] = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                constexpr int kV = kD / 32;  // columns per lane
                for (int r = warp; r < nrows; r += kThreads / 32) {
                    float mm = kNegInf, sum = 0.0f, o[kV];
#pragma unroll
                    for (int x = 0; x < kV; ++x) o[x] = 0.0f;
                    for (int c = c0; c <= c1; ++c) {
                        const int64_t sl = 2 * c + (c == c0 && it.first > per * c ? 1 : 0);
                        const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + sl * kRows + r);
                        const float m_new = fmaxf(mm, ml.x);
                        const float m_use = m_new == kNegInf ? 0.0f : m_new;
                        const float f0 = ex2(mm - m_use), f1 = ex2(ml.x - m_use);
                        mm = m_new;
                        sum = sum * f0 + ml.y * f1;
                        const float* po = a.part_o + (sl * kRows + r) * kD + lane * kV;
#pragma unroll
                        for (int x = 0; x < kV; x += 2) {
                            const float2 v = __ldcg(reinterpret_cast<const float2*>(po + x));
                            o[x] = o[x] * f0 + v.x * f1;
                            o[x + 1] = o[x + 1] * f0 + v.y * f1;
                        }
                    }
                    const int qi = (row0 + r) / a.group, hg = (row0 + r) - qi * a.group;
                    const int64_t orow = static_cast<int64_t>(it.q0 + qi) * hq + it.h * a.group + hg;
                    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                    for (int x = 0; x < kV; x += 2)
                        a.out[(orow * kD + lane * kV + x) >> 1] = pack_bf16x2(o[x] * f, o[x + 1] * f);
                    if (a.lse && lane == 0) a.lse[orow] = sum == 0.0f ? kNegInf : (mm + log2f(sum)) * 0.6931471805599453f;
                }
            }
        }
        if (item_end >= u_end) break;
        // Next item.
        u = item_end;
        it.first = item_end;
        if (++it.rt == it.rts) {
            it.rt = 0;
            if (++it.h == a.c.heads) {
                it.h = 0;
                do load_sequence(a, kRows, ++it.b, it);
                while (it.rts == 0);
            }
        }
    }
}

constexpr int kMaxGrid = 152 * 4;

template <int kD, int kMT>
cudaError_t launch_attention(const AttnArgs& a, int num_sms, cudaStream_t stream) {
    using S = AttnSmem<kD, kMT>;
    static std::atomic<int> per_sm[64];
    int dev = 0;
    cudaGetDevice(&dev);
    int v = per_sm[dev & 63].load(std::memory_order_relaxed);
    if (v == 0) {
        cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<kD, kMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             S::kBytes);
        if (e != cudaSuccess) return e;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&v, kv_attention_kernel<kD, kMT>, kThreads, S::kBytes);
        if (e != cudaSuccess) return e;
        if (v < 1) v = 1;
        per_sm[dev & 63].store(v, std::memory_order_relaxed);
    }
    int grid = num_sms * v;
    if (grid > kMaxGrid) grid = kMaxGrid;
    return launch_dependent(kv_attention_kernel<kD, kMT>, dim3(grid), kThreads, S::kBytes, stream, 1, a);
}

template <int kD>
cudaError_t launch_attention_d(const AttnArgs& a, int mt, int num_sms, cudaStream_t stream) {
    switch (mt) {
        case 1: return launch_attention<kD, 1>(a, num_sms, stream);
        case 2: return launch_attention<kD, 2>(a, num_sms, stream);
        case 3: return launch_attention<kD, 3>(a, num_sms, stream);
        default: return launch_attention<kD, 4>(a, num_sms, stream);
    }
}

int row_tiles_of(int max_q_len, int group) {
    const int64_t rows = static_cast<int64_t>(max_q_len) * group;
    return rows > 48 ? 4 : rows > 32 ? 3 : rows > 16 ? 2 : 1;
}

}  // namespace

size_t kv_attention_workspace(int max_q_len, int group, int head_dim) {
    const size_t rows = 16 * static_cast<size_t>(row_tiles_of(max_q_len, group));
    return kMaxGrid * 16 + 2 * static_cast<size_t>(kMaxGrid) * rows * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_kv_attention(const AttentionProblem& p, int num_sms, cudaStream_t stream) {
    const int mt = row_tiles_of(p.max_q_len, p.group);
    const size_t slots = 2 * static_cast<size_t>(kMaxGrid) * 16 * mt;
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
    a.scale_log2 = p.softmax_scale * 1.4426950408889634f;
    a.c = p.cache;
    a.out = static_cast<uint32_t*>(p.out);
    a.lse = p.lse;
    a.counters = static_cast<int*>(p.workspace);
    a.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(p.workspace) + kMaxGrid * 16);
    a.part_o = a.part_ml + slots * 2;
    a.min_units = 4;
    switch (p.cache.head_dim) {
        case 64: return launch_attention_d<64>(a, mt, num_sms, stream);
        case 128: return launch_attention_d<128>(a, mt, num_sms, stream);
        default: return launch_attention_d<256>(a, mt, num_sms, stream);
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
