// Head norms, rotary positions and the cache's quantisation in one pass over
// the fused projection's rows.
//
// A head vector x of D values, of token t at the positions p_0[t], p_1[t], ...:
//   y = x / sqrt(mean x^2 + eps) * (w + offset)      (queries and keys with a weight)
//   (a, b) -> (a cos - b sin, a sin + b cos)          (pairs of the first R columns)
// where pair i turns by p[axis_i][t] * inv_freq_i. Queries are rounded to bf16
// once; keys go to codes and a scale from fp32, values from their bf16 (the
// append's rule), with no copy of either between.
//
// Angles. A turn is 2^64 units: inv_freq / 2 pi becomes a whole number of
// units, and its product with the position wraps to the angle's remainder
// exactly, with no table and no bound on the position. What is lost is the
// frequency's rounding to a unit, or 2^-62 of itself where that is more. The
// remainder, in [-1/2, 1/2) of a turn, is cut to 32 bits and rounded to fp32:
// 2^-25 of itself and 2^-32 of a turn.
//
// Work split. A CTA is one warp: it takes some rounds of a token's heads, a
// round up to kAhead steps of 32 / (D / 8) vectors of one kind, the next
// round's loads in flight. It finds the token's sines and cosines itself, a few
// per lane, and no warp waits for another. A token is cut into as many pieces
// as fill the SMs (its sines are cheap beside a second wait for memory).
#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {
namespace {

__device__ unsigned int g_rope_index_error;

constexpr int kMaxHalf = 128;  // pairs of a head
constexpr int kCtas = 20;      // warps per SM

enum Kind { kQuery, kKey, kValue };

// A frequency in radians a position, as the bits of its fp64 value, in units of 2^-64 turns, modulo a turn: the 53-bit
// significand times 2^66 / 2 pi, shifted.
__device__ __forceinline__ uint64_t units_of(uint64_t bits) {
    constexpr uint64_t kTurn = 0xA2F9836E4E44152Aull;  // 2^66 / 2 pi
    const int exponent = static_cast<int>(bits >> 52 & 0x7FF);
    const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (exponent ? 1ull << 52 : 0);
    const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
    const int down = 2 + 1075 - max(exponent, 1);  // the value is m 2^(exponent - 1075)
    const uint64_t u = down >= 128 ? 0 : down >= 64 ? hi >> (down - 64) : down > 0 ? (hi << (64 - down)) | (lo >> down) : down > -64 ? lo << -down : 0;
    return bits >> 63 ? 0 - u : u;
}

// Lane l of a vector's kLanes holds columns 8l .. 8l + 7.
template <int kLanes, bool kInterleaved, int kAhead>
__global__ void __launch_bounds__(32, kCtas) rope_append_kernel(const __grid_constant__ RopeProblem p, int pieces, int rounds) {
    __shared__ float2 turns[kMaxHalf];  // (cos, sin) * rope_scale
    constexpr int kPer = 32 / kLanes;   // vectors of a step
    const int lane = threadIdx.x, hl = lane % kLanes, mine = lane / kLanes;
    const int64_t t = blockIdx.x / static_cast<unsigned>(pieces);
    const int piece = blockIdx.x % static_cast<unsigned>(pieces);
    const KvCache& c = p.cache;
    const int half = p.rot / 2;
    // Rounds of queries, then of keys, then of values.
    const int rounds_q = (p.q_heads + kAhead * kPer - 1) / (kAhead * kPer), rounds_k = (c.heads + kAhead * kPer - 1) / (kAhead * kPer);
    const int begin = piece * rounds, end = min(begin + rounds, rounds_q + 2 * rounds_k);
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    auto kind_of = [&](int r) { return r < rounds_q ? kQuery : r < rounds_q + rounds_k ? kKey : kValue; };
    auto first_of = [&](int r) {  // the round's first vector among those of its kind
        return (r < rounds_q ? r : r < rounds_q + rounds_k ? r - rounds_q : r - rounds_q - rounds_k) * kAhead * kPer;
    };
    // A round's vectors: this lane's part of the first, 512 bytes apart, and how many of them are the lane's.
    auto row_of = [&](int r) {
        const Kind kind = kind_of(r);
        const uint16_t* row = kind == kQuery ? p.q + t * p.q_stride : kind == kKey ? p.k + t * p.k_stride : p.v + t * p.v_stride;
        return row + static_cast<int64_t>(first_of(r)) * (8 * kLanes) + lane * 8;
    };
    auto left_of = [&](int r) { return r < end ? (kind_of(r) == kQuery ? p.q_heads : c.heads) - first_of(r) - mine : 0; };
    auto load = [&](const uint16_t* row, int left, int i) {
        return i * kPer < left ? ld_dep_stream_v4(row + i * 256) : make_uint4(0, 0, 0, 0);
    };
    uint4 x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = load(row_of(begin), left_of(begin), i);
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint4 wq = p.q_weight ? ld_dep_v4(p.q_weight + hl * 8) : none, wk = p.k_weight ? ld_dep_v4(p.k_weight + hl * 8) : none;
    int64_t slot = *const_cast<const volatile int64_t*>(p.slots + t);
    if (kind_of(begin) != kValue) {
        for (int i = lane; i < half; i += 32) {
            const uint64_t freq = *const_cast<const volatile uint64_t*>(reinterpret_cast<const uint64_t*>(p.inv_freq) + i);
            int axis = p.axis ? ld_dep_s32(p.axis + i) : 0;
            if (axis < 0 || axis >= p.n_axes) {
                atomicOr(&g_rope_index_error, 1u);
                axis = 0;
            }
            const int64_t pos = *const_cast<const volatile int64_t*>(p.positions + static_cast<int64_t>(axis) * p.tokens + t);
            const uint32_t units = static_cast<uint32_t>(static_cast<uint64_t>(pos) * units_of(freq) >> 32);
            const float at = __int2float_rn(static_cast<int>(units)) * 0x1p-31f;  // half turns
            float sn, cs;
            sincospif(at, &sn, &cs);
            turns[i] = make_float2(cs * p.rope_scale, sn * p.rope_scale);
        }
    }
    if (slot >= static_cast<int64_t>(c.num_pages) << c.page_log2) {
        if (lane == 0) atomicOr(&g_rope_index_error, 1u);
        slot = -1;
    }
    const int64_t place = slot < 0 ? 0 : ((slot >> c.page_log2) * c.heads << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
    __syncwarp();

    // The lane's cosines and sines, two columns each: of its 8 columns' pairs, the first half's sines negative, or of its
    // 4 pairs, the first column's.
    const int reach = p.rot / 16;  // lanes of half the rotated columns
    const bool rotated = hl < 2 * reach, second = hl >= reach, all_rotated = p.rot == 8 * kLanes;
    float2 cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cs[i] = sn[i] = make_float2(0.0f, 0.0f);
        if (rotated) {
            if constexpr (kInterleaved) {
                const float2 u = turns[hl * 4 + i];
                cs[i] = make_float2(u.x, u.x);
                sn[i] = make_float2(-u.y, u.y);
            } else {
                const float4 u = *reinterpret_cast<const float4*>(turns + (second ? hl - reach : hl) * 8 + 2 * i);
                cs[i] = make_float2(u.x, u.z);
                sn[i] = second ? make_float2(u.y, u.w) : make_float2(-u.y, -u.w);
            }
        }
    }
    const int partner = rotated ? (second ? lane - reach : lane + reach) : lane;

    // Norm and turn of a vector (a turn is linear, so that the reciprocal root comes last and its sum is not waited for).
    auto turned = [&](float2 (&f)[4], const float2 (&w)[4], bool normed) {
        float r = 1.0f;
        if (normed) {
            float2 sum = __fmul2_rn(f[0], f[0]);
#pragma unroll
            for (int j = 1; j < 4; ++j) sum = __ffma2_rn(f[j], f[j], sum);
            float all = sum.x + sum.y;
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
            asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(fmaf(all, 1.0f / (8 * kLanes), p.eps)));
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = __fmul2_rn(f[j], w[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 other = make_float2(f[j].y, f[j].x);
            if constexpr (!kInterleaved) {
                other.x = __shfl_sync(0xffffffffu, f[j].x, partner);
                other.y = __shfl_sync(0xffffffffu, f[j].y, partner);
            }
            const float2 z = __ffma2_rn(other, sn[j], __fmul2_rn(f[j], cs[j]));
            if (all_rotated || rotated) f[j] = z;
        }
        if (normed) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = __fmul2_rn(f[j], make_float2(r, r));
        }
    };
    auto weight = [&](const uint4& packed, float2 (&w)[4]) {
        unpack_bf16x8(packed, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __fadd2_rn(w[j], make_float2(p.weight_offset, p.weight_offset));
    };
    auto store = [&](float2 (&f)[4], uint32_t top, int h, uint8_t* codes, float* scales) {
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float s = quant_head(f, top);
        if (slot < 0 || h >= c.heads) return;
        const int64_t at = place + (static_cast<int64_t>(h) << c.page_log2);
        reinterpret_cast<uint2*>(codes)[at * kLanes + hl] = pack_e4m3x8(f);
        if (hl == 0) scales[at] = s;
    };

    for (int r = begin; r < end; ++r) {
        const int first = first_of(r), left = left_of(r), left_next = left_of(r + 1);
        const uint16_t* const row_next = row_of(r + 1);
        const Kind kind = kind_of(r);
        // Each step's registers are asked for again as soon as they are read.
        if (kind == kQuery) {
            float2 w[4];
            weight(wq, w);
            uint4* const out = reinterpret_cast<uint4*>(p.q_out) + (t * p.q_heads + first) * kLanes + lane;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                float2 f[4];
                unpack_bf16x8(x[i], f);
                x[i] = load(row_next, left_next, i);
                if (first + i * kPer >= p.q_heads) continue;
                turned(f, w, p.q_weight != nullptr);
                if (i * kPer < left) out[i * 32] = pack_bf16x8(f);
            }
        } else {
            float2 w[4];
            weight(wk, w);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                float2 f[4];
                unpack_bf16x8(x[i], f);
                uint32_t top = top_bits(x[i]) << 16;
                x[i] = load(row_next, left_next, i);
                if (first + i * kPer >= c.heads) continue;
                if (kind == kKey) {
                    turned(f, w, p.k_weight != nullptr);
                    top = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        top = max(top, max(__float_as_uint(f[j].x) & 0x7FFFFFFFu, __float_as_uint(f[j].y) & 0x7FFFFFFFu));
                    store(f, top, first + i * kPer + mine, c.k, c.k_scale);
                } else {
                    store(f, top, first + i * kPer + mine, c.v, c.v_scale);
                }
            }
        }
    }
}

template <int kLanes, int kAhead>
cudaError_t launch(const RopeProblem& p, int num_sms, cudaStream_t stream) {
    constexpr int kRound = kAhead * 32 / kLanes;
    const int64_t whole = (static_cast<int64_t>(p.q_heads) + kRound - 1) / kRound + 2 * ((static_cast<int64_t>(p.cache.heads) + kRound - 1) / kRound);
    // Pieces of a token: enough for every warp that fits the SMs at once.
    const int64_t room = (static_cast<int64_t>(num_sms) * kCtas + p.tokens - 1) / p.tokens;
    const int64_t rounds = (whole + room - 1) / room;
    const int64_t pieces = (whole + rounds - 1) / rounds;
    if (p.tokens * pieces > INT32_MAX) return cudaErrorInvalidConfiguration;
    auto kernel = p.interleaved ? rope_append_kernel<kLanes, true, kAhead> : rope_append_kernel<kLanes, false, kAhead>;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(p.tokens * pieces)), 32, 0, stream, 1, p, static_cast<int>(pieces),
                            static_cast<int>(rounds));
}

// A step at a time while that gives no more warps than fit: a token's heads are then all on their way at once.
template <int kLanes>
cudaError_t launch_ahead(const RopeProblem& p, int num_sms, cudaStream_t stream) {
    const int64_t vectors = (p.q_heads + 2 * static_cast<int64_t>(p.cache.heads)) * p.tokens;
    return vectors * kLanes / 32 <= static_cast<int64_t>(num_sms) * kCtas ? launch<kLanes, 1>(p, num_sms, stream)
                                                                          : launch<kLanes, 4>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeProblem& p, int num_sms, cudaStream_t stream) {
    switch (p.cache.head_dim) {
        case 64: return launch_ahead<8>(p, num_sms, stream);
        case 128: return launch_ahead<16>(p, num_sms, stream);
        default: return launch_ahead<32>(p, num_sms, stream);
    }
}

unsigned int read_and_clear_rope_index_error() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_rope_index_error, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_rope_index_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace fp8act
