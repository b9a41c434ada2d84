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
// frequency's rounding to a unit, or 2^-62 of itself where that is more, and what
// is cut off the remainder, in [-1/2, 1/2) of a turn, behind 32 bits.
//
// Work split. A lane holds two chunks of 8 columns of a vector, those whose
// columns turn together, so that a turn needs no other lane; D / 16 lanes hold
// the vector, and a warp has 512 / D heads of one kind (with fewer heads than that
// in all, those of several tokens). It keeps them: a CTA's
// warps go through tokens, each with its heads, their weights in registers and the
// loads of the next two vectors and their slot in flight, and the CTA finds the
// next tokens' sines and cosines, a pair a thread, while it works on the present
// ones. Two vectors a lane go through each step together: a query's of two tokens,
// or a key and a value of one, since a warp with two keys kept the others waiting.
// More heads than a CTA's warps hold are other CTAs'.
//
// What bounds it (4096 tokens x 32 heads of 128: 15.1 us, 4.2 TB/s of the least
// traffic): the chains of a round of two tokens, 3200 clocks with 4 warps a
// scheduler to hide them (norm and turn 950, a key and a value to codes 1250,
// unpacking and the next loads 500). One vector after the other, the slot read
// when it is needed and the keys in warps of their own took 19.6 us, a warp per
// token that finds its own sines 17.9, with one chunk a lane and a vector's halves
// exchanged 21.0; the next rows brought to L2 ahead change nothing. One token
// takes 2.5 us, a trip to memory and one to the slots.
#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {
namespace {

__device__ unsigned int g_rope_index_error;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCtas = 2;       // per SM

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

// Sixteen columns of a vector: two chunks of 8.
struct Half {
    float2 a[4], b[4];
};
__device__ __forceinline__ void unpack(const uint4 (&x)[2], Half& f) {
    unpack_bf16x8(x[0], f.a);
    unpack_bf16x8(x[1], f.b);
}

// The largest magnitude of `most` and the two of `f`; NaN if one is.
__device__ __forceinline__ float largest(float most, const float2& f) {
    asm("{\n.reg .f32 a, b;\nabs.f32 a, %1;\nabs.f32 b, %2;\nmax.NaN.f32 %0, %0, a;\nmax.NaN.f32 %0, %0, b;\n}" : "+f"(most) : "f"(f.x), "f"(f.y));
    return most;
}

// kLanes = D / 16 lanes hold a vector.
template <int kLanes, bool kInterleaved, int kIt, int kTps>
__global__ void __launch_bounds__(kThreads, kCtas) rope_append_kernel(const __grid_constant__ RopeProblem p) {
    constexpr int kD = 16 * kLanes;
    constexpr int kHps = 32 / kLanes / kTps;                // heads of a step, of each of kTps tokens
    constexpr int kTile = kIt * kTps;                       // tokens of a tile
    constexpr int kPairs = (kD / 2 * kTile + 95) / 96;      // pairs of a thread, at most (a CTA has at least 3 warps)
    __shared__ __align__(16) float2 turns[2][kTile][kD / 2];  // (cos, sin) * rope_scale
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hl = lane % kLanes, sub = lane / kLanes / kHps;
    const KvCache& c = p.cache;
    const int half = p.rot / 2, tiles = (p.tokens + kTile - 1) / kTile;
    // Steps of queries, then those of keys and of values.
    const int steps_q = (p.q_heads + kHps - 1) / kHps, steps_k = (c.heads + kHps - 1) / kHps;
    const int s = blockIdx.y * (blockDim.x >> 5) + warp;
    // This warp's vectors of a tile: the same heads of its kIt tokens, or, so that no warp has keys alone, which take
    // longest, the keys and the values of one of its two.
    constexpr bool kBoth = kIt == 2;
    const bool query = s < steps_q;
    const int kv_step = s - steps_q, of = kBoth ? kv_step % 2 : kv_step / steps_k;  // the token; keys, values (or neither)
    auto kind_of = [&](int i) { return query ? kQuery : (kBoth ? i : of) == 0 ? kKey : kValue; };
    auto offset_of = [&](int i) { return kBoth && !query ? of : i * kTps + sub; };  // of the token in the tile
    const int heads = query ? p.q_heads : c.heads;
    const int h = (query ? s : kBoth ? kv_step / 2 : kv_step - of * steps_k) * kHps + lane / kLanes % kHps;
    const bool mine = h < heads && (kBoth || of < 2);  // (past the values' heads: an idle warp)
    const uint16_t* const weight = query ? p.q_weight : kind_of(0) == kKey ? p.k_weight : nullptr;
    const bool normed = weight != nullptr;
    // The lane's chunks: columns i and i + R / 2 turn together (or, interleaved, neighbours); what does not turn is shared
    // out after that.
    const int reach = p.rot / 16;  // chunks of half the rotated columns
    const bool rotated = hl < reach;
    const int chunk_a = kInterleaved || !rotated ? 2 * hl : hl, chunk_b = kInterleaved || !rotated ? 2 * hl + 1 : hl + reach;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    const uint16_t* row[kIt];
#pragma unroll
    for (int i = 0; i < kIt; ++i)
        row[i] = (kind_of(i) == kQuery ? p.q : kind_of(i) == kKey ? p.k : p.v) + (mine ? h : 0) * kD + chunk_a * 8;
    const int apart = (chunk_b - chunk_a) * 8;
    // A tile's vectors and, for what goes to the cache, its slots.
    constexpr int kSlots = kBoth ? 1 : kIt;
    uint4 x[kIt][2];
    int64_t next_slots[kSlots];
    auto load = [&](int tile, int i) {
        const int64_t t = static_cast<int64_t>(tile) * kTile + offset_of(i);
        const int64_t stride = kind_of(i) == kQuery ? p.q_stride : kind_of(i) == kKey ? p.k_stride : p.v_stride;
        x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
        if (i < kSlots) next_slots[i] = -1;
        if (mine && t < p.tokens) {
            x[i][0] = ld_dep_stream_v4(row[i] + t * stride);
            x[i][1] = ld_dep_stream_v4(row[i] + t * stride + apart);
            if (i < kSlots && !query) next_slots[i] = *const_cast<const volatile int64_t*>(p.slots + t);
        }
    };
#pragma unroll
    for (int i = 0; i < kIt; ++i) load(blockIdx.x, i);
    Half w;
    {
        const uint4 none = make_uint4(0, 0, 0, 0);
        const uint4 packed[2] = {normed ? ld_dep_v4(weight + chunk_a * 8) : none, normed ? ld_dep_v4(weight + chunk_b * 8) : none};
        unpack(packed, w);
        const float2 offset = make_float2(p.weight_offset, p.weight_offset);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w.a[j] = __fadd2_rn(w.a[j], offset);
            w.b[j] = __fadd2_rn(w.b[j], offset);
        }
    }

    // This thread's pairs of a tile: their units a position, and where their positions are.
    uint64_t units[kPairs];
    const int64_t* position[kPairs];
    int pair[kPairs], token[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
        const int at = threadIdx.x + j * blockDim.x;
        token[j] = half > 0 ? min(at / half, kTile) : kTile;
        pair[j] = at - token[j] * half;
        units[j] = 0;
        position[j] = p.positions;
        if (token[j] < kTile) {
            units[j] = units_of(*const_cast<const volatile uint64_t*>(reinterpret_cast<const uint64_t*>(p.inv_freq) + pair[j]));
            int axis = p.axis ? ld_dep_s32(p.axis + pair[j]) : 0;
            if (axis < 0 || axis >= p.n_axes) {
                atomicOr(&g_rope_index_error, 1u);
                axis = 0;
            }
            position[j] += static_cast<int64_t>(axis) * p.tokens;
        }
    }
    // A lane's pairs 2j and 2j + 1 of its 8 lie together, beside the other lanes'.
    auto place_of = [](int pair) { return ((pair / 2 % 4) * kLanes + pair / 8) * 2 + pair % 2; };
    auto position_of = [&](int tile, int j) -> int64_t {
        const int64_t t = static_cast<int64_t>(tile) * kTile + token[j];
        return token[j] < kTile && tile < tiles && t < p.tokens ? *const_cast<const volatile int64_t*>(position[j] + t) : 0;
    };
    auto turn_by = [&](const int64_t (&pos)[kPairs], int buffer) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            if (token[j] >= kTile) continue;
            const uint32_t u = static_cast<uint32_t>(static_cast<uint64_t>(pos[j]) * units[j] >> 32);
            // The upper 24 bits, in half turns, are an fp32 number; the lower 8 turn a little further.
            const float at = __int2float_rn(static_cast<int>(u & ~0xFFu)) * 0x1p-31f;
            const float more = __uint2float_rn(u & 0xFFu) * 1.4629180792671596e-9f;  // pi 2^-31
            float sn, cs;
            sincospif(at, &sn, &cs);
            turns[buffer][token[j]][place_of(pair[j])] = make_float2(fmaf(-more, sn, cs) * p.rope_scale, fmaf(more, cs, sn) * p.rope_scale);
        }
    };
    int64_t pos[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) pos[j] = position_of(blockIdx.x, j);
    turn_by(pos, 0);
    __syncthreads();

    // Norm and turn of a tile's first n vectors. (The reciprocal root comes first, as in the formula: a finite vector whose sum
    // of squares passes fp32's range is then zeros, and not infinity times zero.)
    auto turned = [&](const int n, Half (&f)[kIt], const float2 (&turn)[kTile][kD / 2]) {
        if (normed) {
            float r[kIt];
#pragma unroll
            for (int i = 0; i < n; ++i) {
                float2 sum = __fmul2_rn(f[i].a[0], f[i].a[0]);
#pragma unroll
                for (int j = 1; j < 4; ++j) sum = __ffma2_rn(f[i].a[j], f[i].a[j], sum);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = __ffma2_rn(f[i].b[j], f[i].b[j], sum);
                r[i] = sum.x + sum.y;
            }
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) r[i] += __shfl_xor_sync(0xffffffffu, r[i], o);
#pragma unroll
            for (int i = 0; i < n; ++i) {
                asm("rsqrt.approx.f32 %0, %1;" : "=f"(r[i]) : "f"(fmaf(r[i], 1.0f / kD, p.eps)));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[i].a[j] = __fmul2_rn(__fmul2_rn(f[i].a[j], make_float2(r[i], r[i])), w.a[j]);
                    f[i].b[j] = __fmul2_rn(__fmul2_rn(f[i].b[j], make_float2(r[i], r[i])), w.b[j]);
                }
            }
        }
        if (rotated) {
            // The lane's 8 pairs: the two chunks' columns of one number, or, interleaved, 4 in each chunk.
#pragma unroll
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = f[i].a[j], b = f[i].b[j];
                    const float4 u = *reinterpret_cast<const float4*>(turn[offset_of(i)] + (j * kLanes + hl) * 2);
                    if constexpr (kInterleaved) {
                        // (pairs 2j, 2j + 1 of the lane's 8 are chunk a's columns 4j .. for j < 2, then chunk b's)
                        float2& y0 = j < 2 ? f[i].a[2 * j] : f[i].b[2 * j - 4];
                        float2& y1 = j < 2 ? f[i].a[2 * j + 1] : f[i].b[2 * j - 3];
                        y0 = make_float2(fmaf(-u.y, y0.y, u.x * y0.x), fmaf(u.y, y0.x, u.x * y0.y));
                        y1 = make_float2(fmaf(-u.w, y1.y, u.z * y1.x), fmaf(u.w, y1.x, u.z * y1.y));
                    } else {
                        f[i].a[j] = make_float2(fmaf(-u.y, b.x, u.x * a.x), fmaf(-u.w, b.y, u.z * a.y));
                        f[i].b[j] = make_float2(fmaf(u.y, a.x, u.x * b.x), fmaf(u.w, a.y, u.z * b.y));
                    }
                }
        }
    };
    uint16_t* const out = reinterpret_cast<uint16_t*>(p.q_out) + h * kD + chunk_a * 8;
    const int64_t out_stride = static_cast<int64_t>(p.q_heads) * kD;
    int buffer = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        int64_t pos_next[kPairs];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) pos_next[j] = position_of(tile + gridDim.x, j);
        Half f[kIt];
        int64_t slots[kSlots];
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            unpack(x[i], f[i]);
            if (i < kSlots) slots[i] = next_slots[i];
            load(tile + gridDim.x, i);
        }
        if (query) {
            turned(kIt, f, turns[buffer]);
#pragma unroll
            for (int i = 0; i < kIt; ++i) {
                const int64_t t = static_cast<int64_t>(tile) * kTile + offset_of(i);
                if (mine && t < p.tokens) {
                    *reinterpret_cast<uint4*>(out + t * out_stride) = pack_bf16x8(f[i].a);
                    *reinterpret_cast<uint4*>(out + t * out_stride + apart) = pack_bf16x8(f[i].b);
                }
            }
        } else {
            if (kind_of(0) == kKey) turned(kSlots, f, turns[buffer]);
            uint32_t top[kIt];
#pragma unroll
            for (int i = 0; i < kIt; ++i) {
                float most = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    most = largest(most, f[i].a[j]);
                    most = largest(most, f[i].b[j]);
                }
                top[i] = __float_as_uint(most) & 0x7FFFFFFFu;
            }
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1)
#pragma unroll
                for (int i = 0; i < kIt; ++i) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
            for (int i = 0; i < kIt; ++i) {
                int64_t& slot = slots[kBoth ? 0 : i];
                if (slot >= static_cast<int64_t>(c.num_pages) << c.page_log2) {
                    atomicOr(&g_rope_index_error, 1u);
                    slot = -1;
                }
                const bool there = mine && slot >= 0;
                // (a lane with nothing to store must not take its warp through the divisions that all-zero vectors get)
                const float scale = quant_head(f[i].a, f[i].b, there ? top[i] : __float_as_uint(1.0f));
                if (!there) continue;
                const bool key = kind_of(i) == kKey;
                const int64_t at = (((slot >> c.page_log2) * c.heads + h) << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
                uint2* const to = reinterpret_cast<uint2*>((key ? c.k : c.v) + at * kD);
                to[chunk_a] = pack_e4m3x8(f[i].a);
                to[chunk_b] = pack_e4m3x8(f[i].b);
                if (hl == 0) (key ? c.k_scale : c.v_scale)[at] = scale;
            }
        }
        if (tile + static_cast<int>(gridDim.x) >= tiles) break;
        buffer ^= 1;
        turn_by(pos_next, buffer);
        __syncthreads();  // the next turns are there, and the warps have read the ones before the present
    }
}

template <int kLanes, int kIt, int kTps>
cudaError_t launch(const RopeProblem& p, int num_sms, cudaStream_t stream) {
    constexpr int kHps = 32 / kLanes / kTps, kTile = kIt * kTps;
    const int64_t steps = (static_cast<int64_t>(p.q_heads) + kHps - 1) / kHps + 2 * ((static_cast<int64_t>(p.cache.heads) + kHps - 1) / kHps);
    const int64_t groups = (steps + kWarps - 1) / kWarps, warps = (steps + groups - 1) / groups;
    if (groups > 65535) return cudaErrorInvalidConfiguration;
    const int64_t tiles = (static_cast<int64_t>(p.tokens) + kTile - 1) / kTile;
    const int64_t resident = (num_sms * (kCtas * kWarps / warps) + groups - 1) / groups;
    auto kernel = p.interleaved ? rope_append_kernel<kLanes, true, kIt, kTps> : rope_append_kernel<kLanes, false, kIt, kTps>;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(tiles < resident ? tiles : resident), static_cast<unsigned>(groups)),
                            static_cast<int>(warps) * 32, 0, stream, 1, p);
}

// Many tokens: two at a time, or, where a warp has room for more heads than there are, that many. (3 heads on 1 of 128,
// 20000 tokens: 23.0 us, and 27.5 where one token a warp and round took 29.2.) With no more than a few for every CTA, one (us,
// one and two at a time: 24 heads on 4 of 128, 256 tokens 2.9 and 3.7, 512 3.75 and 3.9, 2500 9.7 and 9.2; 64 on 8, 64 tokens
// 2.9 and 3.2, 384 6.7 and 5.8; in between either may be ahead, 1000 tokens of 24 on 4 5.2 and 5.4).
template <int kLanes>
cudaError_t launch_tokens(const RopeProblem& p, int num_sms, cudaStream_t stream) {
    constexpr int kPer = 32 / kLanes;
    const int heads = p.q_heads > p.cache.heads ? p.q_heads : p.cache.heads;
    const int64_t steps = (static_cast<int64_t>(p.q_heads) + kPer - 1) / kPer + 2 * ((static_cast<int64_t>(p.cache.heads) + kPer - 1) / kPer);
    if (p.tokens * steps <= 2 * static_cast<int64_t>(num_sms) * kCtas * kWarps) return launch<kLanes, 1, 1>(p, num_sms, stream);
    if constexpr (kPer >= 8)
        if (heads <= kPer / 8) return launch<kLanes, 1, 8>(p, num_sms, stream);
    if constexpr (kPer >= 4)
        if (heads <= kPer / 4) return launch<kLanes, 1, 4>(p, num_sms, stream);
    if (heads <= kPer / 2) return launch<kLanes, 1, 2>(p, num_sms, stream);
    return launch<kLanes, 2, 1>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeProblem& p, int num_sms, cudaStream_t stream) {
    switch (p.cache.head_dim) {
        case 64: return launch_tokens<4>(p, num_sms, stream);
        case 128: return launch_tokens<8>(p, num_sms, stream);
        default: return launch_tokens<16>(p, num_sms, stream);
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
