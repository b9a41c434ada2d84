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
// Angles. A turn is 2^64 units: inv_freq / 2 pi, taken in 64 bits, becomes a
// whole number of units, and its product with the position wraps to the angle's
// remainder exactly, with no table and no bound on the position. What is lost
// is the frequency's own rounding, 2^-52 of the number of turns. The remainder,
// in (-1/2, 1/2] of a turn, is rounded to fp32, 2^-25 of itself.
//
// Work split. A CTA takes one token: R / 2 threads find its sines and cosines
// once for all heads, while the D / 8 lanes of each vector wait for their 16
// bytes. Nothing is shared between tokens.
#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {
namespace {

__device__ unsigned int g_rope_index_error;

constexpr int kMaxHalf = 128;  // pairs of a head

// Lane l of a vector's kLanes holds columns 8l .. 8l + 7.
template <int kLanes>
__global__ void __launch_bounds__(512) rope_append_kernel(const __grid_constant__ RopeProblem p) {
    __shared__ float2 turns[kMaxHalf];  // (cos, sin) * rope_scale
    const int64_t t = blockIdx.x;
    const int hl = threadIdx.x % kLanes, group = threadIdx.x / kLanes, groups = blockDim.x / kLanes;
    const KvCache& c = p.cache;
    const int half = p.rot / 2, vectors = p.q_heads + 2 * c.heads;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    auto load = [&](int vec) {
        const int h = vec - p.q_heads;
        const uint16_t* at = h < 0          ? p.q + t * p.q_stride + vec * (8 * kLanes)
                             : h < c.heads  ? p.k + t * p.k_stride + h * (8 * kLanes)
                                            : p.v + t * p.v_stride + (h - c.heads) * (8 * kLanes);
        return vec < vectors ? ld_dep_stream_v4(at + hl * 8) : make_uint4(0, 0, 0, 0);
    };
    uint4 x = load(group), ahead = load(group + groups);
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint4 wq = p.q_weight ? ld_dep_v4(p.q_weight + hl * 8) : none, wk = p.k_weight ? ld_dep_v4(p.k_weight + hl * 8) : none;
    int64_t slot = *const_cast<const volatile int64_t*>(p.slots + t);
    for (int i = threadIdx.x; i < half; i += blockDim.x) {
        const double freq = *const_cast<const volatile double*>(p.inv_freq + i);
        int axis = p.axis ? ld_dep_s32(p.axis + i) : 0;
        if (axis < 0 || axis >= p.n_axes) {
            atomicOr(&g_rope_index_error, 1u);
            axis = 0;
        }
        const int64_t pos = *const_cast<const volatile int64_t*>(p.positions + axis * p.tokens + t);
        const double turn = freq * 0.15915494309189535;  // 1 / 2 pi
        const uint64_t units = __double2ull_rn((turn - floor(turn)) * 0x1p64);
        const float at = __ll2float_rn(static_cast<int64_t>(static_cast<uint64_t>(pos) * units)) * 0x1p-63f;  // half turns
        float sn, cs;
        sincospif(at, &sn, &cs);
        turns[i] = make_float2(cs * p.rope_scale, sn * p.rope_scale);
    }
    if (slot >= static_cast<int64_t>(c.num_pages) << c.page_log2) {
        if (threadIdx.x == 0) atomicOr(&g_rope_index_error, 1u);
        slot = -1;
    }
    const int64_t place = slot < 0 ? 0 : ((slot >> c.page_log2) * c.heads << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
    __syncthreads();

    // The lane's sines and cosines: of its 8 columns' pairs, or of its 4 pairs.
    const int reach = p.rot / 16;  // lanes of half the rotated columns
    const bool rotated = hl < 2 * reach, second = hl >= reach;
    float2 turn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = p.interleaved ? hl * 4 + i / 2 : (second ? hl - reach : hl) * 8 + i;
        turn[i] = rotated ? turns[at] : make_float2(1.0f, 0.0f);
        if (!p.interleaved && !second) turn[i].y = -turn[i].y;  // the other half's columns enter with this sign
    }
    const int lane = threadIdx.x & 31;
    const int partner = rotated ? (second ? lane - reach : lane + reach) : lane;

    const int first_of_warp = group - lane / kLanes;  // (the whole warp goes round as long as its first vector is one)
    for (int base = 0; first_of_warp + base < vectors; base += groups) {
        const int vec = group + base;
        const bool is_q = vec < p.q_heads, is_v = vec >= p.q_heads + c.heads;
        float f[8];
        unpack_bf16x8(x, f);
        x = ahead;
        ahead = load(vec + 2 * groups);
        if (__any_sync(0xffffffffu, !is_v)) {
            float y[8];
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(f[i], f[i], sum);
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = f[i];
            if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
                const float r = rsqrtf(sum * (1.0f / (8 * kLanes)) + p.eps);
                float w[8];
                unpack_bf16x8(is_q ? wq : wk, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = y[i] * r * (w[i] + p.weight_offset);
            }
            float z[8];
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    z[i] = rotated ? y[i] * turn[i].x - y[i + 1] * turn[i].y : y[i];
                    z[i + 1] = rotated ? y[i + 1] * turn[i].x + y[i] * turn[i].y : y[i + 1];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float other = __shfl_sync(0xffffffffu, y[i], partner);
                    z[i] = rotated ? fmaf(other, turn[i].y, y[i] * turn[i].x) : y[i];
                }
            }
            if (!is_v) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = z[i];
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
        if (__any_sync(0xffffffffu, !is_q))
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (vec >= vectors) continue;
        if (is_q) {
            reinterpret_cast<uint4*>(p.q_out)[(t * p.q_heads + vec) * kLanes + hl] = make_uint4(
                pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        } else if (slot >= 0) {
            const float s = quant_head(f, top);
            const int64_t at = place + (static_cast<int64_t>(vec - p.q_heads - (is_v ? c.heads : 0)) << c.page_log2);
            reinterpret_cast<uint2*>(is_v ? c.v : c.k)[at * kLanes + hl] = pack_e4m3x8(f);
            if (hl == 0) (is_v ? c.v_scale : c.k_scale)[at] = s;
        }
    }
}

}  // namespace

cudaError_t launch_rope_append(const RopeProblem& p, cudaStream_t stream) {
    const int lanes = p.cache.head_dim / 8;
    const int64_t all = static_cast<int64_t>(p.q_heads + 2 * p.cache.heads) * lanes;
    const int most = p.tokens > 608 ? 256 : 512;
    const int threads = all >= most ? most : static_cast<int>((all + 31) / 32 * 32);
    auto kernel = lanes == 8 ? rope_append_kernel<8> : lanes == 16 ? rope_append_kernel<16> : rope_append_kernel<32>;
    return launch_dependent(kernel, dim3(p.tokens), threads, 0, stream, 1, p);
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
