// The two elementwise operators that feed a block-FP8 product: RMS norm with
// the residual's addition, and silu(gate) * up, each ending in the product's
// own activation format (E4M3 codes, one fp32 scale per 128 columns).
//   norm: h = x + residual (stored as bf16), y = h / sqrt(mean h^2 + eps) * (weight + offset)
//   silu: y = gate / (1 + exp(-gate)) * up
// Both read and write each value once, so memory bounds them: 4096 x 5120 with
// residual moves 147 MB in 26.1 us (5.6 TB/s, 0.83 of a copy's rate), 4096 x
// 8704 gates 179 MB in 29.7 us (6.0 TB/s, 0.89; with loads that pass L1 by
// 0.7 us more). One row takes 1.8 us, a launch
// with one trip to memory and the row's reductions. The sum of squares is fp32.
// Arithmetic goes in pairs and the scale and its reciprocal without divisions:
// at 250 instructions per 8 columns issue slots were 72 % busy (27.4 us).
#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {
namespace {

// One CTA per row; thread t holds the 8-column chunks t, t + blockDim, ... so
// a half-warp always holds one 128-wide quantisation group and the row is
// read once. blockDim is a multiple of 32.
template <int kChunks, bool kResidual>
__global__ void __launch_bounds__(1024) rmsnorm_quant_kernel(const uint4* x, const uint4* residual, const uint4* weight, float eps,
                                     float weight_offset, int chunks, uint2* q, float* sa, uint4* residual_out) {
    __shared__ float part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    x += row * chunks;
    q += row * chunks;
    sa += row * (chunks / 16);
    if (kResidual) {
        residual += row * chunks;
        residual_out += row * chunks;
    }
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    uint4 wv[kChunks];  // (after the wait too: a weight may be a cast or a sum made just before)
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        wv[i] = c < chunks ? ld_dep_v4(weight + c) : make_uint4(0, 0, 0, 0);
    }
    float2 h[kChunks][4], ss2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        const bool in = c < chunks;
        unpack_bf16x8(in ? ld_dep_v4(x + c) : make_uint4(0, 0, 0, 0), h[i]);
        if (kResidual) {
            float2 r[4];
            unpack_bf16x8(in ? ld_dep_v4(residual + c) : make_uint4(0, 0, 0, 0), r);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[i][j] = __fadd2_rn(h[i][j], r[j]);
            if (in) residual_out[c] = pack_bf16x8(h[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) ss2 = __ffma2_rn(h[i][j], h[i][j], ss2);
    }
    float ss = ss2.x + ss2.y;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = lane < (blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rstd = rsqrtf(ss / static_cast<float>(chunks * 8) + eps);
    const float2 rstd2 = make_float2(rstd, rstd), offset2 = make_float2(weight_offset, weight_offset);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        const bool in = c < chunks;
        float2 w[4];
        unpack_bf16x8(wv[i], w);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __fmul2_rn(__fmul2_rn(h[i][j], rstd2), __fadd2_rn(w[j], offset2));
        uint2 codes;
        const float s = quant_f32_group_halfwarp(w, codes);
        if (in) {
            q[c] = codes;
            if ((lane & 15) == 0) sa[c / 16] = s;
        }
    }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSiluCtas = 6;  // per SM, at 40 registers a thread
// silu(gate) * up of one row [gate (I) | up (I)]: a half-warp per 128-wide
// group, warps striding over (row, pair of groups).
__global__ void __launch_bounds__(256) silu_mul_quant_kernel(const uint4* gate_up, int64_t M, int groups, uint2* q, float* sa) {
    const int lane = threadIdx.x & 31, hl = lane & 15;
    const int pairs = (groups + 1) / 2;
    const int64_t items = M * pairs;
    const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    int64_t row = item / pairs;
    int pair = static_cast<int>(item - row * pairs);
    const int64_t step_rows = step / pairs;
    const int step_pairs = static_cast<int>(step - step_rows * pairs);
    uint4 va, vb;
    auto load = [&]() {
        const int g = pair * 2 + (lane >> 4);
        const bool in = item < items && g < groups;
        const uint4* p = gate_up + row * groups * 32 + g * 16 + hl;
        va = in ? ld_dep_v4(p) : make_uint4(0, 0, 0, 0);
        vb = in ? ld_dep_v4(p + groups * 16) : make_uint4(0, 0, 0, 0);
    };
    load();
    while (item < items) {
        float2 a[4], b[4];
        unpack_bf16x8(va, a);
        unpack_bf16x8(vb, b);
        const int64_t at = row * groups + pair * 2 + (lane >> 4);
        const bool in = pair * 2 + (lane >> 4) < groups;
        item += step;  // the next item's loads run under this one's arithmetic
        row += step_rows;
        pair += step_pairs;
        if (pair >= pairs) {
            pair -= pairs;
            ++row;
        }
        load();
        // gate / 4 times the reciprocal of (1 + exp(-gate)) / 4, which stays below 2^126, where the approximation would
        // return 0, up to the gates (-88.7) whose exponential is infinite and whose quotient is 0 by the formula.
        // The exponential, the reciprocal and the product are within 2 fp32 ulp each, but the exponent's rounding
        // makes a relative error of up to ln 2 times half its ulp besides: 2^-21 for gates within 11 of 0, 2^-18 (41 ulp)
        // at -60 and beyond. Codes keep 4 bits of it: with the exponent's remainder added, or with expf, the codes of
        // 4096 x 8704 are as far from those of 64 bits as these (2.0e-4 of their norm), in 39.8 and 37.7 us.
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 t = __ffma2_rn(a[j], make_float2(-kLog2e, -kLog2e), make_float2(-2.0f, -2.0f));
            const float2 d = __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), make_float2(0.25f, 0.25f));
            const float2 g = __fmul2_rn(a[j], make_float2(0.25f, 0.25f));
            a[j] = __fmul2_rn(__fmul2_rn(g, make_float2(rcp_approx_ftz(d.x), rcp_approx_ftz(d.y))), b[j]);
        }
        uint2 codes;
        const float s = quant_f32_group_halfwarp(a, codes);
        if (in) {
            q[at * 16 + hl] = codes;
            if (hl == 0) sa[at] = s;
        }
    }
}

template <int kChunks>
cudaError_t launch_norm(const void* x, const void* residual, const void* weight, float eps, float weight_offset,
                        int64_t M, int chunks, void* q, float* sa, void* residual_out, cudaStream_t stream) {
    const int threads = ((chunks + kChunks - 1) / kChunks + 31) / 32 * 32;
    return launch_dependent(residual ? rmsnorm_quant_kernel<kChunks, true> : rmsnorm_quant_kernel<kChunks, false>,
                            dim3(static_cast<unsigned>(M)), threads, 0, stream, 1, static_cast<const uint4*>(x),
                            static_cast<const uint4*>(residual), static_cast<const uint4*>(weight), eps, weight_offset,
                            chunks, static_cast<uint2*>(q), sa, static_cast<uint4*>(residual_out));
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const void* x, const void* residual, const void* weight, float eps,
                                 float weight_offset, int M, int K, void* q, float* sa, void* residual_out,
                                 cudaStream_t stream) {
    const int chunks = K / 8;
    // One chunk per thread wherever a CTA holds the row: 4096 x 5120 with residual took 27.4 us so, with 2 or 4 chunks
    // per thread 28.9 or 32.5. (CTAs that stay and request the next row early: 26.7 to 31, then 26.2 with a CTA a row.)
    if (chunks <= 1024)
        return launch_norm<1>(x, residual, weight, eps, weight_offset, M, chunks, q, sa, residual_out, stream);
    return launch_norm<4>(x, residual, weight, eps, weight_offset, M, chunks, q, sa, residual_out, stream);
}

cudaError_t launch_silu_mul_quant(const void* gate_up, int M, int I, void* q, float* sa, int num_sms,
                                  cudaStream_t stream) {
    const int groups = I / kGroup;
    const int64_t warps = static_cast<int64_t>(M) * ((groups + 1) / 2);
    int64_t blocks = (warps + 7) / 8;
    // No more CTAs than run at once: 4096 x 8704 took 30.0 us, with 8 per SM, a third of them in a second wave, 34.4,
    // with 8 at 32 registers (spills) 33.6.
    if (blocks > kSiluCtas * static_cast<int64_t>(num_sms)) blocks = kSiluCtas * static_cast<int64_t>(num_sms);
    return launch_dependent(silu_mul_quant_kernel, dim3(static_cast<unsigned>(blocks)), 256, 0, stream, 1,
                            static_cast<const uint4*>(gate_up), static_cast<int64_t>(M), groups,
                            static_cast<uint2*>(q), sa);
}

}  // namespace fp8act
