// Device and host helpers of the operators between the linear layers (norm,
// gated activation, cache, attention, verification).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "act_group.cuh"
#include "common.cuh"
#include "sm100_ptx.cuh"

namespace fp8act {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One 32-bit integer that the previous grid may have written (a length, a
// page, a token): read after the wait, as the loads of common.cuh are.
__device__ __forceinline__ int ld_dep_s32(const int* p) {
    int v;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Eight bf16 values to fp32.
__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

// The same in pairs, for the two-wide fp32 instructions.
__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float2 (&f)[4]) {
    f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
    f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
    f[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z));
    f[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
}
__device__ __forceinline__ uint4 pack_bf16x8(const float2 (&f)[4]) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                      pack_bf16x2(f[3].x, f[3].y));
}

__device__ __forceinline__ uint2 pack_e4m3x8(const float2 (&f)[4]) {
    return make_uint2(cvt_e4m3x2(f[0].x, f[0].y) | (cvt_e4m3x2(f[1].x, f[1].y) << 16),
                      cvt_e4m3x2(f[2].x, f[2].y) | (cvt_e4m3x2(f[3].x, f[3].y) << 16));
}

// The largest bit pattern of 8 bf16 magnitudes: NaN and infinity order above every finite value.
__device__ __forceinline__ uint32_t top_bits(const uint4& x) {
    const uint32_t t = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    return max(t & 0xFFFFu, t >> 16);
}

// Quantises one 128-wide group of fp32 values held by a half-warp (8 per
// lane; the whole warp executes the call): s = amax / 448 (1 for an all-zero
// group), code = E4M3(f / s). s is the IEEE quotient: q0 = amax * RN(1/448) is
// within 2 ulp, its remainder 448 q0 - amax is a small multiple of an ulp and
// so exact, and amax / 448 = amax / (7 * 64) lies at least 1/14 ulp from any
// rounding midpoint, far more than the corrected sum's error before its one
// rounding. f is itself a rounded fp32 result here, so its quotient is taken as
// f * y, y the approximate reciprocal after a Newton-Raphson step, within 2 fp32
// ulp of the IEEE one: a code differs from the IEEE quotient's only where that
// lies within 2 ulp of a rounding midpoint, closer than f's own error. Outside
// [2^-100, 2^100], where the remainder or 1 / s nears the ends of the range,
// the divisions are done.
__device__ __forceinline__ float quant_f32_group_halfwarp(float2 (&f)[4], uint2& codes) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float s;
    if (amax >= 0x1p-100f && amax <= 0x1p100f) {
        constexpr float kInv448 = 1.0f / kE4M3Max;
        const float s0 = __fmul_rn(amax, kInv448);
        s = __fmaf_rn(-__fmaf_rn(kE4M3Max, s0, -amax), kInv448, s0);
        const float y0 = rcp_approx_ftz(s);
        const float y = __fmaf_rn(__fmaf_rn(-s, y0, 1.0f), y0, y0);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(f[i], make_float2(y, y));
    } else {
        s = amax == 0.0f ? 1.0f : __fdiv_rn(amax, kE4M3Max);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(__fdiv_rn(f[i].x, s), __fdiv_rn(f[i].y, s));
    }
    codes = pack_e4m3x8(f);
    return s;
}

// Quantises one head vector, 8 or 16 fp32 values a lane: s = amax / 448 (1 for
// an all-zero vector), which become the quotients by s. `top` is the bit pattern of
// the largest magnitude, where NaN and infinity order above every finite value;
// a vector that holds one becomes zeros with a NaN scale. The quotients are
// formed as in act_group.cuh: for bf16 values those of the IEEE division, for
// rounded fp32 ones within an ulp of it.
template <class... Chunk>
__device__ __forceinline__ float quant_head_chunks(uint32_t top, Chunk&... chunks) {
    const float amax = __uint_as_float(top);
    float s;
    if (amax >= kFastQuotientMinAmax && amax <= kFastQuotientMaxAmax) {
        constexpr float kInv448 = 1.0f / kE4M3Max;
        const float s0 = __fmul_rn(amax, kInv448);
        s = __fmaf_rn(-__fmaf_rn(kE4M3Max, s0, -amax), kInv448, s0);
        const float y0 = rcp_approx_ftz(s);
        const float y = __fmaf_rn(__fmaf_rn(-s, y0, 1.0f), y0, y0);
        const float2 y2 = make_float2(y, y), minus_s = make_float2(-s, -s);
        auto quotients = [&](float2 (&f)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 q0 = __fmul2_rn(f[i], y2);
                f[i] = __ffma2_rn(__ffma2_rn(minus_s, q0, f[i]), y2, q0);
            }
        };
        (quotients(chunks), ...);
    } else {
        const bool finite = top < 0x7F800000u;
        s = top == 0 ? 1.0f : finite ? __fdiv_rn(amax, kE4M3Max) : __uint_as_float(0x7FFFFFFFu);
        auto quotients = [&](float2 (&f)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = finite ? make_float2(__fdiv_rn(f[i].x, s), __fdiv_rn(f[i].y, s)) : make_float2(0.0f, 0.0f);
        };
        (quotients(chunks), ...);
    }
    return s;
}
__device__ __forceinline__ float quant_head(float2 (&f)[4], uint32_t top) { return quant_head_chunks(top, f); }
__device__ __forceinline__ float quant_head(float2 (&f)[4], float2 (&g)[4], uint32_t top) { return quant_head_chunks(top, f, g); }

// Launch with programmatic stream serialization (and a cluster size when it
// is above 1): the kernel may start before the previous one has finished and
// waits for it itself.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster,
                             A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace fp8act
