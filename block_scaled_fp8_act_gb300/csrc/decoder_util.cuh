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

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ uint2 pack_e4m3x8(const float (&f)[8]) {
    return make_uint2(cvt_e4m3x2(f[0], f[1]) | (cvt_e4m3x2(f[2], f[3]) << 16),
                      cvt_e4m3x2(f[4], f[5]) | (cvt_e4m3x2(f[6], f[7]) << 16));
}

// Quantises one 128-wide group of fp32 values held by a half-warp (8 per
// lane; the whole warp executes the call): s = amax / 448 (1 for an all-zero
// group), code = E4M3(f / s). f is itself a rounded fp32 result here, so the
// quotient is taken as f * RN(1 / s), within 1.5 fp32 ulp of the IEEE one: a
// code differs from the IEEE quotient's only where that lies within 1.5 ulp
// of a rounding midpoint, closer than f's own error. Outside [2^-100, 2^100],
// where 1 / s nears the ends of the range, the division is done.
__device__ __forceinline__ float quant_f32_group_halfwarp(float (&f)[8], uint2& codes) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = amax == 0.0f ? 1.0f : __fdiv_rn(amax, kE4M3Max);
    if (amax >= 0x1p-100f && amax <= 0x1p100f) {
        const float y = __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= y;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __fdiv_rn(f[i], s);
    }
    codes = pack_e4m3x8(f);
    return s;
}

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
