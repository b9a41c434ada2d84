// Writing new keys and values into the paged E4M3 cache.
//
// A head vector x of D values becomes D codes and one fp32 scale by the
// activation rule: s = amax / 448 (1 for an all-zero vector), code = E4M3(x / s)
// with the IEEE quotient. A vector that holds a NaN or an infinity is stored as
// zero codes with a NaN scale: it reads back as NaN, and as its codes are
// finite it cannot reach a query that does not attend to it (0 * code stays 0).
//
// A vector is read once and written once, by 8 to 32 lanes; nothing is shared
// between vectors, so a token's place costs one load of its slot and no order
// is kept. 4096 tokens x 4 heads x 128 (12.7 MB) take 4.3 us, 2.9 TB/s: the
// slot, then the vector (not read for a negative slot), then the store, one
// vector in flight per group of lanes, and the launch. A batch of 102 tokens
// takes the same trips, 1.6 us.
#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {
namespace {

__device__ unsigned int g_kv_index_error;

// kLanes = D / 8 lanes hold one vector, 8 values each. The quotients are
// formed as in act_group.cuh (short fused multiply-add sequences that give the
// IEEE division's codes for every bf16 pair in range); the maximum is taken on
// the bit patterns, where NaN and infinity order above every finite value.
template <int kLanes>
__global__ void __launch_bounds__(256) kv_append_kernel(const uint4* k, const uint4* v, const int64_t* slots,
                                                        int64_t vectors, int heads, int64_t k_stride, int64_t v_stride,
                                                        KvCache c) {
    const int hl = threadIdx.x % kLanes;
    const int64_t vec = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / kLanes;
    const int per_token = 2 * heads;
    const int64_t t = vec / per_token;
    const int j = static_cast<int>(vec - t * per_token);
    const bool is_v = j >= heads;
    const int h = is_v ? j - heads : j;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    int64_t slot = -1;
    if (vec < vectors) {
        slot = *const_cast<const volatile int64_t*>(slots + t);
        if (slot >= static_cast<int64_t>(c.num_pages) << c.page_log2) {
            if (hl == 0) atomicOr(&g_kv_index_error, 1u);
            slot = -1;
        }
    }
    uint4 x = make_uint4(0, 0, 0, 0);
    if (slot >= 0) x = ld_dep_stream_v4(is_v ? v + t * v_stride + h * kLanes + hl : k + t * k_stride + h * kLanes + hl);
    uint32_t top = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float amax = __uint_as_float(top << 16);
    float f[8], s;
    unpack_bf16x8(x, f);
    if (amax >= kFastQuotientMinAmax && amax <= kFastQuotientMaxAmax) {
        constexpr float kInv448 = 1.0f / kE4M3Max;
        const float s0 = __fmul_rn(amax, kInv448);
        s = __fmaf_rn(-__fmaf_rn(kE4M3Max, s0, -amax), kInv448, s0);
        const float y0 = rcp_approx_ftz(s);
        const float y = __fmaf_rn(__fmaf_rn(-s, y0, 1.0f), y0, y0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q0 = __fmul_rn(f[i], y);
            f[i] = __fmaf_rn(-__fmaf_rn(s, q0, -f[i]), y, q0);
        }
    } else {
        const bool finite = top < 0x7F80u;
        s = top == 0 ? 1.0f : finite ? __fdiv_rn(amax, kE4M3Max) : __uint_as_float(0x7FFFFFFFu);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = finite ? __fdiv_rn(f[i], s) : 0.0f;
    }
    if (slot < 0) return;
    const int64_t page = slot >> c.page_log2;
    const int64_t at = ((page * heads + h) << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
    reinterpret_cast<uint2*>(is_v ? c.v : c.k)[at * kLanes + hl] = pack_e4m3x8(f);
    if (hl == 0) (is_v ? c.v_scale : c.k_scale)[at] = s;
}

}  // namespace

cudaError_t launch_kv_append(const void* k, const void* v, const int64_t* slots, int T, int64_t k_stride,
                             int64_t v_stride, const KvCache& cache, cudaStream_t stream) {
    const int lanes = cache.head_dim / 8;
    const int64_t vectors = 2 * static_cast<int64_t>(T) * cache.heads;
    const int64_t blocks = (vectors * lanes + 255) / 256;
    auto kernel = lanes == 8 ? kv_append_kernel<8> : lanes == 16 ? kv_append_kernel<16> : kv_append_kernel<32>;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(blocks)), 256, 0, stream, 1,
                            static_cast<const uint4*>(k), static_cast<const uint4*>(v), slots, vectors, cache.heads,
                            k_stride / 8, v_stride / 8, cache);
}

unsigned int read_and_clear_kv_index_error() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv_index_error, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_kv_index_error, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace fp8act
