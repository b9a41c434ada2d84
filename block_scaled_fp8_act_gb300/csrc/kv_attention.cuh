// What the two attention kernels share: arguments, the list of work units, and
// the record of items that cross CTAs.
#pragma once

#include <cuda_fp16.h>

#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {

constexpr float kNegInf = -__builtin_huge_valf();

// An item (sequence, KV head, row tile) that starts in a CTA and goes on in the next.
struct __align__(16) SplitItem {
    int parts, second;  // CTAs it spans (0: no such item); whether its part of the first CTA is that CTA's second
    int q0, h, row0, nrows, pad[2];
};

struct AttnArgs {
    const uint16_t* q;
    int64_t q_stride;
    const int* cu_q;
    const int* kv_lens;
    const int* table;
    int64_t table_stride;
    int batch, tokens, group;
    int rows;  // of a row tile
    float scale_log2;
    KvCache c;
    uint32_t* out;     // bf16 [tokens, heads * group, D]
    float* lse;        // [tokens, heads * group] or null
    float* part_o;     // [2 * grid][rows][D]
    float* part_ml;    // [2 * grid][rows][2]
    SplitItem* split;  // [grid]
    unsigned int* index_error;
};

// CTAs of the main kernel (two per SM at most) that the workspace is made for.
constexpr int kMaxAttnGrid = 2 * 160;

// Asynchronous copies to shared memory; zeros are written where `in` is false, and nothing is read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}

// Two E4M3 codes (the low or the high 16 bits of `codes`) to f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_lo_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(r) : "r"(codes));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(r) : "r"(codes));
    return r;
}

// The power of two below a scale, as its bits; 0 for a NaN scale (a poisoned token).
__device__ __forceinline__ uint32_t scale_exponent(float s) {
    const uint32_t e = __float_as_uint(s) & 0x7F800000u;
    return e == 0x7F800000u ? 0u : e;
}

// One item and where it lies in the unit list. A unit is kTok cached tokens of
// a row tile; an item counts kCost units beside its own.
struct Item {
    int b, h, rt;      // sequence, KV head, row tile
    int nq, q0, len;   // new tokens, first one's row in q, cached tokens
    int rts, tiles;    // row tiles of this sequence and units of each, kCost included
    int64_t first;     // index of the item's first unit
};

template <int kTok, int kCost>
struct Units {
    static __device__ __forceinline__ void load_sequence(const AttnArgs& a, int b, Item& it) {
        const int q0 = ld_dep_s32(a.cu_q + b), q1 = ld_dep_s32(a.cu_q + b + 1);
        int len = ld_dep_s32(a.kv_lens + b);
        const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.tokens;
        it.q0 = q0;
        it.nq = ok ? q1 - q0 : 0;
        const int64_t most = a.table_stride << a.c.page_log2;
        if (!ok || len < 0 || len > most) {
            atomicOr(a.index_error, 1u);
            len = len < 0 ? 0 : static_cast<int>(len > most ? most : len);
        }
        it.len = len;
        it.rts = (it.nq * a.group + a.rows - 1) / a.rows;
        it.tiles = (len + kTok - 1) / kTok + kCost;  // (an empty sequence still writes its rows)
    }

    // Units per CTA: an even share, but not less than is worth a part of an item.
    static __device__ __forceinline__ int64_t per_cta(int64_t total, int least) {
        const int64_t per = (total + gridDim.x - 1) / gridDim.x;
        return per < least ? least : per;
    }

    struct Scratch {
        int64_t total, first;
        int b;
    };

    // This CTA's units [u, u_end) and the item that holds the first one; false if it has none. Called by the whole
    // CTA.
    static __device__ __forceinline__ bool first_item(const AttnArgs& a, int least, Scratch& sh, Item& it, int64_t& per,
                                                      int64_t& u, int64_t& u_end) {
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x;
            auto units_of = [&](int b) -> int64_t {
                if (b >= a.batch) return 0;
                Item x;
                load_sequence(a, b, x);
                return static_cast<int64_t>(a.c.heads) * x.rts * x.tiles;
            };
            const int64_t u_lane = units_of(lane);
            int64_t total = 0;
            for (int b0 = 0; b0 < a.batch; b0 += 32) {
                int64_t n = b0 == 0 ? u_lane : units_of(b0 + lane);
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
                total += n;
            }
            const int64_t u0 = per_cta(total, least) * blockIdx.x;
            int64_t base = 0;
            for (int b0 = 0; b0 < a.batch && u0 < total; b0 += 32) {
                const int64_t n = b0 == 0 ? u_lane : units_of(b0 + lane);
                int64_t incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += v;
                }
                const int64_t lo = base + incl - n;
                if (u0 >= lo && u0 < lo + n) {
                    sh.b = b0 + lane;
                    sh.first = lo;
                }
                base += __shfl_sync(0xffffffffu, incl, 31);
                if (base > u0) break;
            }
            if (lane == 0) {
                sh.total = total;
                a.split[blockIdx.x].parts = 0;
            }
        }
        __syncthreads();
        per = per_cta(sh.total, least);
        u = per * blockIdx.x;
        u_end = u + per < sh.total ? u + per : sh.total;
        if (u >= u_end) return false;
        it.b = sh.b;
        load_sequence(a, it.b, it);
        const int64_t rel = (u - sh.first) / it.tiles;
        it.h = static_cast<int>(rel / it.rts);
        it.rt = static_cast<int>(rel % it.rts);
        it.first = sh.first + rel * it.tiles;
        return true;
    }

    static __device__ __forceinline__ void next_item(const AttnArgs& a, Item& it) {
        it.first += it.tiles;
        if (++it.rt == it.rts) {
            it.rt = 0;
            if (++it.h == a.c.heads) {
                it.h = 0;
                do load_sequence(a, ++it.b, it);
                while (it.rts == 0);
            }
        }
    }
};

// The record of an item that starts in this CTA and goes on in the next; `slot` is its part here.
__device__ __forceinline__ void write_split(const AttnArgs& a, const Item& it, int64_t per, int slot, int row0, int nrows) {
    SplitItem sp = {};
    sp.parts = static_cast<int>((it.first + it.tiles - 1) / per) - static_cast<int>(blockIdx.x) + 1;
    sp.second = slot & 1;
    sp.q0 = it.q0;
    sp.h = it.h;
    sp.row0 = row0;
    sp.nrows = nrows;
    a.split[blockIdx.x] = sp;
}

// The kernel for wide row tiles of head size 128 (kv_attention_tc.cu); the
// caller launches the join of the split items after it.
cudaError_t launch_attention_tc(const AttnArgs& a, int num_sms, cudaStream_t stream);

}  // namespace fp8act
