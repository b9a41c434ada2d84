// What the two attention kernels share: arguments, the list of work units, and
// the record of items that cross CTAs.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "decoder_util.cuh"
#include "kernels.h"
#include "scores.cuh"

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
    Scores scores;
    // the accumulated weights alone
    float* mass;       // [pages, heads, page]
    bool accumulate;
    const int* old_lens;  // [batch] or null: all but the new tokens
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

// Rows of queries to shared memory as f16 in the order of the MMA's B fragments, each scaled by a power of two so that its
// largest value is in [1, 2): bf16 then fits f16 exactly down to 2^-17 of that, and below to within 2^-25 of it. `load`
// gives 8 values of a row, `scale` takes the row's power of two. Called by the whole CTA; `rows` is a multiple of 8.
template <int kD, int kThreads, class Load, class Scale>
__device__ __forceinline__ void stage_queries(uint8_t* q, int rows, Load load, Scale scale) {
    constexpr int kLanes = kD / 8, kKS = kD / 32;
    static_assert(kLanes <= 32 && 8 % (32 / kLanes) == 0, "whole warps of rows");
    const int c = threadIdx.x % kLanes;
    for (int r = threadIdx.x / kLanes; r < rows; r += kThreads / kLanes) {
        const uint4 x = load(r, c);
        // (a warp's rows are all below `rows` or none is, so that the whole warp is here)
        uint32_t top = top_bits(x);
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // (a zero row's exponent is as good as any)
        const uint32_t e = top == 0 ? 127 : min(max(top >> 7, 1u), 253u);
        const float up = __uint_as_float((254 - e) << 23);  // 2^(127 - e)
        if (c == 0) scale(r, __uint_as_float(e << 23));
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
        reinterpret_cast<uint4*>(q)[((r >> 3) * kKS + ks) * 32 + (r & 7) * 4 + (c % 8) / 2] = make_uint4(h[0], h[1], h[2], h[3]);
    }
}

// One token's codes and its neighbours' from the cache's tensor map to shared memory.
__device__ __forceinline__ void load_tokens(uint32_t dst, const CUtensorMap* map, uint32_t bar, int line) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(0), "r"(line)
        : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float4 lds_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// 32 rows of queries of head size 128 as the two E4M3 parts of a tcgen05 operand (128-byte rows, swizzled), the low one
// `apart` bytes behind the high one: a row, scaled by a power of two so that its largest value is in [128, 256), is
// E4M3(q) + E4M3(q - E4M3(q)), exact down to 2^-9 of its largest value and within 2^-17 of that below. `at` is the
// element of the lane's row, rows from `valid` on are zero; `scale` takes a row and its power of two. By a whole warp; the
// caller fences the asynchronous proxy.
template <class Scale>
__device__ __forceinline__ void stage_query_parts(uint8_t* q, int apart, const uint16_t* src, int64_t at, int valid, Scale scale) {
    const int lane = threadIdx.x & 31;
    // The rows' bf16 values land where the two parts of the row will be (256 bytes either way), all requested together.
    {
        const int c = lane & 15;
#pragma unroll 4
        for (int j = 0; j < 32; j += 2) {
            const int row = j + (lane >> 4);
            const int64_t from = __shfl_sync(0xffffffffu, at, row) + c * 8;
            const bool in = row < valid;
            cp_async16(ptx::smem_u32(q) + (c >> 3) * apart + row * 128 + (((c & 7) ^ (row & 7)) << 4), src + (in ? from : 0), in);
        }
        cp_async_wait_all();
        __syncwarp();
    }
    // 4 lanes a row, 32 columns each.
    const int quarter = lane & 3;
#pragma unroll 1
    for (int row = lane >> 2; row < 32; row += 8) {
        uint8_t* const to_row = q + row * 128;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = *reinterpret_cast<const uint4*>(to_row + (quarter >> 1) * apart + ((((quarter & 1) * 4 + i) ^ (row & 7)) << 4));
        __syncwarp();  // before the row's other lanes write over them
        uint32_t top = max(max(top_bits(v[0]), top_bits(v[1])), max(top_bits(v[2]), top_bits(v[3])));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // (a zero row's exponent is as good as any)
        const uint32_t e = top == 0 ? 127 : min(max(top >> 7, 8u), 253u);
        const float up = __uint_as_float((261 - e) << 23);  // 2^(134 - e)
        if (quarter == 0) scale(row, __uint_as_float((e - 7) << 23));
        const bool bad = top >= 0x7F80u;  // NaN or infinite: the whole row is NaN
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float f[8];
                unpack_bf16x8(v[2 * i + (w >> 1)], f);
                float d[4];
                hi[w] = 0;
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const float x0 = f[(w & 1) * 4 + j] * up, x1 = f[(w & 1) * 4 + j + 1] * up;
                    const uint32_t pair = cvt_e4m3x2(x0, x1), back = e4m3x2_lo_to_f16x2(pair);
                    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&back));
                    d[j] = x0 - b.x;
                    d[j + 1] = x1 - b.y;
                    hi[w] |= pair << (8 * j);
                }
                lo[w] = cvt_e4m3x2(d[0], d[1]) | (cvt_e4m3x2(d[2], d[3]) << 16);
                if (bad) hi[w] = 0x7F7F7F7Fu;
            }
            uint8_t* const to = to_row + (((quarter * 2 + i) ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(to + apart) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// One item and where it lies in the unit list. A unit is kTok cached tokens of
// a row tile; an item counts kCost units beside its own.
struct Item {
    int b, h, rt;      // sequence, KV head, row tile
    int nq, q0, len;   // new tokens, first one's row in q, cached tokens
    int rts, tiles;    // row tiles of this sequence and units of each, kCost included
    int prefix;        // positions that every row sees (0 in a plain list)
    int skip;          // kMass: tiles left out behind the prefix's
    int64_t first;     // index of the item's first unit
};

// kScored: units are the tiles that the sequence's rows may see. kMass: those and the ones whose weights start from zero;
// an item has all the sequence's rows, and a token tile counts as often as they have 64 (at most 16 times).
enum class List { kPlain, kScored, kMass };
__device__ __forceinline__ int old_end(const AttnArgs& a, int b, int len, int nq) {  // positions before it keep their weight
    return !a.accumulate ? 0 : a.old_lens ? ld_dep_s32(a.old_lens + b) : len - nq;
}
__device__ __forceinline__ int mass_weight(int rows) { return min(max((rows + 63) / 64, 1), 16); }

template <int kTok, int kCost, List kList>
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
        it.prefix = 0;
        if constexpr (kList == List::kMass) {
            const int kept = old_end(a, b, len, it.nq);
            it.prefix = it.nq > 0 ? prefix_of(a.scores, b, len) : 0;
            const int lo = min(it.nq > 0 ? min(first_seen(a.scores, q0, len, it.nq, 0), kept) : kept, len);
            const Reach r = reach_of<kTok>(it.prefix, lo, len);
            it.skip = r.skip;
            it.rts = len > 0 && (it.nq > 0 || kept < len) ? 1 : 0;
            it.tiles = r.end * mass_weight(it.nq * a.group) + kCost;
        }
        if constexpr (kList == List::kScored) {
            it.prefix = prefix_of(a.scores, b, len);
            if (it.nq > 0) it.tiles = reach_of<kTok>(it.prefix, first_seen(a.scores, q0, len, it.nq, 0), len).end + kCost;
        }
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
                if constexpr (kList != List::kMass) a.split[blockIdx.x].parts = 0;
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

// What the rows of one row tile, row0 .. row0 + nrows - 1 of a sequence, see (kScored).
struct TileReach {
    Reach tiles;
    int lo, limit;  // no row needs a mask in [lo, limit), but for the prefix
};
template <int kTok>
__device__ __forceinline__ TileReach tile_reach(const AttnArgs& a, const Item& it, int row0, int nrows) {
    const int q_first = row0 / a.group, q_last = (row0 + nrows - 1) / a.group;
    TileReach r;
    r.tiles = reach_of<kTok>(it.prefix, first_seen(a.scores, it.q0, it.len, it.nq, q_first), it.len - it.nq + q_last + 1);
    r.lo = first_seen(a.scores, it.q0, it.len, it.nq, q_last);
    r.limit = it.len - it.nq + q_first + 1;
    return r;
}

// The kernel for wide row tiles of head size 128 (kv_attention_tc.cu); the
// caller launches the join of the split items after it.
cudaError_t launch_attention_tc(const AttnArgs& a, int num_sms, cudaStream_t stream);

// The weights of cached tokens from many rows of head size 128 (kv_mass_tc.cu).
cudaError_t launch_mass_tc(const AttnArgs& a, int num_sms, cudaStream_t stream);

}  // namespace fp8act
