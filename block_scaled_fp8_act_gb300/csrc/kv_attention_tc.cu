// Attention over the E4M3 cache for wide row tiles (verify steps, chunks of a
// prompt; head size 128) on the 5th-generation tensor cores. The mathematics,
// the masks and the work list are those of kv_attention.cu; a unit is a row
// tile x 128 cached tokens.
//
// S = Q K^T takes the cached codes as they are (kind::f8f6f4, fed by tensor
// copies, no conversion): a query row, scaled by a power of two so that its
// largest value is in [128, 256), is the sum of two E4M3 rows, hi = E4M3(q) and
// lo = E4M3(q - hi), whose products add up in one accumulator. A bf16 value
// has 8 significant bits and each part 4, so hi + lo is exact down to 2^-9 of
// the row's largest value, and within 2^-17 of it below. O += P V runs in f16
// (kind::f16; an E4M3 P would have 4 bits): four warps widen the value codes
// times s_v 2^6 / R, R the power of two below the largest s_v so far, so that
// values keep their 11 bits down to 2^-20 of the largest; the weights, scaled by
// 2^6 too, keep theirs down to 2^-20 of the row's reference, and go from
// registers to tensor memory over the scores they came from. A token whose value
// scale is NaN (poisoned) gets zero values and a NaN key scale, which reaches
// the rows that see it and no other.
//
// Two score tiles are in flight, each with a warpgroup whose warps own 32 rows:
// with more than 128 rows they are the two halves of a 256-row tile on the same
// cached tokens, which are loaded and widened once for both; else they are the
// even and the odd token tiles of one row tile of up to 128 rows, whose two
// results join in tensor memory at the end (warps without rows skip the
// softmax). While one warpgroup works the tensor cores serve the other. A
// row's reference moves only when a score passes it by 2^8, so the output
// accumulator is seldom rescaled.
//
// A softmax thread has 2 of every 8 columns of its rows (the accumulator layout
// of the warp-level MMAs), 16 rows of the warp at a time: with a row per thread
// every thread read all 128 key scales from shared memory, a third of what moves
// there in all (16 tokens x 6 heads over 131072: 81.7 us, now 62.0; 512 over
// 16384: 135.7 and 122.8, with the queries' way through shared memory below; now
// 60.0 and 117.6 with a faster join).
// The two passes of 16 rows are a loop: the hot code of the roles that share an
// instruction cache stays small.
//
// What bounds it: the chain of a score tile, 128 rows x 128 tokens, of about 4900
// clocks: S 520 clocks, softmax 2500, weights through tensor memory, P V 520, and
// the waits between. Two such chains keep the tensor cores half busy (512 tokens
// x 24 heads over 16384: 863 TFLOP/s, S counted once); there is no
// room for a third, whose scores would take the columns of an output, and score
// tiles of 64 tokens do not help, since an MMA 64 columns wide takes longer than
// one of 128 (104 clocks against 64). Measured and slower: the softmax on 16
// warps with 96 registers, the weights taken first and the maximum checked after,
// a third widened buffer. The kernel spills (364 bytes of stores and 468 of loads
// a thread with one row tile, 280 and 328 with two); of which role is not known.
//
// Every wait is bounded by wall time. The first that gives up sets the error
// word and the CTA's abort flag; every role then leaves its loop, copies and
// MMAs in flight are waited for, tensor memory is freed.
#include <atomic>

#include "host_util.h"
#include "kv_attention.cuh"
#include "tc_ptx.cuh"

namespace fp8act {

__device__ unsigned int g_attn_timeout;

namespace {

constexpr int kTok = 128;
constexpr int kD = 128;
constexpr int kLeastUnits = 2;  // least share of a CTA

constexpr int kThreads = 512;  // warps 0 keys, 1 values, 2 MMA; 4..7 widening; 8..11 and 12..15 softmax
// The softmax warps take what the other two warpgroups hand back of their
// registers, 256 x 64 + 256 x 192 = 512 x 128, exactly the launch's.
constexpr int kRegsOther = 64, kRegsSoftmax = 192;
static_assert(256 * kRegsOther + 256 * kRegsSoftmax <= kThreads * 128, "register split exceeds the launch's registers");
constexpr int kTileBytes = kTok * kD;
constexpr int kKSets = 4;  // tiles whose key scales are at hand (the values widened are at most 2 behind)

template <bool kPair>  // two row tiles of 128 on the same tokens
struct Tc {
    // Units that an item counts beside its own, for its queries and its result. (Rows up to 128, 16 tokens x 6 heads over
    // 131072: 5 units 63.6 us, 8 62.0; two row tiles, 512 tokens over 16384: 4 units 122.8 us, 6 126.5.)
    static constexpr int kItemCost = kPair ? 4 : 8;
    using Work = Units<kTok, kItemCost>;
    static constexpr int kQTiles = kPair ? 2 : 1;
    static constexpr int kKStages = kPair ? 3 : 4;
    static constexpr int kVStages = kPair ? 2 : 3;
    static constexpr int kQ = 0;                                   // per tile: hi, lo
    static constexpr int kK = kQ + kQTiles * 2 * kTileBytes;
    static constexpr int kV8 = kK + kKStages * kTileBytes;
    static constexpr int kV16 = kV8 + kVStages * kTileBytes;       // 2 buffers of two 64-column halves
    static constexpr int kScale8 = kV16 + 2 * 2 * kTileBytes;      // per value stage: key scales, value scales
    static constexpr int kScaleK = kScale8 + kVStages * 2 * kTok * 4;  // ring of kKSets: key scales
    static constexpr int kR = kScaleK + kKSets * kTok * 4;         // the same ring: R
    static constexpr int kQScale = kR + kKSets * 4;
    static constexpr int kML = kQScale + kQTiles * 128 * 4;        // second result's (maximum, sum, R) per row
    static constexpr int kBytes = kML + 128 * 16 + 1024;           // (the base is rounded up to 1024)
};

struct TcExtra {
    unsigned long long wait_ns;  // bound of every wait
    int withhold;                // test hook: the CTA's first key tile is never requested
};

__device__ __forceinline__ void st_16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
// Score tiles move in the layout of the warp-level MMAs' accumulators: lane l holds rows l / 4 (+ 8) of 16 and of every 8
// columns two, 2 (l % 4) and the next. 128 columns of the 16 lanes at `taddr`: v[4 n + 2 i + j] is row l / 4 + 8 i,
// column 8 n + 2 (l % 4) + j.
__device__ __forceinline__ void ld_16x256b_x16(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}
// The same layout with a column holding two f16: r[2 n + i] is row l / 4 + 8 i, column 4 n + l % 4.
__device__ __forceinline__ void st_16x128b_x16(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x16.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
        "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The whole warp executes these, and one elected lane issues the MMA.
// D[tmem] (+)= A[tmem] x B[smem desc], f16 with fp32 accumulation.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p, e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D[tmem] (+)= A[smem desc] x B[smem desc], E4M3 with fp32 accumulation.
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n"
        ".reg .pred p, e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t mbar) {
    asm volatile(
        "{\n"
        ".reg .pred e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
        "}\n" ::"r"(mbar)
        : "memory");
}

// Descriptor of the widened values as the N x K operand with N contiguous
// (128-byte swizzle): blocks of 64 columns x 8 tokens, column blocks 16 KB
// apart (leading byte offset), token blocks 1 KB apart (stride byte offset).
__device__ __forceinline__ uint64_t desc_values(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(kTileBytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
constexpr uint32_t kIdescScores = tc::idesc_e4m3_f32(128, kTok);
constexpr uint32_t kIdescValues = (1u << 4)                                   // D fp32; A, B f16
                                  | (1u << 16)                                // B with N contiguous
                                  | (static_cast<uint32_t>(kD >> 3) << 17) | (128u >> 4 << 24);

__device__ __forceinline__ void load_tokens(uint32_t dst, const CUtensorMap* map, uint32_t bar, int line) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(0), "r"(line)
        : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrive on `bar` (one of its expected arrivals) once this thread's cp.asyncs so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float4 lds_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Where the key scale of a tile's token lies, so that a lane reads those of its columns 4 at a time.
__device__ __forceinline__ int scale_at(int t) { return (t & ~15) | ((t >> 1 & 3) << 2) | ((t >> 3 & 1) << 1) | (t & 1); }

template <typename T>
__device__ __forceinline__ void swap(T& a, T& b) {
    const T c = a;
    a = b;
    b = c;
}

template <bool kPair>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tc_kernel(const __grid_constant__ AttnArgs a,
                                                                      const __grid_constant__ CUtensorMap k_map,
                                                                      const __grid_constant__ CUtensorMap v_map,
                                                                      const TcExtra x) {
    using C = Tc<kPair>;
    using Work = typename C::Work;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - ptx::smem_u32(smem_raw));
    __shared__ typename Work::Scratch scratch;
    __shared__ __align__(8) uint64_t bars[2 * C::kKStages + 2 * C::kVStages + 2 * 2 + 3 * 2 + 4 + kKSets];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const uint32_t k_full = ptx::smem_u32(bars), k_empty = k_full + 8 * C::kKStages;
    const uint32_t v8_full = k_empty + 8 * C::kKStages, v8_empty = v8_full + 8 * C::kVStages;
    const uint32_t v16_full = v8_empty + 8 * C::kVStages, v16_empty = v16_full + 16;
    const uint32_t s_full = v16_empty + 16, p_full = s_full + 16, pv_done = p_full + 16;  // [slot]
    const uint32_t q_full = pv_done + 16, item_done = q_full + 8, ml_full = item_done + 8, drain = ml_full + 8;
    const uint32_t ks_full = drain + 8;  // [set]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kKStages; ++i) {
            ptx::mbar_init(k_full + 8 * i, 1);
            ptx::mbar_init(k_empty + 8 * i, 1);
        }
        for (int i = 0; i < C::kVStages; ++i) {
            ptx::mbar_init(v8_full + 8 * i, 1 + 32);  // the copies' bytes and the scales' 32 lanes
            ptx::mbar_init(v8_empty + 8 * i, 4);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(v16_full + 8 * i, 4);
            ptx::mbar_init(v16_empty + 8 * i, 1);
            ptx::mbar_init(s_full + 8 * i, 1);
            ptx::mbar_init(p_full + 8 * i, 4);
            ptx::mbar_init(pv_done + 8 * i, 1);
        }
        ptx::mbar_init(q_full, kPair ? 8 : 4);
        ptx::mbar_init(item_done, 1);
        ptx::mbar_init(ml_full, 4);
        ptx::mbar_init(drain, 1);
        for (int i = 0; i < kKSets; ++i) ptx::mbar_init(ks_full + 8 * i, 4);
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 2) {
        tc::tmem_alloc(ptx::smem_u32(&s_tmem), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = s_tmem;  // columns: scores of slot 0 and 1, outputs of slot 0 and 1

    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    Item it;
    int64_t per, u, u_end;
    const bool any = Work::first_item(a, kLeastUnits, scratch, it, per, u, u_end);
    const int64_t u_begin = u;
    // Tiles used by the items before, K and V alike.
    uint32_t seq = 0;

    // A bounded wait by the whole warp; false once any wait of the CTA has run out.
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        // (the timer is far from the SM and is read only after a while)
        bool ok = ptx::mbar_try_wait(bar, parity);
        uint64_t start = 0;
        for (uint32_t n = 1; !ok; ++n) {
            ok = ptx::mbar_try_wait(bar, parity);
            if (!ok && n % 64 == 0) {
                const uint64_t now = ptx::globaltimer_ns();
                if (start == 0) start = now;
                if (s_abort || now - start > x.wait_ns) break;
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) {
            s_abort = 1;
            atomicOr(&g_attn_timeout, 1u);
        }
        return ok;
    };

    // What every role knows of an item.
    struct Span {
        int row0, nrows, slots;  // rows of the row tile; row halves in use (kPair) or 2
        int f0, n;               // first token tile and how many
        bool whole;              // no other CTA works on the item
    };
    auto span_of = [&]() {
        Span s;
        const int t0 = static_cast<int>(u - it.first);
        const int64_t item_end = it.first + it.tiles;
        const int t1 = static_cast<int>((item_end < u_end ? item_end : u_end) - it.first);
        s.row0 = it.rt * a.rows;
        s.nrows = min(it.nq * a.group - s.row0, a.rows);
        s.slots = kPair && s.nrows <= 128 ? 1 : 2;
        const int seen = max(it.len - it.nq + (s.row0 + s.nrows - 1) / a.group + 1, 0);
        s.f0 = max(t0 - C::kItemCost, 0);
        s.n = max(min((seen + kTok - 1) / kTok, t1 - C::kItemCost) - s.f0, 0);
        s.whole = t0 == 0 && t1 == it.tiles;
        return s;
    };
    auto next = [&](const Span& s) -> bool {  // to the next item of this CTA
        seq += s.n;
        u = it.first + it.tiles;
        if (u >= u_end) return false;
        Work::next_item(a, it);
        return true;
    };

    if (warp < 8) {
    tc::regs_decrease<kRegsOther>();
    if (!any) {
        // nothing to do: only tensor memory to free
    } else if (warp < 2) {
        // ------------------------------------------------------------ copies
        const bool values = warp == 1;
        const int stages = values ? C::kVStages : C::kKStages;
        const uint32_t full = values ? v8_full : k_full, empty = values ? v8_empty : k_empty;
        const uint32_t ring = base + (values ? C::kV8 : C::kK);
        const CUtensorMap* map = values ? &v_map : &k_map;
        const int page = 1 << a.c.page_log2, box = min(page, kTok);
        bool ok = true;
        uint32_t n = 0;  // tiles requested
        while (ok) {
            const Span s = span_of();
            const int* table = a.table + it.b * a.table_stride;
            // Pages of 4 tiles at a time, one per 16 tokens and lane, looked up one such span ahead.
            auto look_up = [&](int t) -> int {
                const int pos = t * kTok + lane * 16;
                if (t >= s.f0 + s.n || pos >= it.len) return -1;
                const int p = ld_dep_s32(table + (pos >> a.c.page_log2));
                if (p >= 0 && p < a.c.num_pages) return p;
                atomicOr(a.index_error, 1u);
                return -1;
            };
            int ahead = look_up(s.f0), now = -1;
            for (int i = 0; i < s.n && ok; ++i, ++n) {
                if ((i & 3) == 0) {
                    now = ahead;
                    ahead = look_up(s.f0 + i + 4);
                }
                const uint32_t round = values ? n / C::kVStages : n / C::kKStages;  // (constant divisors)
                const uint32_t stage = n - round * stages, bar = full + 8 * stage;
                if (round > 0 && !(ok = wait(empty + 8 * stage, (round - 1) & 1))) break;
                const int pos = (s.f0 + i) * kTok;
                // Lane j < 128 / box: copy j of the tile, if it holds a token.
                const int mine = __shfl_sync(0xffffffffu, now, (i & 3) * 8 + min(lane * box / 16, 7));
                const bool copy = lane < kTok / box && pos + lane * box < it.len && mine >= 0;
                const uint32_t copies = __ballot_sync(0xffffffffu, copy);
                const bool withheld = x.withhold && !values && n == 0;
                if (lane == 0 && !withheld) ptx::mbar_arrive_expect_tx(bar, __popc(copies) * box * kD);
                __syncwarp();
                if (copy && !withheld) {
                    const int64_t token = ((static_cast<int64_t>(mine) * a.c.heads + it.h) << a.c.page_log2) +
                                          ((pos + lane * box) & (page - 1));
                    load_tokens(ring + stage * kTileBytes + lane * box * kD, map, bar, static_cast<int>(token));
                }
                if (values) {  // both scales travel with the values
                    const uint32_t dst = base + C::kScale8 + stage * 2 * kTok * 4;
#pragma unroll
                    for (int j = 0; j < kTok / 32; ++j) {
                        const int t = j * 32 + lane;
                        const int p = __shfl_sync(0xffffffffu, now, (i & 3) * 8 + t / 16);
                        const bool in = p >= 0 && pos + t < it.len;
                        const int64_t at =
                            in ? ((static_cast<int64_t>(p) * a.c.heads + it.h) << a.c.page_log2) + ((pos + t) & (page - 1)) : 0;
                        cp_async4(dst + t * 4, a.c.k_scale + at, in);
                        cp_async4(dst + kTok * 4 + t * 4, a.c.v_scale + at, in);
                    }
                    cp_async_arrive(bar);
                }
            }
            if (!ok || !next(s)) break;
        }
        // Every copy must have landed before the CTA leaves (its consumer has usually seen it).
        for (uint32_t i = n > stages ? n - stages : 0; i < n; ++i)
            if (!(x.withhold && !values && i == 0) &&
                !ptx::mbar_wait(full + 8 * (i % stages), (i / stages) & 1) && lane == 0)
                atomicOr(&g_attn_timeout, 2u);
    } else if (warp == 2) {
        // --------------------------------------------------------------- MMA
        bool ok = true;
        uint32_t item = 0;
        uint32_t waited[2] = {0, 0};  // weight tiles waited for per slot
        while (ok) {
            const Span s = span_of();
            const int depth = s.slots;                            // score tiles in flight
            const int jobs = kPair ? s.n * s.slots : s.n;
            auto slot_of = [&](int j) { return depth == 2 ? j & 1 : 0; };
            auto tile_of = [&](int j) { return kPair ? j >> (depth - 1) : j; };  // (depth is 1 or 2)
            auto first_use = [&](int j) { return !kPair || slot_of(j) == 0; };
            auto last_use = [&](int j) { return !kPair || slot_of(j) == s.slots - 1; };
            auto keys = [&](int j) {  // wait for the keys of score tile j
                const uint32_t n = seq + tile_of(j);
                if (j < jobs && first_use(j)) ok = wait(k_full + 8 * (n % C::kKStages), (n / C::kKStages) & 1);
                return ok;
            };
            auto scores = [&](int j) {
                const int slot = slot_of(j);
                const uint32_t stage = (seq + tile_of(j)) % C::kKStages;
                const uint32_t q = base + C::kQ + (kPair ? slot : 0) * 2 * kTileBytes, k = base + C::kK + stage * kTileBytes;
                const uint64_t q_desc = tc::desc_kmajor_sw128(q), k_desc = tc::desc_kmajor_sw128(k);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int i = 0; i < kD / 32; ++i)  // (a descriptor counts 16 bytes)
                        mma_e4m3_ss(tmem + slot * 128, q_desc + (part * kTileBytes + 32 * i) / 16, k_desc + 2 * i, kIdescScores,
                                    part + i > 0 ? 1u : 0u);
                commit_elected(s_full + 8 * slot);
                if (last_use(j)) commit_elected(k_empty + 8 * stage);
            };
            if (!(ok = wait(q_full, item & 1))) break;
            tc::fence_after_sync();
            for (int j = 0; j < depth && j < jobs && keys(j); ++j) scores(j);
            for (int j = 0; j < jobs && ok; ++j) {
                const int slot = slot_of(j);
                const uint32_t buf = (seq + tile_of(j)) & 1;
                if (first_use(j) && !(ok = wait(v16_full + 8 * buf, (seq + tile_of(j)) >> 1 & 1))) break;
                if (!keys(j + depth) || !(ok = wait(p_full + 8 * slot, waited[slot]++ & 1))) break;
                tc::fence_after_sync();
                const uint64_t v_desc = desc_values(base + C::kV16 + buf * 2 * kTileBytes);
                const bool fresh = kPair ? tile_of(j) == 0 : j < 2;
#pragma unroll
                for (int i = 0; i < kTok / 16; ++i)
                    mma_f16_ts(tmem + 256 + slot * 128, tmem + slot * 128 + 8 * i, v_desc + 2048 * i / 16, kIdescValues,
                               fresh && i == 0 ? 0u : 1u);
                commit_elected(pv_done + 8 * slot);
                if (last_use(j)) commit_elected(v16_empty + 8 * buf);
                if (j + depth < jobs) scores(j + depth);
            }
            if (!ok) break;
            commit_elected(item_done);
            ++item;
            if (!next(s)) break;
        }
        // No MMA may still run when tensor memory is freed or the CTA leaves.
        commit_elected(drain);
        if (!ptx::mbar_wait(drain, 0)) atomicOr(&g_attn_timeout, 4u);
        __syncwarp();
    } else if (warp >= 4) {
        // ---------------------------------------------------------- widening
        const int t = threadIdx.x - 128;  // this thread's token of a tile
        bool ok = true;
        while (ok) {
            const Span s = span_of();
            float r_ref = 0x1p-100f;
            for (int i = 0; i < s.n && ok; ++i) {
                const uint32_t n = seq + i, stage = n % C::kVStages, buf = n & 1;
                if (!(ok = wait(v8_full + 8 * stage, (n / C::kVStages) & 1))) break;
                // R: the power of two below the largest value scale so far, the same in every warp.
                const float* sc = reinterpret_cast<const float*>(smem + C::kScale8 + stage * 2 * kTok * 4);
                uint32_t rb = 0;
#pragma unroll
                for (int j = 0; j < kTok / 32; ++j) rb = max(rb, scale_exponent(sc[kTok + j * 32 + lane]));
                rb = __reduce_max_sync(0xffffffffu, rb);
                r_ref = fmaxf(__uint_as_float(rb), r_ref);
                const bool in = (s.f0 + i) * kTok + t < it.len;  // else anything may be there
                const float sv = sc[kTok + t], sk = sc[t];
                const bool poisoned = !(fabsf(sv) < 3e38f);
                // The softmax may go ahead with the key scales.
                reinterpret_cast<float*>(smem + C::kScaleK)[(n % kKSets) * kTok + scale_at(t)] = poisoned ? sv : sk;
                if (t == 0) reinterpret_cast<float*>(smem + C::kR)[n % kKSets] = r_ref;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ks_full + 8 * (n % kKSets));
                if (n >= 2 && !(ok = wait(v16_empty + 8 * buf, ((n >> 1) - 1) & 1))) break;
                const float f = in && !poisoned ? sv * __fdividef(0x1p6f, r_ref) : 0.0f;
                const uint8_t* v8 = smem + C::kV8 + stage * kTileBytes + t * kD;
                uint8_t* v16 = smem + C::kV16 + buf * 2 * kTileBytes + t * 128;
                const __half2 f2 = __float2half2_rn(f);
                // code * s_v 2^6 / R in one f16 rounding of the product of the code and the f16 scale's two parts
                const __half2 g2 = __float2half2_rn(f - __low2float(f2));
                auto widen = [&](uint32_t h) {
                    const __half2 c = *reinterpret_cast<const __half2*>(&h);
                    const __half2 w = __hfma2(c, f2, __hmul2(c, g2));
                    return *reinterpret_cast<const uint32_t*>(&w);
                };
#pragma unroll 4
                for (int c = 0; c < 8; ++c) {
                    uint4 v = *reinterpret_cast<const uint4*>(v8 + ((c ^ (t & 7)) << 4));
                    if (!in || poisoned) v = make_uint4(0, 0, 0, 0);
                    const uint4 lo = make_uint4(widen(e4m3x2_lo_to_f16x2(v.x)), widen(e4m3x2_hi_to_f16x2(v.x)),
                                                widen(e4m3x2_lo_to_f16x2(v.y)), widen(e4m3x2_hi_to_f16x2(v.y)));
                    const uint4 hi = make_uint4(widen(e4m3x2_lo_to_f16x2(v.z)), widen(e4m3x2_hi_to_f16x2(v.z)),
                                                widen(e4m3x2_lo_to_f16x2(v.w)), widen(e4m3x2_hi_to_f16x2(v.w)));
                    uint8_t* half = v16 + (c >> 2) * kTileBytes;  // columns 64 (c / 4) ..
                    *reinterpret_cast<uint4*>(half + ((((c & 3) * 2) ^ (t & 7)) << 4)) = lo;
                    *reinterpret_cast<uint4*>(half + ((((c & 3) * 2 + 1) ^ (t & 7)) << 4)) = hi;
                }
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(v16_full + 8 * buf);
                    ptx::mbar_arrive(v8_empty + 8 * stage);
                }
            }
            if (!ok || !next(s)) break;
        }
    }
    } else {
        // ----------------------------------------------------------- softmax
        tc::regs_increase<kRegsSoftmax>();
        const int slot = (warp - 8) >> 2, quad = warp & 3;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const uint32_t t_s = lane_base + slot * 128, t_o = lane_base + 256 + slot * 128;
        const int row_in = (kPair ? slot * 128 : 0) + quad * 32 + lane;  // this thread's row of the row tile
        float* qscale = reinterpret_cast<float*>(smem + C::kQScale);
        float4* ml = reinterpret_cast<float4*>(smem + C::kML);
        uint32_t jobs_done = 0, item = 0;
        bool ok = any;
        while (ok) {
            const Span s = span_of();
            // Queries. The MMAs of the item before have read theirs (item_done was waited for).
            const int r = s.row0 + row_in;
            if (kPair || slot == 0) {
                // A warp's rows are those that its threads own. Their bf16 values land where the two parts of the row will be
                // (256 bytes either way), all requested together.
                uint8_t* const q = smem + C::kQ + slot * 2 * kTileBytes + quad * 32 * 128;
                {
                    const int qi = r / a.group, hg = r - qi * a.group;
                    const int64_t at = (it.q0 + qi) * a.q_stride + (it.h * a.group + hg) * kD;
                    const int c = lane & 15;
#pragma unroll 4
                    for (int j = 0; j < 32; j += 2) {
                        const int row = j + (lane >> 4);
                        const int64_t from = __shfl_sync(0xffffffffu, at, row) + c * 8;
                        const bool in = row_in - lane + row < s.nrows;
                        cp_async16(ptx::smem_u32(q) + (c >> 3) * kTileBytes + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                                   a.q + (in ? from : 0), in);
                    }
                    cp_async_wait_all();
                    __syncwarp();
                }
                // 4 lanes a row, 32 columns each.
                const int quarter = lane & 3;
#pragma unroll 1
                for (int row = lane >> 2; row < 32; row += 8) {
                    uint8_t* const at = q + row * 128;
                    uint4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = *reinterpret_cast<const uint4*>(at + (quarter >> 1) * kTileBytes +
                                                               ((((quarter & 1) * 4 + i) ^ (row & 7)) << 4));
                    __syncwarp();  // before the row's other lanes write over them
                    uint32_t top = max(max(top_bits(v[0]), top_bits(v[1])), max(top_bits(v[2]), top_bits(v[3])));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // (a zero row's exponent is as good as any)
                    const uint32_t e = top == 0 ? 127 : min(max(top >> 7, 8u), 253u);
                    const float up = __uint_as_float((261 - e) << 23);  // 2^(134 - e)
                    if (quarter == 0) qscale[row_in - lane + row] = fmaxf(__uint_as_float((e - 7) << 23) * a.scale_log2, 0x1p-126f);
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
                        uint8_t* const to = at + (((quarter * 2 + i) ^ (row & 7)) << 4);
                        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(to + kTileBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(q_full);
            }
            if (!(ok = wait(q_full, item & 1))) break;
            const bool rows_here = row_in - lane < s.nrows;                         // of this warp
            const int all_see = it.len - it.nq + (r - lane) / a.group + 1;          // positions below it need no mask
            // A thread works on 4 rows of its warp's 32, lane / 4 + 8 i, and a quarter of their columns. A row's reference:
            // the largest (q . k) s_k that moved it, not yet times qs, and what is subtracted from a score in the exponent.
            // The weights carry 2^kLift.
            constexpr float kLift = 6.0f;
            float qs[4], m[4], mq[4], l[4], r_ref = 0x1p-100f;
            int limit[4];  // first position that the row does not see
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = row_in - lane + (lane >> 2) + 8 * i;
                qs[i] = qscale[at];
                limit[i] = it.len - it.nq + (s.row0 + at) / a.group + 1;
                m[i] = kNegInf;
                mq[i] = 0.0f;
                l[i] = 0.0f;
            }
            // The value that row `lane` of the warp's has, from the threads' four.
            auto of_row = [&](const float (&x)[4]) {
                const int from = (lane & 7) * 4;
                float y = __shfl_sync(0xffffffffu, x[0], from);
#pragma unroll
                for (int i = 1; i < 4; ++i) {
                    const float z = __shfl_sync(0xffffffffu, x[i], from);
                    if (lane >> 3 == i) y = z;
                }
                return y;
            };
            const int first = kPair ? 0 : slot, step = kPair ? 1 : 2;
            const int last = slot < s.slots ? s.n : 0;
            int mine = 0;
            for (int i = first; i < last && ok; i += step, ++mine) {
                const uint32_t n = seq + i, set = n % kKSets;
                if (!(ok = wait(ks_full + 8 * set, (n / kKSets) & 1))) break;
                if (!(ok = wait(s_full + 8 * slot, jobs_done & 1))) break;
                tc::fence_after_sync();
                if (rows_here) {
                    const uint32_t ks = base + C::kScaleK + set * kTok * 4 + (lane & 3) * 16;
                    const float r_new = reinterpret_cast<const float*>(smem + C::kR)[set];
                    const int pos = (s.f0 + i) * kTok;
                    const bool edge = pos + kTok > all_see;
                    float alpha[4] = {1.0f, 1.0f, 1.0f, 1.0f};
                    bool rescale = false;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {  // rows lane / 4 + 16 h (+ 8)
                        const uint32_t t_half = t_s + (static_cast<uint32_t>(16 * h) << 16);
                        uint32_t v[64];
                        ld_16x256b_x16(t_half, v);
                        float4 k4[2];  // a step ahead
                        k4[0] = lds_v4(ks);
                        tc::wait_ld();
                        float top[2] = {kNegInf, kNegInf};
                        auto scaled = [&](bool masked) {
#pragma unroll
                            for (int j = 0; j < kTok / 16; ++j) {
                                if (j + 1 < kTok / 16) k4[(j + 1) & 1] = lds_v4(ks + (j + 1) * 64);
                                const float4 k = k4[j & 1];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int n = 2 * j + e;
#pragma unroll
                                    for (int x = 0; x < 2; ++x) {
                                        uint32_t &v0 = v[4 * n + 2 * x], &v1 = v[4 * n + 2 * x + 1];
                                        float2 y = __fmul2_rn(make_float2(__uint_as_float(v0), __uint_as_float(v1)),
                                                              e ? make_float2(k.z, k.w) : make_float2(k.x, k.y));
                                        if (masked) {
                                            const int end = limit[x] - pos - 2 * (lane & 3);
                                            if (8 * n >= end) y.x = kNegInf;
                                            if (8 * n + 1 >= end) y.y = kNegInf;
                                        }
                                        top[x] = fmaxf(top[x], fmaxf(y.x, y.y));
                                        v0 = __float_as_uint(y.x);
                                        v1 = __float_as_uint(y.y);
                                    }
                                }
                            }
                        };
                        if (edge)
                            scaled(true);
                        else
                            scaled(false);
                        // A reference moves only when the row's maximum passes it by 2^8.
                        bool moves = false;
#pragma unroll
                        for (int x = 0; x < 2; ++x) moves |= (top[x] - m[x]) * qs[x] > 8.0f;
                        if (__any_sync(0xffffffffu, moves)) {
                            rescale = true;
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int row = x;
                                top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
                                top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
                                if ((top[x] - m[row]) * qs[row] > 8.0f) {
                                    const float mq_new = fmaf(top[x], qs[row], -kLift);
                                    alpha[row] = ex2(fmaf(m[row], qs[row], -kLift) - mq_new);
                                    m[row] = top[x];
                                    mq[row] = mq_new;
                                }
                            }
                        }
                        uint32_t w[32];
                        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                        for (int n = 0; n < 16; ++n)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const float q = qs[x], ref = -mq[x];
                                const float2 y = __ffma2_rn(make_float2(__uint_as_float(v[4 * n + 2 * x]),
                                                                        __uint_as_float(v[4 * n + 2 * x + 1])),
                                                            make_float2(q, q), make_float2(ref, ref));
                                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                                sum[x] = __fadd2_rn(sum[x], e);
                                const __half2 e16 = __floats2half2_rn(e.x, e.y);
                                w[2 * n + x] = *reinterpret_cast<const uint32_t*>(&e16);
                            }
                        st_16x128b_x16(t_half, w);  // over the scores
#pragma unroll
                        for (int x = 0; x < 2; ++x) l[x] = fmaf(l[x], alpha[x], sum[x].x + sum[x].y);
                        // The other rows' values take the place of these.
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            swap(qs[x], qs[x + 2]);
                            swap(m[x], m[x + 2]);
                            swap(mq[x], mq[x + 2]);
                            swap(l[x], l[x + 2]);
                            swap(alpha[x], alpha[x + 2]);
                            swap(limit[x], limit[x + 2]);
                        }
                    }
                    const float gain = r_new == r_ref ? 1.0f : __fdividef(r_ref, r_new);
                    r_ref = r_new;
                    rescale |= gain != 1.0f;  // (the same in every lane)
                    if (mine > 0 && rescale) {
                        if (!(ok = wait(pv_done + 8 * slot, (jobs_done - 1) & 1))) break;
                        tc::fence_after_sync();
                        const float beta = of_row(alpha) * gain;
#pragma unroll 1
                        for (int c = 0; c < kD; c += 16) {
                            uint32_t o[16];
                            tc::ld_32x32b_x16(t_o + c, o);
                            tc::wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * beta);
                            st_16(t_o + c, o);
                        }
                    }
                    wait_st();
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(p_full + 8 * slot);
                ++jobs_done;
            }
            if (!ok) break;
            // The item's result: o = sum p s_v v / (2^6 / R) and, per row, its reference (log2) and sum of p, both with the
            // weights' 2^kLift.
            float mx, sum;
            {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
                    mq[i] = m[i] == kNegInf ? kNegInf : mq[i];
                }
                mx = of_row(mq);
                sum = of_row(l);
            }
            if (!kPair && slot == 1) {
                ml[row_in] = make_float4(mx, sum, r_ref, 0.0f);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ml_full);
            }
            if (!(ok = wait(item_done, item & 1))) break;
            tc::fence_after_sync();
            if (kPair || slot == 0) {
                float f0 = r_ref * 0x1p-6f, f1 = 0.0f;
                bool has1 = false;
                if (!kPair) {
                    if (!(ok = wait(ml_full, item & 1))) break;
                    const float4 other = ml[row_in];
                    const float most = fmaxf(mx, other.x), use = most == kNegInf ? 0.0f : most;
                    const float e0 = ex2(mx - use), e1 = ex2(other.x - use);
                    f0 *= e0;
                    f1 = other.z * 0x1p-6f * e1;
                    sum = sum * e0 + other.y * e1;
                    mx = most;
                    has1 = s.n > 1;
                }
                const bool has0 = s.n > 0 && slot < s.slots;
                const int part = 2 * blockIdx.x + (it.first > u_begin ? 1 : 0);
                const int qi = r / a.group, hg = r - qi * a.group;
                const int64_t orow = static_cast<int64_t>(it.q0 + qi) * (a.c.heads * a.group) + it.h * a.group + hg;
                const int64_t prow = static_cast<int64_t>(part) * a.rows + row_in;
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                if (rows_here) {
                    // Through the shared memory of the warp's own queries, which no MMA reads any more, so that 8 lanes
                    // store 32 columns of a row (with a lane per row each store touched 32 lines: 13000 clocks an item).
                    uint8_t* const stage = smem + C::kQ + slot * 2 * kTileBytes + quad * 32 * 128;
                    const float f = s.whole ? inv : 1.0f;
                    const int64_t mine_at = (s.whole ? orow : prow) * kD;
#pragma unroll 1
                    for (int c = 0; c < kD; c += 32) {
                        uint32_t o0[32], o1[32];
                        if (has0) tc::ld_32x32b_x32(t_o + c, o0);
                        if (has1) tc::ld_32x32b_x32(t_o + 128 + c, o1);
                        tc::wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            float o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                o[i] = has0 && f0 != 0.0f ? __uint_as_float(o0[j + i]) * f0 : 0.0f;
                                if (has1 && f1 != 0.0f) o[i] = fmaf(__uint_as_float(o1[j + i]), f1, o[i]);
                            }
                            *reinterpret_cast<float4*>(stage + lane * 128 + (((j >> 2) ^ (lane & 7)) << 4)) =
                                make_float4(o[0] * f, o[1] * f, o[2] * f, o[3] * f);
                        }
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int row = j * 4 + (lane >> 3), at = c + (lane & 7) * 4;
                            const float4 o = *reinterpret_cast<const float4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
                            const int64_t to = __shfl_sync(0xffffffffu, mine_at, row) + at;
                            if (row_in - lane + row < s.nrows) {
                                if (s.whole)
                                    *reinterpret_cast<uint2*>(a.out + (to >> 1)) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
                                else
                                    *reinterpret_cast<float4*>(a.part_o + to) = o;
                            }
                        }
                        __syncwarp();
                    }
                    if (row_in < s.nrows) {
                        if (!s.whole)
                            *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(mx, sum);
                        else if (a.lse)
                            a.lse[orow] = sum == 0.0f ? kNegInf : (mx + log2f(sum)) * 0.6931471805599453f;
                    }
                }
                if (!s.whole && u == it.first && warp == 8 && lane == 0) write_split(a, it, per, part, s.row0, s.nrows);
            }
            tc::fence_before_sync();
            ++item;
            if (!next(s)) break;
        }
    }

    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 2) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <bool kPair>
cudaError_t launch(const AttnArgs& a, int num_sms, cudaStream_t stream) {
    using C = Tc<kPair>;
    static std::atomic<bool> configured[64];
    int dev = 0;
    cudaGetDevice(&dev);
    auto kernel = kv_attention_tc_kernel<kPair>;
    if (!configured[dev & 63].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
        if (e != cudaSuccess) return e;
        configured[dev & 63].store(true, std::memory_order_relaxed);
    }
    // The cache as rows of one token and head; a copy is a page's tokens, 128 at most.
    const uint64_t tokens = static_cast<uint64_t>(a.c.num_pages) * a.c.heads << a.c.page_log2;
    const uint32_t box = 1u << a.c.page_log2 < kTok ? 1u << a.c.page_log2 : kTok;
    CUtensorMap k_map, v_map;
    if (!encode_tmap_2d_u8(&k_map, a.c.k, kD, tokens, kD, kD, box, true) ||
        !encode_tmap_2d_u8(&v_map, a.c.v, kD, tokens, kD, kD, box, true))
        return cudaErrorInvalidValue;
    const TcExtra x = {tile_wait_limit_ns(), tile_withhold_first_load() ? 1 : 0};
    return launch_dependent(kernel, dim3(num_sms), kThreads, C::kBytes, stream, 1, a, k_map, v_map, x);
}

}  // namespace

cudaError_t launch_attention_tc(const AttnArgs& a, int num_sms, cudaStream_t stream) {
    return a.rows > 128 ? launch<true>(a, num_sms, stream) : launch<false>(a, num_sms, stream);
}

unsigned int read_and_clear_attn_timeout() {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_timeout, sizeof(v)) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (v) {
        const unsigned int zero = 0;
        cudaMemcpyToSymbol(g_attn_timeout, &zero, sizeof(zero));
    }
    return v;
}

}  // namespace fp8act
