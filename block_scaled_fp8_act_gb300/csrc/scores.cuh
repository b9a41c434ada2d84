// Scores that are more than a scaled product, for the attention kernels and the
// accumulated weights: a cap, a bias by distance, and which positions a row sees.
// A changed score times Scores::unit is an exponent of 2: the unit is the cap, or
// 1. With masks alone (kMasked) the rows' scales stay factors of the exponent.
#pragma once

#include "decoder_util.cuh"
#include "kernels.h"

namespace fp8act {

// Scores are carried in units of the cap while there is one, so that its division is the queries' scale's and its product
// the exponent's: tanh(z) of a thread's scores, kPairs pairs that `get` gives and `set` takes; the whole warp calls it. To
// within 2^-22 of a score up to |z| = 0.625 and 2^-21 beyond. Near zero, where most scores are, tanh(z) / z is a polynomial
// in z^2 (interpolated at the Chebyshev points of [0, 0.625^2], 1.0e-7 off in fp32), 3.5 two-wide instructions a score;
// 1 - 2 / (1 + e^2z) takes two of the special functions' and loses a small score's bits in the difference, so it is for
// warps that hold a larger one. Which form a score gets goes by its own value alone.
template <int kPairs, class Get, class Set>
__device__ __forceinline__ void cap_scores(Get get, Set set) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const float2 z = get(i);
        most = fmaxf(most, fmaxf(fabsf(z.x), fabsf(z.y)));
    }
    const bool far = __any_sync(0xffffffffu, most > 0.625f);
    auto near = [&](const float2& z) {
        const float2 u = __fmul2_rn(z, z);
        auto both = [](float x) { return make_float2(x, x); };
        float2 p = __ffma2_rn(both(-0.005657135f), u, both(0.020588191f));
        p = __ffma2_rn(p, u, both(-0.05372011f));
        p = __ffma2_rn(p, u, both(0.13331114f));
        p = __ffma2_rn(p, u, both(-0.3333326f));
        return __fmul2_rn(z, __ffma2_rn(p, u, both(1.0f)));
    };
    if (!far) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) set(i, near(get(i)));
        return;
    }
    auto any = [](float z) {  // (one at a time: in pairs the tcgen05 kernel spilled half as much again)
        const float u = z * z;
        float p = fmaf(-0.005657135f, u, 0.020588191f);
        p = fmaf(p, u, -0.05372011f);
        p = fmaf(p, u, 0.13331114f);
        p = fmaf(p, u, -0.3333326f);
        p = z * fmaf(p, u, 1.0f);
        const float e = ex2(fabsf(z) * 2.8853900817779268f);  // 2 / ln 2
        return fabsf(z) > 0.625f ? copysignf(fmaf(-2.0f, rcp_approx_ftz(1.0f + e), 1.0f), z) : p;
    };
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const float2 z = get(i);
        set(i, make_float2(any(z.x), any(z.y)));
    }
}

// How a row (new token, query head) scores and what it sees: positions below the sequence's prefix, and [lo, limit).
struct __align__(16) RowScore {
    float qs;  // of the query's scaling, with the softmax's scale, over the unit
    int lo, limit;
    float slope;
};

// The first position that new token qi of a sequence with `len` cached tokens, `nq` of them new, sees behind the prefix.
__device__ __forceinline__ int first_seen(const Scores& s, int q0, int len, int nq, int qi) {
    int64_t lo = 0;
    if (s.window > 0) lo = static_cast<int64_t>(len) - nq + qi - s.window + 1;
    if (s.first) lo = max(lo, static_cast<int64_t>(ld_dep_s32(s.first + q0 + qi)));
    return static_cast<int>(max(lo, int64_t{0}));
}

// Row `row` of a sequence's (rows past its last are as that one), of KV head h.
// Its qs comes from the staging of the queries.
__device__ __forceinline__ RowScore row_score(const Scores& s, int q0, int len, int nq, int group, int h, int row, unsigned int* error) {
    const int qi = min(row / group, nq - 1);
    RowScore r;
    r.qs = 0.0f;
    r.lo = first_seen(s, q0, len, nq, qi);
    r.limit = len - nq + qi + 1;
    r.slope = s.slopes ? ld_dep_f32(s.slopes + h * group + row % group) * (1.4426950408889634f / s.unit) : 0.0f;
    if (s.first && qi > 0 && ld_dep_s32(s.first + q0 + qi) < ld_dep_s32(s.first + q0 + qi - 1)) atomicOr(error, 1u);
    return r;
}

// A row's qs from its power of two; bounded, so that a tiny cap of huge queries is still 0 times a product of 0.
__device__ __forceinline__ float row_scale(float step, float scale) { return fminf(fmaxf(step * scale, 0x1p-126f), 3e38f); }

__device__ __forceinline__ int prefix_of(const Scores& s, int b, int len) {
    return s.prefix ? min(max(ld_dep_s32(s.prefix + b), 0), len) : 0;
}

// Tiles of kTok positions that a sequence's or a row tile's rows may see: [0, prefix) and then from `skip` further on.
// Tile v of them is at position at(v) * kTok.
struct Reach {
    int prefix_tiles, skip, end;
    __device__ __forceinline__ int at(int v) const { return v < prefix_tiles ? v : v + skip; }
};
template <int kTok>
__device__ __forceinline__ Reach reach_of(int prefix, int lo, int limit) {
    Reach r;
    r.prefix_tiles = (prefix + kTok - 1) / kTok;
    const int start = max(lo / kTok, r.prefix_tiles);
    r.skip = start - r.prefix_tiles;
    r.end = r.prefix_tiles + max((max(limit, 0) + kTok - 1) / kTok - start, 0);
    return r;
}

// Whether positions [pos, pos + n) hold one that some row of a row tile does not see; `lo` is its last row's, `limit` its
// first one's.
__device__ __forceinline__ bool on_edge(int pos, int n, int prefix, int lo, int limit) {
    if (lo <= prefix) return pos + n > max(limit, prefix);
    return pos + n > prefix && (pos < lo || pos + n > limit);
}

}  // namespace fp8act
