// What the two kernels of the choice of blocks share (select_blocks.cu, select_tiles.cu): a query's exact
// scores, the best of them, and reductions over a warp.
#pragma once

#include <cfloat>

#include "mma_tiles.cuh"
#include "selected.h"

namespace dfs {

struct Choice {
    SelectShape s;
    const __nv_bfloat16 *q, *means;
    int32_t sink, local;
    int32_t* blocks;
    int32_t tile;                  // queries of a block of threads: 32, or fewer for many key blocks
    int32_t stride;                // floats of a query's scores
};
// many queries, top up to kTilesTop (select_tiles.cu), which a list of 32 candidates in shared memory serves; for more a
// warp a query (16 x 16384 queries of 256 blocks: 111 us with top 20, 215 with 21, 426 with 32, 368 with 33, 355 with 64)
constexpr int kTilesTop = 20;
int launch_select_tiles(const Choice& a, cudaStream_t stream);

#ifdef __CUDACC__
namespace select {

using tiles::kFull;

// Norms are kept away from 0, where squares of denormal size are lost.
constexpr float kLeastNorm = 1e-16f;

// The bits of a sum of squares, which order as it does (infinities and NaN above all).
__device__ __forceinline__ float squares(uint32_t w, float sum) {
    const float x = __uint_as_float(w << 16), y = __uint_as_float(w & 0xffff0000u);
    return fmaf(y, y, fmaf(x, x, sum));
}

// |Q| |K| of a query whose group's heads have squares adding up to `query`, against means with up to `mean`; K is the mean
// once for each head.  No sum of products of theirs is larger.
__device__ __forceinline__ float reach_of(int G, float query, float mean) {
    return sqrtf((float)G) * (sqrtf(query) + kLeastNorm) * (sqrtf(mean) + kLeastNorm);
}
// Twice what a score in fp32 is off by at most (select_blocks.cu), and what its 64 G products may lose below 2^-126.
__device__ __forceinline__ float twice_eps(int G, float reach) { return (float)G * (2.02f * 68.f * 1.1920929e-7f * reach + 1e-35f); }

// x + y = sum + error, without rounding (Knuth's two-sum)
__device__ __forceinline__ float two_sum(float x, float y, float* error) {
    const float s = __fadd_rn(x, y), z = __fsub_rn(s, x);
    *error = __fadd_rn(__fsub_rn(x, __fsub_rn(s, z)), __fsub_rn(y, z));
    return s;
}

// The score as fp64 would have it or better, in every lane; NaN counts as -infinity.  Products of two bf16 values
// are exact in fp32 from 2^-126 on, and their sum is held in three fp32 parts (the machine's fp64 rate is a sixtieth of
// its fp32's: with 16 heads a group most of the choice's time went there); in fp64 where a product is smaller, and not
// 0 by one of its factors, or so large that a sum may not be finite.
__device__ __forceinline__ double exact_score(const uint32_t* q, int64_t head_words, int G, const uint32_t* mean, int lane) {
    const uint32_t w = mean[lane];
    const float m0 = __uint_as_float(w << 16), m1 = __uint_as_float(w & 0xffff0000u);
    float a = 0.f, b = 0.f, c = 0.f;
    bool exact = true;
    auto add = [&](float x, float m) {
        const float product = __fmul_rn(x, m);
        exact &= (fabsf(product) >= FLT_MIN && fabsf(product) < 1e30f) || x == 0.f || m == 0.f;
        float e, f;
        a = two_sum(a, product, &e);
        b = two_sum(b, e, &f);
        c = __fadd_rn(c, f);
    };
#pragma unroll 4
    for (int h = 0; h < G; ++h) {
        const uint32_t x = q[h * head_words + lane];
        add(__uint_as_float(x << 16), m0);
        add(__uint_as_float(x & 0xffff0000u), m1);
    }
    double t = (double)a + ((double)b + (double)c);
    if (!__all_sync(kFull, exact)) {
        t = 0.0;
#pragma unroll 1
        for (int h = 0; h < G; ++h) {
            const uint32_t x = q[h * head_words + lane];
            t += (double)__uint_as_float(x << 16) * (double)m0 + (double)__uint_as_float(x & 0xffff0000u) * (double)m1;
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) t += __shfl_xor_sync(kFull, t, off);
    return t == t ? t : -INFINITY;
}

// The best `want` (up to 64) of the scores handed in by rising index, two places a lane.
struct Best {
    double t[2];
    int c[2];
    int have = 0;

    __device__ __forceinline__ void put(int place, double x, int index, int lane) {
        if (lane != (place & 31)) return;
        t[place >> 5] = x;
        c[place >> 5] = index;
    }
    __device__ void offer(double x, int index, int want, int lane) {
        if (have < want) return put(have++, x, index, lane);
        // the worst: the least score, among equals the highest index
        double wt = INFINITY;
        int wc = -1, wp = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (lane + 32 * j < want && (wc < 0 || t[j] < wt || (t[j] == wt && c[j] > wc))) {
                wt = t[j];
                wc = c[j];
                wp = lane + 32 * j;
            }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            const double ot = __shfl_xor_sync(kFull, wt, off);
            const int oc = __shfl_xor_sync(kFull, wc, off), op = __shfl_xor_sync(kFull, wp, off);
            if (oc >= 0 && (wc < 0 || ot < wt || (ot == wt && oc > wc))) {
                wt = ot;
                wc = oc;
                wp = op;
            }
        }
        if (x > wt) put(wp, x, index, lane);
    }
};

// Over a warp, of numbers.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_min(float x) {
    float y;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t ballot2(bool a, bool b) {
    const unsigned lo = __ballot_sync(kFull, a), hi = __ballot_sync(kFull, b);
    return lo | (uint64_t)hi << 32;
}

// The want-th largest of a warp's values, two a lane (-infinity: none), more than `want` of them: by
// bisection on values.
__device__ __forceinline__ float nth_largest(const float (&x)[2], int want) {
    float lo = fminf(x[0] > -INFINITY ? x[0] : INFINITY, x[1] > -INFINITY ? x[1] : INFINITY);
    float hi = fmaxf(x[0] < INFINITY ? x[0] : -INFINITY, x[1] < INFINITY ? x[1] : -INFINITY);
    lo = warp_min(lo);
    hi = warp_max(hi);
    if (__popcll(ballot2(x[0] >= hi, x[1] >= hi)) >= want) return hi;
    for (;;) {                               // more than `want` reach lo, fewer reach hi
        const float mid = lo + 0.5f * (hi - lo);
        if (!(mid > lo && mid < hi)) return lo;
        const int n = __popcll(ballot2(x[0] >= mid, x[1] >= mid));
        if (n == want) return warp_min(fminf(x[0] >= mid ? x[0] : INFINITY, x[1] >= mid ? x[1] : INFINITY));
        if (n > want) lo = mid;
        else hi = mid;
    }
}

// A query's forced blocks among its first nv: those below `sink`, and near0 .. near1 - 1 (none below sink).
struct Forced {
    int sink, near0, near;         // near = near1 - near0
    __device__ __forceinline__ Forced(int sinks, int local, int home, int nv) {
        sink = min(sinks, nv);
        near0 = max(home - local + 1, sink);
        near = max(min(home + local, nv) - near0, 0);
    }
    __device__ __forceinline__ int count() const { return sink + near; }
    __device__ __forceinline__ int at(int x) const { return x < sink ? x : near0 + x - sink; }
    __device__ __forceinline__ bool has(int c) const { return c < sink || (unsigned)(c - near0) < (unsigned)near; }
    // of them below c
    __device__ __forceinline__ int below(int c) const { return c < sink ? c : sink + min(max(c - near0, 0), near); }
};

}  // namespace select
#endif

}  // namespace dfs
