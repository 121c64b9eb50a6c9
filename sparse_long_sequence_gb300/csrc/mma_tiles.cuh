// Warp tiles of 64 keys against rows of 64 bf16 features on m16n8k16 products, with every operand
// held in registers as it is loaded from global memory (no shared memory, no transposes of the
// queries).
//
// Lane (g, t) = (lane / 4, lane % 4) of a warp loads 16 bytes at 8 t and at 32 + 8 t of row g of
// eight rows: words 0..3 and 4..7.  Step s of a product over the features takes words 2s and
// 2s + 1: the features come in another order than in memory, in both operands the same.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "selected.h"

namespace dfs {
namespace tiles {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values (lane (g, t): row g, columns 2t and 2t + 1) transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Two weights as pairs of bf16 values, high + low, so that the products lose 2^-16 of a weight and not 2^-8.  The high
// ones are cut, not rounded, and 2^-22 of the weight goes on top: the low ones are above 0 wherever the weight is, and
// an infinite value times both stays infinite.
__device__ __forceinline__ void split_weights(float x, float y, uint32_t* high, uint32_t* low) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    constexpr float kUp = 1.f + 2.384185791015625e-7f;
    *high = __byte_perm(a, b, 0x7632);
    *low = pack(fmaf(x, kUp, -__uint_as_float(a & 0xffff0000u)), fmaf(y, kUp, -__uint_as_float(b & 0xffff0000u)));
}

// This lane's words of a row; zeros where the row is not to be read.
__device__ __forceinline__ void load_row(const __nv_bfloat16* row, bool live, int t, uint32_t (&w)[8]) {
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (live) {
        a = reinterpret_cast<const uint4*>(row)[t];
        b = reinterpret_cast<const uint4*>(row)[4 + t];
    }
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}
// 64 key rows from `base`; rows from `rows` on are zeros and not read.
__device__ __forceinline__ void load_keys(const __nv_bfloat16* base, int rows, int lane, uint32_t (&k)[8][8]) {
#pragma unroll
    for (int o = 0; o < 8; ++o) {
        const int r = 8 * o + (lane >> 2);
        load_row(base + (int64_t)r * kHeadDim, r < rows, lane & 3, k[o]);
    }
}
// Values as the left operand of the second product (features by keys).
__device__ __forceinline__ void turn_values(uint32_t (&v)[8][8]) {
#pragma unroll
    for (int o = 0; o < 8; ++o)
#pragma unroll
        for (int c = 0; c < 8; ++c) v[o][c] = transposed(v[o][c]);
}

// s[M]: products of keys 16 M + g (0, 1) and 16 M + 8 + g (2, 3) with queries 2t (0, 2) and 2t + 1 (1, 3).
__device__ __forceinline__ void score(const uint32_t (&k)[8][8], const uint32_t (&q)[8], float (&s)[4][4]) {
#pragma unroll
    for (int M = 0; M < 4; ++M) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[M][j] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            mma(s[M], k[2 * M][2 * e], k[2 * M + 1][2 * e], k[2 * M][2 * e + 1], k[2 * M + 1][2 * e + 1], q[2 * e], q[2 * e + 1]);
    }
}
// o[j] += the weights p (laid out as score's result) times the turned values: features F(2j, g) (0, 1)
// and F(2j + 1, g) (2, 3) of queries 2t (0, 2) and 2t + 1 (1, 3), F(c, g) = 32 (c / 4) + 8 (g / 2) + 2 (c % 4) + g % 2.
__device__ __forceinline__ void weigh(const uint32_t (&v)[8][8], const float (&p)[4][4], float (&o)[4][4]) {
#pragma unroll
    for (int M = 0; M < 4; ++M) {
        uint32_t w[2][2];                    // high and low, of keys 16 M + g and 16 M + 8 + g
#pragma unroll
        for (int e = 0; e < 2; ++e) split_weights(p[M][2 * e], p[M][2 * e + 1], &w[0][e], &w[1][e]);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const uint32_t b0 = transposed(w[part][0]), b1 = transposed(w[part][1]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                mma(o[j], v[2 * M][2 * j], v[2 * M][2 * j + 1], v[2 * M + 1][2 * j], v[2 * M + 1][2 * j + 1], b0, b1);
        }
    }
}
// Where feature f stands in a row that the lanes write as 8 g + c.
__host__ __device__ __forceinline__ constexpr int place_of(int f) {
    return 8 * (2 * ((f & 31) >> 3) + (f & 1)) + (f >> 5) * 4 + ((f & 7) >> 1);
}

// Over the eight lanes of a query's column.
__device__ __forceinline__ float column_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
    x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
    return fmaxf(x, __shfl_xor_sync(kFull, x, 16));
}
__device__ __forceinline__ float column_sum(float x) {
    x += __shfl_xor_sync(kFull, x, 4);
    x += __shfl_xor_sync(kFull, x, 8);
    return x + __shfl_xor_sync(kFull, x, 16);
}

}  // namespace tiles
}  // namespace dfs
