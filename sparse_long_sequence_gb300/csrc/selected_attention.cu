// Attention over the key blocks that each query lists:
//   out_i = sum_j p_ij v_j,  p_ij = exp(q_i.k_j / 8 - lse_i),
// j over the visible keys of the listed blocks; a row without such keys is 0, its lse -infinity.
//
// Few queries: one block of threads for a query and up to eight heads of its group (the eight
// columns of the products).  Its warps take the listed blocks in turn, each with a running maximum
// and sum in registers, and join through shared memory.  A block's keys and values go from global
// memory into the products' registers.  Bound by the cache's bytes, or by a launch.
#include <atomic>

#include "mma_tiles.cuh"
#include "selected.h"

namespace dfs {
namespace {

using namespace tiles;

constexpr float kScale2 = 0.125f * 1.4426950408889634f;      // 1 / sqrt(64) in units of log 2
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kFewWarps = 8;

// The listed blocks that count: entry x of a query's list does if it is above all entries before it
// (which -1 is not) and has visible keys.  Warp-wide; bit x of the result.
__device__ __forceinline__ uint64_t live_slots(const int32_t* list, int top, int32_t limit, int lane) {
    uint64_t live = 0;
    int before = -1;
    for (int x0 = 0; x0 < top; x0 += 32) {
        const int x = x0 + lane;
        const int c = x < top ? list[x] : -1;
        int high = c;                                        // the largest up to this lane
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
            const int o = __shfl_up_sync(kFull, high, off);
            if (lane >= off) high = max(high, o);
        }
        int prev = __shfl_up_sync(kFull, high, 1);
        prev = max(lane ? prev : -1, before);
        const bool in = c > prev && (int64_t)c * kBlockKeys < limit;
        live |= (uint64_t)__ballot_sync(kFull, in) << x0;
        before = max(before, __shfl_sync(kFull, high, 31));
    }
    return live;
}

__global__ void __launch_bounds__(32 * kFewWarps) selected_few_kernel(const __grid_constant__ SelectedArgs a) {
    __shared__ float part[kFewWarps][8][kHeadDim];
    __shared__ float2 stat[kFewWarps][8];                    // maximum (of scores in units of log 2), sum
    const SelectShape& s = a.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int warps = blockDim.x >> 5, octets = (s.G + 7) / 8;
    const int64_t row = blockIdx.x / octets, u = row / s.n, i = row % s.n, b = u / s.Hk;
    const int h0 = (int)(blockIdx.x % octets) * 8, heads = min(8, s.G - h0);
    const int64_t first = (b * s.Hq + (u % s.Hk) * s.G + h0) * s.n + i;      // row of head h: + h n
    const int32_t limit = row_limit(s, b, i);
    const int32_t* list = a.blocks + row * s.top;

    uint32_t q[8];
    load_row(a.q + (first + g * s.n) * kHeadDim, g < heads, t, q);
    float o[4][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j >> 2][j & 3] = 0.f;
    uint64_t live = live_slots(list, s.top, limit, lane);
    for (int k = 0; live; ++k, live &= live - 1) {
        if (k % warps != warp) continue;
        const int32_t c = list[__ffsll((long long)live) - 1];
        const int64_t key0 = (int64_t)c * kBlockKeys;
        const int rows = min(kBlockKeys, (int)(limit - key0));
        uint32_t keys[8][8], values[8][8];
        load_keys(a.k + (u * s.m + key0) * kHeadDim, rows, lane, keys);
        load_keys(a.v + (u * s.m + key0) * kHeadDim, rows, lane, values);
        float x[4][4];
        score(keys, q, x);
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int M = 0; M < 4; ++M)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[M][j] = 16 * M + 8 * (j >> 1) + g < rows ? x[M][j] * kScale2 : -INFINITY;
                top[j & 1] = fmaxf(top[j & 1], x[M][j]);
            }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float now = fmaxf(m[e], column_max(top[e]));
            const float base = now == -INFINITY ? 0.f : now, shrink = exp2_fast(m[e] - base);
            float sum = 0.f;
#pragma unroll
            for (int M = 0; M < 4; ++M)
#pragma unroll
                for (int j = e; j < 4; j += 2) {
                    x[M][j] = exp2_fast(x[M][j] - base);
                    sum += x[M][j];
                }
            l[e] = l[e] * shrink + column_sum(sum);
            m[e] = now;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[j][e] *= shrink;
                o[j][e + 2] *= shrink;
            }
        }
        turn_values(values);
        weigh(values, x, o);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float* dst = &part[warp][2 * t + e][8 * g];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<float4*>(dst + 4 * j) = make_float4(o[2 * j][e], o[2 * j][e + 2], o[2 * j + 1][e], o[2 * j + 1][e + 2]);
        if (g == 0) stat[warp][2 * t + e] = make_float2(m[e], l[e]);
    }
    __syncthreads();
    for (int x = threadIdx.x; x < heads * 32; x += blockDim.x) {
        const int h = x >> 5, f = 2 * (x & 31);
        float top = -INFINITY;
        for (int w = 0; w < warps; ++w) top = fmaxf(top, stat[w][h].x);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f, y0 = 0.f, y1 = 0.f;
        for (int w = 0; w < warps; ++w) {
            const float e = exp2_fast(stat[w][h].x - base);
            sum += e * stat[w][h].y;
            y0 += e * part[w][h][place_of(f)];
            y1 += e * part[w][h][place_of(f + 1)];
        }
        const float r = limit && top != -INFINITY ? 1.f / sum : 0.f;
        const int64_t at = first + h * s.n;
        *reinterpret_cast<uint32_t*>(a.out + at * kHeadDim + f) = pack(y0 * r, y1 * r);
        if (a.lse && f == 0) a.lse[at] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

int launch_few(const SelectedArgs& a, cudaStream_t stream) {
    const SelectShape& s = a.s;
    const int64_t grid = s.B * s.Hk * s.n * ((s.G + 7) / 8);
    if (grid > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    const int warps = s.top < kFewWarps ? s.top : kFewWarps;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        selected_few_kernel<<<(unsigned)grid, 32 * warps, 0, stream>>>(a);
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "selected_few_kernel");
}

}  // namespace

size_t selected_workspace(const SelectShape&) { return 0; }

int launch_selected(const SelectedArgs& a, char*, cudaStream_t stream) { return launch_few(a, stream); }

}  // namespace dfs
