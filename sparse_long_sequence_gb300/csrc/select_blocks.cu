// The choice of key blocks: for each query and key head the `top` visible blocks with the largest
//   score(i, c) = sum over the group's heads h and features f of q_h,i,f mean_c,f,
// ties to the lowest index, the forced blocks (the first `sink`, and those less than `local` from the
// query's own) before all others, written in ascending order with -1 behind them.
//
// A block of eight warps takes up to 16 queries of a unit (sequence and key head).  First the scores
// on m16n8k16 products (16 blocks by 8 queries, the heads one after the other along the summed index),
// kept in shared memory as fp32; then a warp a query: the top-th largest value by bisection on values.
// The products are exact in fp32, their sums are not: a tensor core adds 16 products and the sum so
// far with an error of at most 17 2^-23 of the largest of them, so a score is off by at most
//   eps = 4 G 17 2^-23 sum_f |q_f| max |mean|.
// Blocks more than 2 eps above the top-th value are in, those more than 2 eps below are out, and what
// lies between is summed again in fp64, where 64 G products of bf16 values lose nothing that matters.
// So the choice is that of exact scores, whatever order they are added in.
#include <atomic>
#include <cfloat>

#include "layer_ops.h"
#include "mma_tiles.cuh"
#include "selected.h"

namespace dfs {
namespace {

using namespace tiles;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMostQueries = 16;

struct Choice {
    SelectShape s;
    const __nv_bfloat16 *q, *means;
    int32_t sink, local;
    int32_t* blocks;
    int32_t tile;                  // queries of a block of threads: 16, or fewer for many key blocks
    int32_t stride;                // floats of a query's scores
};

__device__ __forceinline__ float abs_sum(uint32_t w) {
    return fabsf(__uint_as_float(w << 16)) + fabsf(__uint_as_float(w & 0xffff0000u));
}

// The score in fp64, in every lane; NaN counts as -infinity.
__device__ __forceinline__ double exact_score(const uint32_t* q, int64_t head_words, int G, const uint32_t* mean, int lane) {
    const uint32_t w = mean[lane];
    const double m0 = __uint_as_float(w << 16), m1 = __uint_as_float(w & 0xffff0000u);
    double t = 0.0;
    for (int h = 0; h < G; ++h) {
        const uint32_t x = q[h * head_words + lane];
        t += (double)__uint_as_float(x << 16) * m0 + (double)__uint_as_float(x & 0xffff0000u) * m1;
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

__global__ void __launch_bounds__(kThreads) select_blocks_kernel(const __grid_constant__ Choice a) {
    extern __shared__ __align__(16) float scores[];          // [tile][stride]
    __shared__ int32_t limit[kMostQueries];
    __shared__ float mass[kMostQueries];                     // sum |q| over the group's heads
    __shared__ unsigned largest;                             // bits of max |mean|
    const SelectShape& s = a.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int64_t tiles = (s.n + a.tile - 1) / a.tile, u = blockIdx.x / tiles, i0 = (blockIdx.x % tiles) * a.tile;
    const int64_t b = u / s.Hk, head = u % s.Hk;
    const int queries = (int)min((int64_t)a.tile, s.n - i0);
    const __nv_bfloat16* q = a.q + ((b * s.Hq + head * s.G) * s.n + i0) * kHeadDim;    // head h: + h n 64
    const __nv_bfloat16* means = a.means + u * s.nb * kHeadDim;

    if (threadIdx.x == 0) largest = 0;
    if (threadIdx.x < kMostQueries) limit[threadIdx.x] = threadIdx.x < queries ? row_limit(s, b, i0 + threadIdx.x) : 0;
    for (int r = warp; r < queries; r += kWarps) {
        float x = 0.f;
        for (int h = 0; h < s.G; ++h) x += abs_sum(reinterpret_cast<const uint32_t*>(q + (h * s.n + r) * kHeadDim)[lane]);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
        if (lane == 0) mass[r] = x;
    }
    __syncthreads();
    int most = 0;
    for (int r = 0; r < queries; ++r) most = max(most, limit[r]);
    const int seen = (most + kBlockKeys - 1) / kBlockKeys;   // blocks that some query sees

    float top_mean = 0.f;
    bool odd = false;                                        // a mean that is no number
    for (int c0 = 16 * warp; c0 < seen; c0 += 16 * kWarps) {
        uint32_t k[2][8];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int c = c0 + 8 * o + g;
            load_row(means + (int64_t)c * kHeadDim, c < seen, t, k[o]);
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const float x = fabsf(__uint_as_float(k[o][w] << 16)), y = fabsf(__uint_as_float(k[o][w] & 0xffff0000u));
                top_mean = fmaxf(top_mean, fmaxf(x, y));
                odd |= x != x || y != y;
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (8 * half >= queries) break;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            for (int h = 0; h < s.G; ++h) {
                uint32_t x[8];
                const int r = 8 * half + g;
                load_row(q + (h * s.n + r) * kHeadDim, r < queries, t, x);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mma(acc, k[0][2 * e], k[1][2 * e], k[0][2 * e + 1], k[1][2 * e + 1], x[2 * e], x[2 * e + 1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 8 * half + 2 * t + (j & 1);
                if (r < queries) scores[r * a.stride + c0 + g + 8 * (j >> 1)] = acc[j];
            }
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top_mean = fmaxf(top_mean, __shfl_xor_sync(kFull, top_mean, off));
    if (__any_sync(kFull, odd)) top_mean = INFINITY;
    if (lane == 0) atomicMax(&largest, __float_as_uint(top_mean));
    __syncthreads();
    top_mean = __uint_as_float(largest);

    for (int r = warp; r < queries; r += kWarps) {
        int32_t* out = a.blocks + ((u * s.n) + i0 + r) * s.top;
        const int lim = limit[r], nv = (lim + kBlockKeys - 1) / kBlockKeys;
        if (nv <= s.top) {
            for (int x = lane; x < s.top; x += 32) out[x] = x < nv ? x : -1;
            continue;
        }
        float* v = scores + r * a.stride;
        // the query's own position: its limit is one behind it, or (not causal) the length is
        const int64_t len = key_count(s, b);
        const int64_t p = s.causal ? lim - 1 : (s.starts ? (int64_t)s.starts[b] : len - s.n) + i0 + r;
        const int home = (int)(p / kBlockKeys);
        float lo = INFINITY, hi = -INFINITY;
        const int padded = (nv + 127) / 128 * 128;
        for (int c = lane; c < padded; c += 32) {
            float x = -INFINITY;
            if (c < nv) {
                if (c < a.sink || abs(c - home) < a.local) {
                    x = INFINITY;
                } else {
                    x = fminf(fmaxf(v[c], -FLT_MAX), FLT_MAX);       // (NaN: the lowest)
                    lo = fminf(lo, x);
                    hi = fmaxf(hi, x);
                }
            }
            v[c] = x;
        }
        __syncwarp();
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(kFull, lo, off));
            hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, off));
        }
        // the top-th largest value, kth: at least top values reach lo, fewer than top pass hi
        float kth;
        auto reach = [&](float x) {
            int n = 0;
            for (int c = 4 * lane; c < padded; c += 128) {
                const float4 y = *reinterpret_cast<const float4*>(v + c);
                n += (y.x >= x) + (y.y >= x) + (y.z >= x) + (y.w >= x);
            }
            return __reduce_add_sync(kFull, n);
        };
        if (reach(hi) >= s.top) {
            kth = hi;                                        // (the forced and hi's equals are enough)
        } else {
            for (;;) {
                const float mid = lo + 0.5f * (hi - lo);
                if (!(mid > lo && mid < hi)) {
                    kth = lo;
                    break;
                }
                const int n = reach(mid);
                if (n == s.top) {
                    float least = INFINITY;
                    for (int c = lane; c < nv; c += 32)
                        if (v[c] >= mid) least = fminf(least, v[c]);
#pragma unroll
                    for (int off = 16; off >= 1; off >>= 1) least = fminf(least, __shfl_xor_sync(kFull, least, off));
                    kth = least;
                    break;
                }
                if (n > s.top) lo = mid;
                else hi = mid;
            }
        }
        // 2 eps (and what products of denormal size may lose)
        const float eps = 2.02f * 68.f * 1.1920929e-7f * (float)s.G * mass[r] * top_mean + 1e-35f;
        const bool far = !(eps < 1e30f) || !(fabsf(kth) < 1e30f);
        const float above = far ? INFINITY : kth + eps, below = far ? -INFINITY : kth - eps;
        int sure = 0, open = 0;
        for (int c = lane; c < nv; c += 32) {
            const bool in = v[c] == INFINITY || v[c] > above;
            sure += in;
            open += !in && v[c] >= below;
        }
        sure = __reduce_add_sync(kFull, sure);
        open = __reduce_add_sync(kFull, open);
        if (sure + open > s.top) {
            const int want = s.top - sure;                   // 0 where the forced blocks are all
            Best best;
            const uint32_t* row = reinterpret_cast<const uint32_t*>(q + r * kHeadDim);
            for (int c0 = 0; c0 < nv; c0 += 32) {
                const int c = c0 + lane;
                const float x = c < nv ? v[c] : -INFINITY;
                const bool near = c < nv && x != INFINITY && !(x > above) && x >= below;
                for (unsigned m = __ballot_sync(kFull, near); want && m; m &= m - 1) {
                    const int index = c0 + __ffs(m) - 1;
                    const double score = exact_score(row, s.n * (kHeadDim / 2), s.G,
                                                     reinterpret_cast<const uint32_t*>(means + (int64_t)index * kHeadDim), lane);
                    best.offer(score, index, want, lane);
                }
                if (near) v[c] = -INFINITY;
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (lane + 32 * j < want) v[best.c[j]] = INFINITY;
            __syncwarp();
        } else {
            for (int c = lane; c < nv; c += 32)
                if (v[c] >= below) v[c] = INFINITY;
            __syncwarp();
        }
        int at = 0;
        for (int c0 = 0; c0 < nv; c0 += 32) {
            const int c = c0 + lane;
            const bool in = c < nv && (v[c] == INFINITY || v[c] > above);
            const unsigned m = __ballot_sync(kFull, in);
            if (in) out[at + __popc(m & ((1u << lane) - 1))] = c;
            at += __popc(m);
        }
    }
}

}  // namespace

int launch_select_blocks(const SelectShape& s, const void* Q, const void* means, int32_t sink, int32_t local,
                         int32_t* blocks, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    constexpr int kMostSmem = 200 * 1024;
    Choice a{s, static_cast<const __nv_bfloat16*>(Q), static_cast<const __nv_bfloat16*>(means), sink, local, blocks, kMostQueries, 0};
    // whole loads of a warp, and 4 more floats: the lanes of a product's column fall in other banks
    a.stride = (s.nb + 127) / 128 * 128 + 4;
    while ((int64_t)a.tile * a.stride * 4 > kMostSmem) a.tile /= 2;
    const int64_t grid = s.B * s.Hk * ((s.n + a.tile - 1) / a.tile);
    if (grid > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    cudaError_t err = allow_smem(select_blocks_kernel, kMostSmem, ready);
    if (err != cudaSuccess) return cuda_fail(err, "select_blocks_kernel");
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        select_blocks_kernel<<<(unsigned)grid, kThreads, (size_t)a.tile * a.stride * 4, stream>>>(a);
    }
    err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "select_blocks_kernel");
}

}  // namespace dfs
