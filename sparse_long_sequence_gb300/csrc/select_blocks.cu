// The choice of key blocks: for each query and key head the `top` visible blocks with the largest
//   score(i, c) = sum over the group's heads h and features f of q_h,i,f mean_c,f,
// ties to the lowest index, the forced blocks (the first `sink`, and those less than `local` from the
// query's own) before all others, written in ascending order with -1 behind them.
//
// A block of eight warps takes up to 32 queries of a unit (sequence and key head).  First the scores
// on m16n8k16 products (16 blocks by 8 queries, the heads one after the other along the summed index),
// kept in shared memory as fp32; then a warp a query: candidates by the lanes' maxima, and among them the
// top-th largest value by bisection on values.
// The products are exact in fp32, their sums are not: a tensor core adds 16 products and the sum so
// far with an error of at most 17 2^-23 of the largest of them, so a score is off by at most
//   eps = 4 G 17 2^-23 |Q| |K|,
// |Q| the norm of the group's queries, |K| the largest of the means' (taken once for each head).
// Blocks more than 2 eps above the top-th value are in, those more than 2 eps below are out, and what
// lies between is summed again as fp64 would, where products of bf16 values are exact, and so are their sums while
// the products lie within 2^31 / G of each other.  So the choice is that of exact scores, whatever order they are added in.
//
// For few queries bound by latency: 16 queries of up to 1024 blocks, 4 key heads with 4 heads each, take 11.0 us;
// the search is a chain of reductions over one warp.
#include <atomic>
#include <cfloat>

#include "layer_ops.h"
#include "mma_tiles.cuh"
#include "select_common.cuh"

namespace dfs {
namespace {

using namespace tiles;
using namespace select;

constexpr int kWarps = 8;                    // of a block of threads; kMostWarps where few queries have many blocks
constexpr int kMostWarps = 32;
constexpr int kMostQueries = 32;

constexpr int kCandidates = 64;

// The `want` (1 to 32) largest of v[0 .. nv), of which more than `want` are above -infinity and at most `want`
// infinite (those are in), the others finite; v goes on as -infinity to a multiple of 32.  Some x that the
// maxima of at least `want` lanes reach bounds the want-th largest value from below, so that only the values
// above it, a few more than `want`, need a closer look: the candidates, by rising index, two a lane (place
// lane and lane + 32).  Returns false where there are too many of them; else in `taken` a bit for the place of
// each that is chosen.
template <class Exact>
__device__ __forceinline__ bool narrow(const float* v, int nv, int want, float eps, int lane, float* cand_x, int* cand_c,
                                       int (&cand)[2], uint64_t* taken, Exact exact) {
    float best = -INFINITY;
#pragma unroll 4
    for (int c = lane; c < nv; c += 32) best = fmaxf(best, v[c]);
    float lo = -INFINITY;                    // (fewer lanes than `want` have any: all values are candidates)
    if (__popc(__ballot_sync(kFull, best > -INFINITY)) >= want) {
        lo = warp_min(best > -INFINITY ? best : INFINITY);
        float hi = warp_max(best < INFINITY ? best : -INFINITY);
        for (int k = 0; k < 12 && lo < hi; ++k) {
            const float mid = lo + 0.5f * (hi - lo);
            const int n = __popc(__ballot_sync(kFull, best >= mid));
            if (n >= want) lo = mid;
            else hi = mid;
            if (n >= want && n <= want + 2) break;
        }
    }
    const float floor = fmaxf(lo - eps, -FLT_MAX);
    int few = 0;
    for (int c0 = 0; c0 < nv; c0 += 128) {   // (a vote at a time took 1.4 us more of 12.4 for 1024 blocks)
        float y[4];
        unsigned m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = c0 + 32 * j < nv ? v[c0 + 32 * j + lane] : -INFINITY;
        int more = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[j] = __ballot_sync(kFull, y[j] >= floor);
            more += __popc(m[j]);
        }
        if (few + more > kCandidates) return false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (y[j] >= floor) {
                const int place = few + __popc(m[j] & ((1u << lane) - 1));
                cand_x[place] = y[j];
                cand_c[place] = c0 + 32 * j + lane;
            }
            few += __popc(m[j]);
        }
    }
    __syncwarp();
    const float x0 = lane < few ? cand_x[lane] : -INFINITY;
    cand[0] = lane < few ? cand_c[lane] : 0;
    float kth, next = -INFINITY;             // the want-th largest and the largest below it
    if (few <= 32) {                         // the least go one by one
        float x = lane < few ? x0 : INFINITY;
        int left = few;
        while (left > want) {
            next = warp_min(x);
            const bool out = x == next;
            left -= __popc(__ballot_sync(kFull, out));
            if (out) x = INFINITY;
        }
        kth = left == want ? warp_min(x) : next;             // (left < want: equals on the border)
        if (left == want && kth - next > eps) {
            *taken = __ballot_sync(kFull, lane < few && x0 >= kth);
            return true;
        }
    } else {
        cand[1] = lane + 32 < few ? cand_c[lane + 32] : 0;
        const float x[2] = {x0, lane + 32 < few ? cand_x[lane + 32] : -INFINITY};
        kth = nth_largest(x, want);
    }
    const float x1 = lane + 32 < few ? cand_x[lane + 32] : -INFINITY;
    const uint64_t sure = ballot2(x0 > kth + eps, x1 > kth + eps);
    const uint64_t open = ballot2(x0 >= kth - eps, x1 >= kth - eps) & ~sure;
    if (__popcll(sure | open) == want) {
        *taken = sure | open;
        return true;
    }
    const int rest = want - __popcll(sure);
    Best fine;
    for (uint64_t m = open; m; m &= m - 1) {
        const int place = __ffsll((long long)m) - 1;
        fine.offer(exact(__shfl_sync(kFull, place < 32 ? cand[0] : cand[1], place & 31)), place, rest, lane);
    }
    const int a = lane < rest ? fine.c[0] : 64;              // (rest is 32 at most: one place a lane)
    *taken = sure | __reduce_or_sync(kFull, a < 32 ? 1u << a : 0u) |
             (uint64_t)__reduce_or_sync(kFull, a >= 32 && a < 64 ? 1u << (a - 32) : 0u) << 32;
    return true;
}

__global__ void __launch_bounds__(32 * kMostWarps) select_blocks_kernel(const __grid_constant__ Choice a) {
    extern __shared__ __align__(16) float scores[];          // [tile][stride]
    __shared__ int32_t limit[kMostQueries], home[kMostQueries];
    __shared__ float mass[kMostQueries];                     // sum of q^2 over the group's heads
    __shared__ unsigned largest;                             // bits of the largest sum of a mean's squares
    __shared__ float cand_x[kMostWarps][kCandidates];
    __shared__ int cand_c[kMostWarps][kCandidates];
    const SelectShape& s = a.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t tiles = (uint32_t)(s.n + a.tile - 1) / a.tile, ul = blockIdx.x / tiles;
    const int64_t u = ul, i0 = (int64_t)(blockIdx.x - ul * tiles) * a.tile, b = sequence_of(s, u);
    const int queries = (int)min((int64_t)a.tile, s.n - i0);
    const __nv_bfloat16* q = a.q + (u * s.G * s.n + i0) * kHeadDim;                    // head h: + h n 64
    const __nv_bfloat16* means = a.means + u * s.nb * kHeadDim;

    if (threadIdx.x == 0) largest = 0;
    if (threadIdx.x < kMostQueries) {
        const int lim = threadIdx.x < queries ? row_limit(s, b, i0 + threadIdx.x) : 0;
        // the query's own position: its limit is one behind it, or (not causal) the length is
        const int64_t p = s.causal ? lim - 1 : (s.starts ? (int64_t)s.starts[b] : lim - s.n) + i0 + threadIdx.x;
        limit[threadIdx.x] = lim;
        home[threadIdx.x] = (int)(p / kBlockKeys);
    }
    for (int r = warp; r < queries; r += warps) {
        float x = 0.f;
        for (int h = 0; h < s.G; ++h) x = squares(reinterpret_cast<const uint32_t*>(q + (h * s.n + r) * kHeadDim)[lane], x);
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
        if (lane == 0) mass[r] = x;
    }
    __syncthreads();
    const int most = __reduce_max_sync(kFull, limit[lane]);
    const int seen = (most + kBlockKeys - 1) / kBlockKeys;   // blocks that some query sees

    unsigned top_squares = 0;
    for (int c0 = 16 * warp; c0 < seen; c0 += 16 * warps) {
        uint32_t k[2][8];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int c = c0 + 8 * o + g;
            load_row(means + (int64_t)c * kHeadDim, c < seen, t, k[o]);
            float x = 0.f;                   // four lanes a row
#pragma unroll
            for (int w = 0; w < 8; ++w) x = squares(k[o][w], x);
            x += __shfl_xor_sync(kFull, x, 1);
            x += __shfl_xor_sync(kFull, x, 2);
            top_squares = max(top_squares, __float_as_uint(fabsf(x)));
        }
#pragma unroll
        for (int half = 0; half < kMostQueries / 8; ++half) {
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
    top_squares = __reduce_max_sync(kFull, top_squares);
    if (lane == 0) atomicMax(&largest, top_squares);
    __syncthreads();
    const float mean_squares = __uint_as_float(largest);

    for (int r = warp; r < queries; r += warps) {
        const int lim = limit[r], nv = (lim + kBlockKeys - 1) / kBlockKeys;
        int32_t* out = a.blocks + ((u * s.n) + i0 + r) * s.top;
        if (nv <= s.top) {
            for (int x = lane; x < s.top; x += 32) out[x] = x < nv ? x : -1;
            continue;
        }
        float* v = scores + r * a.stride;
        const Forced forced(a.sink, a.local, home[r], nv);
        for (int x = lane; x < forced.count(); x += 32) v[forced.at(x)] = INFINITY;
        if (nv + lane < (nv + 31) / 32 * 32) v[nv + lane] = -INFINITY;
        __syncwarp();
        const float eps = twice_eps(s.G, reach_of(s.G, mass[r], mean_squares));
        uint64_t taken = 0;
        int cand[2];
        if (s.top <= 32 && eps < 1e30f &&
            narrow(v, nv, s.top, eps, lane, cand_x[warp], cand_c[warp], cand, &taken, [&](int c) {
                return exact_score(reinterpret_cast<const uint32_t*>(q + r * kHeadDim), s.n * (kHeadDim / 2), s.G,
                                   reinterpret_cast<const uint32_t*>(means + (int64_t)c * kHeadDim), lane);
            })) {
            const unsigned lo = (unsigned)taken, hi = (unsigned)(taken >> 32), below = (1u << lane) - 1;
            if (lo >> lane & 1) out[__popc(lo & below)] = cand[0];
            if (hi >> lane & 1) out[__popc(lo) + __popc(hi & below)] = cand[1];
            __syncwarp();                                    // (the next query's candidates go to the same places)
            continue;
        }
        // the long way: any number of blocks and any scores
        float lo = INFINITY, hi = -INFINITY;
        const int padded = (nv + 127) / 128 * 128;
        for (int c = lane; c < padded; c += 32) {
            float x = c < nv ? v[c] : -INFINITY;
            if (c < nv && !forced.has(c)) {
                x = fminf(fmaxf(x, -FLT_MAX), FLT_MAX);      // (NaN: the lowest)
                lo = fminf(lo, x);
                hi = fmaxf(hi, x);
            }
            v[c] = x;
        }
        __syncwarp();
        lo = warp_min(lo);
        hi = warp_max(hi);
        // the top-th largest value, kth: at least top values reach lo, fewer than top reach hi
        float kth;
        auto reaching = [&](float x) {
            int n = 0;
            for (int c = 4 * lane; c < padded; c += 128) {
                const float4 y = *reinterpret_cast<const float4*>(v + c);
                n += (y.x >= x) + (y.y >= x) + (y.z >= x) + (y.w >= x);
            }
            return __reduce_add_sync(kFull, n);
        };
        if (reaching(hi) >= s.top) {
            kth = hi;                                        // (the forced and hi's equals are enough)
        } else {
            for (;;) {
                const float mid = lo + 0.5f * (hi - lo);
                if (!(mid > lo && mid < hi)) {
                    kth = lo;
                    break;
                }
                const int n = reaching(mid);
                if (n == s.top) {
                    float least = INFINITY;
                    for (int c = lane; c < nv; c += 32)
                        if (v[c] >= mid) least = fminf(least, v[c]);
                    kth = warp_min(least);
                    break;
                }
                if (n > s.top) lo = mid;
                else hi = mid;
            }
        }
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
            const int rest = s.top - sure;                   // 0 where the forced blocks are all
            Best best;
            const uint32_t* row = reinterpret_cast<const uint32_t*>(q + r * kHeadDim);
            for (int c0 = 0; c0 < nv; c0 += 32) {
                const int c = c0 + lane;
                const float x = c < nv ? v[c] : -INFINITY;
                const bool close = c < nv && x != INFINITY && !(x > above) && x >= below;
                for (unsigned m = __ballot_sync(kFull, close); rest && m; m &= m - 1) {
                    const int index = c0 + __ffs(m) - 1;
                    const double score = exact_score(row, s.n * (kHeadDim / 2), s.G,
                                                     reinterpret_cast<const uint32_t*>(means + (int64_t)index * kHeadDim), lane);
                    best.offer(score, index, rest, lane);
                }
                if (close) v[c] = -INFINITY;
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (lane + 32 * j < rest) v[best.c[j]] = INFINITY;
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
    // Many queries have a thread each: 16 x 16384 queries of 256 blocks take 90 us there and 205 here, 16 x 4096 of
    // 64 blocks 22 and 43, 24 x 1024 of 16 blocks 14 and 18.  There a block of threads goes over the heads of a group one
    // by one, which costs most where few blocks of threads run at once, and here it goes over the key blocks: 8 x 4096 of 64
    // blocks take 31 and 32 us with 4 heads a group, 47 and 46 with 8, 102 and 77 with 16; 32 x 4096 186 and 262 with 16,
    // 556 and 541 with 32; 2 x 32768 of 512 blocks 761 and 1006 with 32; 32768 of them 2371 and 1477 with 64.
    const int64_t queries = s.B * s.Hk * s.n, many = int64_t(24576) / 8 * (s.G > 8 ? s.G : 8);
    if (s.top <= kTilesTop && s.n >= 64 && queries >= 24576 && (s.nb >= 512 ? 4 * queries >= many : s.G <= 24 && queries >= many))
        return launch_select_tiles(a, stream);
    // fewer queries a block of threads where they are many key blocks', or where there are few of them for the SMs
    while (a.tile > 1 && ((int64_t)a.tile * a.stride * 4 > kMostSmem || a.tile / 2 >= s.n)) a.tile /= 2;
    while (a.tile > kWarps && s.B * s.Hk * ((s.n + a.tile - 1) / a.tile) < 2 * 152) a.tile /= 2;
    // (16 queries of 1024 blocks, 4 heads a group: 15.9 us with 8 warps, 11.0 with 32)
    const int per_warp = (s.nb + 31) / 32, warps = a.tile > 2 || per_warp <= kWarps ? kWarps : per_warp < kMostWarps ? per_warp : kMostWarps;
    const int64_t grid = s.B * s.Hk * ((s.n + a.tile - 1) / a.tile);
    if (grid > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    cudaError_t err = allow_smem(select_blocks_kernel, kMostSmem, ready);
    if (err != cudaSuccess) return cuda_fail(err, "select_blocks_kernel");
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        select_blocks_kernel<<<(unsigned)grid, 32 * warps, (size_t)a.tile * a.stride * 4, stream>>>(a);
    }
    err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "select_blocks_kernel");
}

}  // namespace dfs
