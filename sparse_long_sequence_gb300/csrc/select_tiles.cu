// The choice of key blocks (select_blocks.cu says what is chosen and why the result is that of exact scores)
// for many queries: a thread a query.
//
// A block of four warps takes 128 queries of a unit.  Their scores against 128 block means at a time (the next
// ones are on their way meanwhile) are one tcgen05 product (128 x 128, the group's heads one after the other along
// the summed index), and a query's scores lie in its thread's lane of tensor memory.  The thread reads them twice: first for the maxima of 32 groups of
// columns, whose want-th largest bounds the want-th largest score from below; then for the scores above that
// bound, a few more than `want`, which it lists in shared memory.  Among those it finds the want-th largest.  Both
// times 32 values are sorted in registers by a network (Batcher's odd-even merges: 191 comparisons, the same for
// all threads, where bisections would run until the last of 32 threads is done).  (Where the list is full before
// all are in it, the want-th largest of the list is the next bound, and the scores are read again.)  Where scores
// come closer to each other there than they are exact, the warp looks at that query together and sums the close
// ones again as fp64 would; so it does, for all of a query's blocks, where a list stays full or a score is no
// number.
//
// Bound by the issue of instructions and their latencies at 12 warps an SM (shared memory: 66 KB for four): two passes
// over the scores and two sorts a query; the products alone would take a twentieth of the time.  16 x 16384 queries
// of 256 blocks take 90 us, where a warp a query took 194: every step of its searches served one query.
#include <atomic>
#include <cfloat>

#include "dense_ptx.cuh"
#include "layer_ops.h"
#include "row_tiles.cuh"
#include "select_common.cuh"

namespace dfs {
namespace {

using namespace tiles;
using namespace select;

constexpr int kThreads = kTileRows;
constexpr int kRound = 128;                  // block means of a product
constexpr int kMaxima = 32;
constexpr int kList = 32;                    // a query's candidates
static_assert(kList > kTilesTop + 1, "a full list holds more than are wanted");
constexpr int kMeanBytes = kRound * kRowBytes;
constexpr int kEntry = kThreads * 4;         // from a list's entry to its next
constexpr int kListBytes = 2 * kList * kEntry;               // scores, blocks
constexpr int kSmem = kTileBytes + kMeanBytes + kListBytes;

// Batcher's network for 32 values.
struct Network {
    int pairs = 0;
    uint8_t a[191] = {}, b[191] = {};
    constexpr Network() {
        for (int p = 1; p < 32; p *= 2)
            for (int k = p; k >= 1; k /= 2)
                for (int j = k % p; j + k < 32; j += 2 * k)
                    for (int i = 0; i < k && i + j + k < 32; ++i)
                        if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                            a[pairs] = i + j;
                            b[pairs++] = i + j + k;
                        }
    }
};
// Descending.
__device__ __forceinline__ void sort32(float (&x)[32]) {
    constexpr Network net;
    static_assert(net.pairs == 191, "all of the network");
#pragma unroll
    for (int k = 0; k < 191; ++k) {
        const float a = x[net.a[k]], b = x[net.b[k]];
        x[net.a[k]] = fmaxf(a, b);
        x[net.b[k]] = fminf(a, b);
    }
}
// x[i] of descending values, i from 0 to kTilesTop: the largest from x[i] on (as a choice by index it is kept in
// local memory)
__device__ __forceinline__ float pick(const float (&x)[32], int i) {
    float y = -INFINITY;
#pragma unroll
    for (int j = 0; j <= kTilesTop; ++j) y = fmaxf(y, j >= i ? x[j] : -INFINITY);
    return y;
}

__global__ void __launch_bounds__(kThreads, 3) select_tiles_kernel(const __grid_constant__ Choice a, int* status) {
    extern __shared__ __align__(1024) char smem[];
    __shared__ uint64_t bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int seen_smem;
    __shared__ unsigned largest;             // bits of the largest sum of a mean's squares
    const SelectShape& s = a.s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // every unit's last queries first, which see the most blocks where it is causal (90 us for 96 unit by unit)
    const uint32_t parts = (uint32_t)(s.n + kTileRows - 1) / kTileRows, units = gridDim.x / parts, part = blockIdx.x / units;
    const int64_t u = blockIdx.x - part * units, i0 = (int64_t)(parts - 1 - part) * kTileRows, b = sequence_of(s, u);
    const int queries = (int)min((int64_t)kTileRows, s.n - i0);
    const __nv_bfloat16* q0 = a.q + (u * s.G * s.n + i0) * kHeadDim;                   // head h: + h n 64
    const __nv_bfloat16* means = a.means + u * s.nb * kHeadDim;
    const uint32_t q_tile = ptx::smem_u32(smem), mean_tile = q_tile + kTileBytes;
    const float* list_x = reinterpret_cast<const float*>(smem + kTileBytes + kMeanBytes) + tid;    // entry e: + e kThreads
    const int32_t* list_c = reinterpret_cast<const int32_t*>(smem + kTileBytes + kMeanBytes + kList * kEntry) + tid;
    const int pitch = s.top | 1;             // of the results on their way out, where the means were
    int32_t* result = reinterpret_cast<int32_t*>(smem + kTileBytes) + tid * pitch;

    const int lim = tid < queries ? row_limit(s, b, i0 + tid) : 0, nv = (lim + kBlockKeys - 1) / kBlockKeys;
    // the query's own position: its limit is one behind it, or (not causal) the length is
    const int64_t p = s.causal ? lim - 1 : (s.starts ? (int64_t)s.starts[b] : lim - s.n) + i0 + tid;
    const Forced forced(a.sink, a.local, (int)(p / kBlockKeys), nv);
    const int want = s.top - forced.count();                 // besides the forced
    const bool choose = nv > s.top;
    __syncwarp();
    if (warp == 0) ptx::tmem_alloc(&tmem_slot, kRound);
    if (tid == 0) {
        ptx::mbar_init(&bar, 1);
        ptx::fence_mbar_init();
        seen_smem = 0;
        largest = 0;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const int most = __reduce_max_sync(kFull, choose ? nv : 0);
    if (lane == 0) atomicMax(&seen_smem, most);
    __syncthreads();
    const int seen = seen_smem, rounds = (seen + kRound - 1) / kRound;   // blocks that some query has to choose among
    const uint32_t tmem = tmem_slot, mine = tmem + ((uint32_t)(32 * warp) << 16);

    uint32_t phase = 0;
    float mass = 0.f;                        // sum of q^2 over the group's heads
    unsigned top_squares = 0;                // of this thread's means
    int held = -1;                           // the round whose means are there, or on their way
    auto fetch = [&](int round) {
        const int c0 = round * kRound, rows = min(kRound, seen - c0);
        held = round;
#pragma unroll
        for (int x = tid; x < kRound * 8; x += kThreads) {
            const int r = x >> 3, c = x & 7;
            copy16(mean_tile + place(r, c), means + (int64_t)(c0 + (r < rows ? r : 0)) * kHeadDim + 8 * c, r < rows);
        }
    };
    // The scores of round `round` into tensor memory, then the means of round `next` (-1: none) on their way; the
    // first time through also mass and top_squares.
    auto score_round = [&](int round, int next, bool first) {
        const bool begin = held < 0;
        if (held != round) fetch(round);
        for (int h = 0; h < s.G; ++h) {
            if (h > 0) __syncthreads();      // all have read the last head's queries
            if (s.G > 1 || begin) {
#pragma unroll
                for (int x = tid; x < kTileRows * 8; x += kThreads) {
                    const int r = x >> 3, c = x & 7;
                    copy16(q_tile + place(r, c), q0 + (h * s.n + (r < queries ? r : 0)) * kHeadDim + 8 * c, r < queries);
                }
            }
            ptx::cp_async_wait_all();
            ptx::fence_proxy_async_smem();
            __syncthreads();
            __syncwarp();
            if (warp == 0 && ptx::elect_one()) {
                ptx::tc_fence_after();
                constexpr uint32_t kDesc = ptx::mma_idesc_bf16(kTileRows, kRound, false, false);
                const uint64_t qd = ptx::sw128_kmajor_desc(q_tile), md = ptx::sw128_kmajor_desc(mean_tile);
#pragma unroll
                for (int e = 0; e < 4; ++e) ptx::mma_bf16_ss(tmem, qd + 2 * e, md + 2 * e, kDesc, h > 0 || e > 0);
                ptx::mma_commit(&bar);
            }
            __syncwarp();
            if (begin) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 w = *reinterpret_cast<const uint4*>(smem + place(tid, c));
                    mass = squares(w.w, squares(w.z, squares(w.y, squares(w.x, mass))));
                }
            }
            if (first && h == 0) {
                static_assert(kRound == kThreads, "a mean a thread");
                float x = 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 w = *reinterpret_cast<const uint4*>(smem + kTileBytes + place(tid, c));
                    x = squares(w.w, squares(w.z, squares(w.y, squares(w.x, x))));
                }
                top_squares = max(top_squares, __float_as_uint(fabsf(x)));
            }
            ptx::mbar_wait(&bar, phase, status);
            phase ^= 1;
            __syncwarp();
        }
        ptx::tc_fence_after();
        if (next >= 0 && next != round) {
            __syncthreads();                 // all have read these means
            fetch(next);
        }
    };
    // columns c .. c + 31 of the round that begins with block c0; -infinity where the query sees no block, or it is forced
    auto scores = [&](int c0, int c, uint32_t (&v)[32]) {
        __syncwarp();
        ptx::tmem_ld32_issue(mine + c, v);
        ptx::tmem_ld_wait32(v);
        if (!__all_sync(kFull, c0 + c + 32 <= nv)) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c0 + c + j >= nv) v[j] = 0xff800000u;
        }
        if (__any_sync(kFull, c0 + c < forced.sink || (c0 + c < forced.near0 + forced.near && c0 + c + 32 > forced.near0))) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (forced.has(c0 + c + j)) v[j] = 0xff800000u;
        }
    };

    float bound = -INFINITY;
    if (rounds) {
        float top[kMaxima];
#pragma unroll
        for (int j = 0; j < kMaxima; ++j) top[j] = -INFINITY;
        for (int round = rounds - 1; round >= 0; --round) {      // (the first one's scores stay)
            if (round < rounds - 1) {
                ptx::tc_fence_before();
                __syncthreads();             // all have read the last scores
            }
            score_round(round, round ? round - 1 : min(1, rounds - 1), true);
            for (int c = 0; c < kRound && round * kRound + c < seen; c += 32) {
                uint32_t v[32];
                scores(round * kRound, c, v);
#pragma unroll
                for (int j = 0; j < 32; ++j) top[j] = fmaxf(top[j], __uint_as_float(v[j]));
            }
        }
        sort32(top);
        bound = pick(top, want - 1);         // (-infinity where fewer groups have any: all blocks are candidates)
    }
    top_squares = __reduce_max_sync(kFull, top_squares);
    if (lane == 0) atomicMax(&largest, top_squares);
    ptx::tc_fence_before();
    __syncthreads();
    const float eps = twice_eps(s.G, reach_of(s.G, mass, __uint_as_float(largest)));
    const bool far = !(eps < 1e30f);
    float floor = choose && want && !far ? fmaxf(bound - eps, -FLT_MAX) : INFINITY;
    const uint32_t list = mean_tile + kMeanBytes + 4 * tid, full = list + kList * kEntry;
    uint32_t end = list;
    int few;                                 // entries of the list
    float cut = -INFINITY;                   // scores from here on are in: the want-th largest, if the next is far below it
    bool hard = choose && want && far, close = hard;         // for the warp together: all blocks; or the list
    for (int round = 0, tries = 0;;) {
        // the scores from `floor` on, as many as the list holds
        for (int c = 0; c < kRound && round * kRound + c < seen; c += 32) {
            uint32_t v[32];
            scores(round * kRound, c, v);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                asm volatile(
                    "{\n.reg .pred p;\nsetp.lt.u32 p, %0, %4;\nsetp.ge.and.f32 p, %1, %3, p;\n"
                    "@p st.shared.b32 [%0], %1;\n@p st.shared.b32 [%0 + %6], %2;\n@p add.u32 %0, %0, %5;\n}"
                    : "+r"(end)
                    : "f"(__uint_as_float(v[j])), "r"(round * kRound + c + j), "f"(floor), "r"(full), "n"(kEntry), "n"(kList * kEntry)
                    : "memory");
        }
        if (++round < rounds) {
            ptx::tc_fence_before();
            __syncthreads();                 // all have read these scores
            score_round(round, round + 1 < rounds ? round + 1 : -1, false);
            continue;
        }
        few = (int)(end - list) / kEntry;
        const bool open = floor < INFINITY && few > want;
        bool again = false;
        if (__any_sync(kFull, open)) {
            float x[kList];
#pragma unroll
            for (int e = 0; e < kList; ++e) x[e] = e < few ? list_x[e * kThreads] : -INFINITY;
            sort32(x);
            const float kth = pick(x, want - 1), next = pick(x, want);
            if (open && few == kList) {
                again = kth - eps > floor && tries < 4;
                hard = close = !again;
                floor = again ? kth - eps : floor;
            } else if (open) {
                close = !(kth - next > eps);
                cut = kth;
            }
        }
        if (again) end = list;
        else floor = INFINITY;               // (this list stays)
        ptx::tc_fence_before();
        if (!__syncthreads_or(again)) break;
        ++tries;
        round = 0;
        if (rounds > 1) score_round(0, 1, false);
    }
    // (all have read the scores; the means' place is free for the results)
    __syncwarp();
    if (warp == 0) ptx::tmem_dealloc(tmem, kRound);

    if (tid < queries && !choose) {
        for (int x = 0; x < s.top; ++x) result[x] = x < nv ? x : -1;
    } else if (choose && !close) {
        int at = 0, f = 0;
        for (int e = 0; want && e < few; ++e) {
            if (!(list_x[e * kThreads] >= cut)) continue;
            const int c = list_c[e * kThreads];
            while (f < forced.count() && forced.at(f) < c) result[at++] = forced.at(f++);
            result[at++] = c;
        }
        while (f < forced.count()) result[at++] = forced.at(f++);
    }
    __syncwarp();
    for (unsigned todo = __ballot_sync(kFull, close); todo; todo &= todo - 1) {
        const int l = __ffs(todo) - 1, row = 32 * warp + l;  // the query's lane and row
        const int n = __shfl_sync(kFull, few, l), rest = __shfl_sync(kFull, want, l), blocks = __shfl_sync(kFull, nv, l);
        const float e = __shfl_sync(kFull, eps, l);
        const bool all = __shfl_sync(kFull, (int)hard, l);
        Forced f = forced;
        f.sink = __shfl_sync(kFull, forced.sink, l);
        f.near0 = __shfl_sync(kFull, forced.near0, l);
        f.near = __shfl_sync(kFull, forced.near, l);
        auto exact = [&](int c) {
            return exact_score(reinterpret_cast<const uint32_t*>(q0 + row * kHeadDim), s.n * (kHeadDim / 2), s.G,
                               reinterpret_cast<const uint32_t*>(means + (int64_t)c * kHeadDim), lane);
        };
        int32_t* out = result + (l - lane) * pitch;
        Best best;
        int cand = INT32_MAX;                // this lane's chosen block, if it has one
        if (all) {
            for (int c = 0; c < blocks; ++c)
                if (!f.has(c)) best.offer(exact(c), c, rest, lane);
            if (lane < rest) cand = best.c[0];
        } else {
            const float* xs = list_x - tid + row;
            const int32_t* cs = list_c - tid + row;
            const float x[2] = {lane < n ? xs[lane * kThreads] : -INFINITY, -INFINITY};
            const float kth = nth_largest(x, rest);
            const uint64_t sure = ballot2(x[0] > kth + e, x[1] > kth + e);
            const uint64_t open = ballot2(x[0] >= kth - e, x[1] >= kth - e) & ~sure;
            const int left = rest - __popcll(sure);
            for (uint64_t m = open; m; m &= m - 1) {
                const int c = cs[(__ffsll((long long)m) - 1) * kThreads];
                best.offer(exact(c), c, left, lane);
            }
            // the sure ones to lanes 0 .., the others behind them
            if (lane < left) cand = best.c[0];
            cand = __shfl_up_sync(kFull, cand, rest - left);
            if (lane < rest - left) {
                uint64_t m = sure;
                for (int k = 0; k < lane; ++k) m &= m - 1;
                cand = cs[(__ffsll((long long)m) - 1) * kThreads];
            }
            if (lane >= rest) cand = INT32_MAX;
        }
        int rank = 0;
        for (int k = 0; k < rest; ++k) rank += __shfl_sync(kFull, cand, k) < cand;
        if (lane < rest) out[rank + f.below(cand)] = cand;
        for (int x = 0; x < f.count(); ++x) {
            const int c = f.at(x);
            const int before = __popc(__ballot_sync(kFull, lane < rest && cand < c));
            if (lane == 0) out[x + before] = c;
        }
        __syncwarp();
    }
    __syncthreads();
    int32_t* to = a.blocks + (u * s.n + i0) * s.top;
    const int32_t* from = reinterpret_cast<const int32_t*>(smem + kTileBytes);
    for (int r = warp; r < queries; r += kThreads / 32)
        if (lane < s.top) to[r * s.top + lane] = from[r * pitch + lane];
}

}  // namespace

int launch_select_tiles(const Choice& a, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    const int64_t grid = a.s.B * a.s.Hk * ((a.s.n + kTileRows - 1) / kTileRows);
    if (grid > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    int* status = nullptr;
    if (const int st = ready_status(&status)) return st;
    cudaError_t err = allow_smem(select_tiles_kernel, kSmem, ready);
    if (err != cudaSuccess) return cuda_fail(err, "select_tiles_kernel");
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        select_tiles_kernel<<<(unsigned)grid, kThreads, kSmem, stream>>>(a, status);
    }
    err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "select_tiles_kernel");
}

}  // namespace dfs
