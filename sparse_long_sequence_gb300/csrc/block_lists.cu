// For each key block the list of the queries that name it, in rising order (so that what is summed
// over a list is summed in a fixed order), and the lists cut into items of equal work.
//
// Three launches.  (1) A block of threads sets, for a chunk of 64 to 256 queries, one bit a query in
// a bitmap of each key block in shared memory (atomic ors, whose order does not matter) and counts
// the bits.  (2) One block of threads a unit turns the counts into places: a running sum over the
// chunks for each key block, then over the key blocks, and writes the items.  (3) The bitmaps again:
// a query's place in a list is the number of bits before its own.  Bound by the latency of a few
// dependent loads; the lists' own bytes are a few percent of what the attention moves.
#include <atomic>

#include "block_lists.h"
#include "layer_ops.h"

namespace dfs {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;                    // loads of a lane in flight
constexpr int kScanThreads = 1024;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kBitmapBytes = 128 * 1024;

// A warp's 32 queries, `width` lanes a query (a power of two, at least top or 32): calls
// use(query of the 32, block, rank) for the blocks of a query that count, and all(query, their
// number).  Entry x of a query's list counts if it is above all entries before it (which -1 is
// not) and has visible keys.
template <class Use, class All>
__device__ __forceinline__ void each_live(const SelectShape& s, const int32_t* blocks, uint32_t u, int64_t i0, int width,
                                          Use use, All all) {
    const int64_t b = u / (uint32_t)s.Hk;
    const int lane = threadIdx.x & 31, x = lane & (width - 1), first = lane - x;
    const unsigned mine = width == 32 ? kFull : ((1u << width) - 1) << first;
    const int32_t* list = blocks + ((int64_t)u * s.n + i0) * s.top;
    for (int k0 = 0; k0 < width; k0 += kAhead) {             // 32 / width queries a turn
        int c[kAhead][2];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int q = (k0 + k) * (32 / width) + first / width;
            const bool on = k0 + k < width && i0 + q < s.n;
            c[k][0] = on && x < s.top ? list[(int64_t)q * s.top + x] : -1;
            c[k][1] = on && x + 32 < s.top ? list[(int64_t)q * s.top + x + 32] : -1;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (k0 + k >= width) break;
            const int q = (k0 + k) * (32 / width) + first / width;
            const int32_t limit = i0 + q < s.n ? row_limit(s, b, i0 + q) : 0;
            int before = -1, rank = 0;
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                if (part && s.top <= 32) break;
                int high = c[k][part];                       // the largest up to this lane
                for (int off = 1; off < width; off *= 2) {
                    const int o = __shfl_up_sync(kFull, high, off, width);
                    if (x >= off) high = max(high, o);
                }
                const int prev = __shfl_up_sync(kFull, high, 1, width);
                const int over = max(x ? prev : -1, before);
                const bool in = c[k][part] > over && (int64_t)c[k][part] * kBlockKeys < limit;
                const unsigned m = __ballot_sync(kFull, in) & mine;
                if (in) use(q, c[k][part], rank + __popc(m & ((1u << lane) - 1)));
                rank += __popc(m);
                before = max(before, __shfl_sync(kFull, high, width - 1, width));
            }
            if (x == 0 && i0 + q < s.n) all(q, rank);
        }
    }
}

// One bit a query in each block's words.
__device__ __forceinline__ void set_bits(const SelectShape& s, const int32_t* blocks, const BlockLists& l, int64_t u,
                                         int64_t chunk, uint32_t* bits) {
    for (int x = threadIdx.x; x < s.nb * l.words; x += blockDim.x) bits[x] = 0;
    __syncthreads();
    for (int w = threadIdx.x >> 5; w < l.words; w += blockDim.x >> 5)
        each_live(s, blocks, u, (chunk * l.words + w) * 32, l.width,
                  [&](int q, int c, int) { atomicOr(&bits[c * l.words + w], 1u << q); }, [](int, int) {});
    __syncthreads();
}

__global__ void __launch_bounds__(kThreads)
count_lists_kernel(const __grid_constant__ SelectShape s, const int32_t* blocks, const __grid_constant__ BlockLists l) {
    extern __shared__ uint32_t bits[];       // [nb][words]
    const int64_t u = blockIdx.x / (uint32_t)l.chunks, chunk = blockIdx.x % (uint32_t)l.chunks;
    set_bits(s, blocks, l, u, chunk, bits);
    for (int c = threadIdx.x; c < s.nb; c += blockDim.x) {
        int n = 0;
        for (int w = 0; w < l.words; ++w) n += __popc(bits[c * l.words + w]);
        l.counts[(u * l.chunks + chunk) * s.nb + c] = n;
    }
}

// Sums of a block's threads before this one, and of all.
__device__ __forceinline__ int2 before_and_all(int2 x, int2* sums, int2* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 run = x;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const int a = __shfl_up_sync(kFull, run.x, off), b = __shfl_up_sync(kFull, run.y, off);
        if (lane >= off) run = make_int2(run.x + a, run.y + b);
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    int2 before = make_int2(run.x - x.x, run.y - x.y), total = make_int2(0, 0);
    for (int w = 0; w < kScanThreads / 32; ++w) {
        if (w == warp) before = make_int2(before.x + total.x, before.y + total.y);
        total = make_int2(total.x + sums[w].x, total.y + sums[w].y);
    }
    __syncthreads();
    *all = total;
    return before;
}

__global__ void __launch_bounds__(kScanThreads)
place_lists_kernel(const __grid_constant__ SelectShape s, const __grid_constant__ BlockLists l) {
    __shared__ int2 sums[kScanThreads / 32];
    const int64_t u = blockIdx.x;
    int32_t* counts = l.counts + u * l.chunks * s.nb;
    int32_t *base = l.base + u * (s.nb + 1), *item_base = l.item_base + u * (s.nb + 1);
    int2 done = make_int2(0, 0);
    for (int c0 = 0; c0 < s.nb; c0 += kScanThreads) {
        const int c = c0 + threadIdx.x;
        int n = 0;
        if (c < s.nb) {
            int32_t* at = counts + c;
            int k = 0;
            for (; k + 8 <= l.chunks; k += 8) {              // eight loads in flight
                int32_t x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = at[(int64_t)(k + j) * s.nb];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    at[(int64_t)(k + j) * s.nb] = n;
                    n += x[j];
                }
            }
            for (; k < l.chunks; ++k) {
                const int32_t x = at[(int64_t)k * s.nb];
                at[(int64_t)k * s.nb] = n;
                n += x;
            }
        }
        const int64_t rows = (int64_t)n * s.G;
        const int items = (int)((rows + l.item_rows - 1) / l.item_rows);
        int2 all;
        const int2 before = before_and_all(make_int2(n, items), sums, &all);
        if (c < s.nb) {
            base[c] = done.x + before.x;
            item_base[c] = done.y + before.y;
            int4* out = l.items + u * l.most_items + done.y + before.y;
            for (int k = 0; k < items; ++k)
                out[k] = make_int4(c, k * l.item_rows, min(l.item_rows, (int)rows - k * l.item_rows), done.x + before.x);
        }
        done = make_int2(done.x + all.x, done.y + all.y);
    }
    if (threadIdx.x == 0) {
        base[s.nb] = done.x;
        item_base[s.nb] = done.y;
    }
}

__global__ void __launch_bounds__(kThreads)
fill_lists_kernel(const __grid_constant__ SelectShape s, const int32_t* blocks, const __grid_constant__ BlockLists l) {
    extern __shared__ uint32_t bits[];       // [nb][words], then [nb]
    const int64_t u = blockIdx.x / (uint32_t)l.chunks, chunk = blockIdx.x % (uint32_t)l.chunks;
    set_bits(s, blocks, l, u, chunk, bits);
    // where the chunk's queries of each block begin
    int32_t* begin = reinterpret_cast<int32_t*>(bits + s.nb * l.words);
    for (int c = threadIdx.x; c < s.nb; c += blockDim.x)
        begin[c] = l.base[u * (s.nb + 1) + c] + l.counts[(u * l.chunks + chunk) * s.nb + c];
    __syncthreads();
    uint32_t* entries = l.entries + u * s.n * l.ranks;
    for (int w = threadIdx.x >> 5; w < l.words; w += blockDim.x >> 5) {
        const int64_t i0 = (chunk * l.words + w) * 32;
        each_live(s, blocks, u, i0, l.width,
                  [&](int q, int c, int rank) {
                      const uint32_t* b = bits + c * l.words;
                      int at = begin[c] + __popc(b[w] & ((1u << q) - 1));
                      for (int k = 0; k < w; ++k) at += __popc(b[k]);
                      entries[at] = (uint32_t)(i0 + q) << 6 | rank;
                  },
                  [&](int q, int count) { l.live[u * s.n + i0 + q] = count; });
    }
}

}  // namespace

size_t plan_block_lists(const SelectShape& s, int32_t item_rows, char* ws, BlockLists* l) {
    const size_t units = (size_t)s.B * s.Hk;
    l->ranks = s.top < s.nb ? s.top : s.nb;
    l->item_rows = item_rows;
    l->width = 1;
    while (l->width < s.top && l->width < 32) l->width *= 2;
    l->words = 8;
    while (l->words > 2 && (int64_t)s.nb * l->words * 4 > kBitmapBytes) l->words /= 2;
    l->chunks = (int32_t)((s.n + 32 * l->words - 1) / (32 * l->words));
    const int64_t named = s.n * l->ranks;    // (query, block) pairs of a unit
    l->most_items = (int32_t)((named < s.nb ? named : s.nb) + named * s.G / item_rows);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = ws ? ws + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    l->entries = reinterpret_cast<uint32_t*>(take(units * named * 4));
    l->base = reinterpret_cast<int32_t*>(take(units * (s.nb + 1) * 4));
    l->item_base = reinterpret_cast<int32_t*>(take(units * (s.nb + 1) * 4));
    l->items = reinterpret_cast<int4*>(take(units * l->most_items * 16));
    l->live = reinterpret_cast<int32_t*>(take(units * s.n * 4));
    l->counts = reinterpret_cast<int32_t*>(take(units * l->chunks * s.nb * 4));
    return at;
}

int launch_block_lists(const SelectShape& s, const int32_t* blocks, const BlockLists& l, cudaStream_t stream) {
    static std::atomic<uint64_t> count_ready{0}, fill_ready{0};
    const int64_t units = s.B * s.Hk, grid = units * l.chunks;
    if (grid > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    cudaError_t err = allow_smem(count_lists_kernel, kBitmapBytes, count_ready);
    if (err == cudaSuccess) err = allow_smem(fill_lists_kernel, kBitmapBytes + kMaxKeys / kBlockKeys * 4, fill_ready);
    if (err != cudaSuccess) return cuda_fail(err, "the block lists");
    const size_t smem = (size_t)s.nb * l.words * 4;
    const int threads = 32 * l.words;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        count_lists_kernel<<<(unsigned)grid, threads, smem, stream>>>(s, blocks, l);
    }
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        place_lists_kernel<<<(unsigned)units, kScanThreads, 0, stream>>>(s, l);
    }
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        fill_lists_kernel<<<(unsigned)grid, threads, smem + (size_t)s.nb * 4, stream>>>(s, blocks, l);
    }
    err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "the block lists");
}

}  // namespace dfs
