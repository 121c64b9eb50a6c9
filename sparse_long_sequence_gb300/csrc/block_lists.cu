// For each key block the list of the queries that name it, in rising order (so that what is summed
// over a list is summed in a fixed order), and where each block's tiles of rows begin.
//
// Sums launches.  (1) A block of threads sets, for a chunk of 32 to 256 queries, one bit a query in
// a bitmap of each key block in shared memory (atomic ors, whose order does not matter) and counts
// the bits.  (2) One block of threads a unit (or several, and one after them) turns the counts into places: a running sum over the
// chunks for each key block, then over the key blocks.  (3) The bitmaps again:
// a query's place in a list is the number of bits before its own.  (1) and (2) are bound by the latency of a
// few dependent loads, (3) by the scattered stores of the entries, 4 bytes each: 16 x 16384 queries of 16 blocks
// take 10, 6 and 25 us.  (A thread that writes a block's entries in order, four a store, halves the
// sectors and takes 64: the first blocks', which every query lists, are one thread's work.)
#include <atomic>

#include "block_lists.h"
#include "layer_ops.h"
#include "sm100_ptx.cuh"

namespace dfs {
namespace {

constexpr int kThreads = 256;
constexpr int kScanThreads = 1024;
constexpr int kScanBlocks = 256;             // key blocks that the scan takes at a time, by four runs of chunks
constexpr int kPartBlocks = 64;              // a block of threads', where there are more of both
constexpr unsigned kFull = 0xffffffffu;
constexpr int kBitmapBytes = 64 * 1024;

// A warp's 32 queries, `width` lanes a query (a power of two) and four entries of its list a lane:
// calls use(query of the 32, four entries, which of them count, the rank of the first that does, their
// number) a lane, and all(query, the number of all).  An entry counts if it is above all entries before it (which -1 is not) and has visible keys.
template <class Use, class All>
__device__ __forceinline__ void each_live(const SelectShape& s, const int32_t* blocks, uint32_t u, int64_t i0, int width,
                                          Use use, All all) {
    const int lane = threadIdx.x & 31, x = lane & (width - 1), per = 32 / width;
    const uint32_t b = sequence_of(s, u);
    const int32_t len = key_count(s, b);
    const int64_t first = (s.starts ? (int64_t)s.starts[b] : len - s.n) + i0;
    const int32_t* list = blocks + ((int64_t)u * s.n + i0) * s.top + 4 * x;
    const bool whole = (s.top & 3) == 0;
#pragma unroll 2
    for (int k = 0; k < width; ++k) {
        const int q = k * per + lane / width;
        const bool on = i0 + q < s.n && 4 * x < s.top;
        int c[4] = {-1, -1, -1, -1};
        if (on && whole) {
            const int4 v = *reinterpret_cast<const int4*>(list + q * s.top);
            c[0] = v.x;
            c[1] = v.y;
            c[2] = v.z;
            c[3] = v.w;
        } else if (on) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * x + j < s.top) c[j] = list[q * s.top + j];
        }
        const int64_t p = first + q;
        const int32_t limit = p < 0 || p >= len || i0 + q >= s.n ? 0 : s.causal ? (int32_t)p + 1 : len;
        const int32_t blocks_seen = (limit + kBlockKeys - 1) / kBlockKeys;
        int high = max(max(c[0], c[1]), max(c[2], c[3])), before = -1;       // the largest of the lanes before
        for (int off = 1; off < width; off *= 2) {
            const int o = __shfl_up_sync(kFull, high, off, width);
            if (x >= off) {
                before = max(before, o);
                high = max(high, o);
            }
        }
        bool in[4];
        int count = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            in[j] = c[j] > before && c[j] < blocks_seen;
            before = max(before, c[j]);
            count += in[j];
        }
        int rank = count;
        for (int off = 1; off < width; off *= 2) {
            const int o = __shfl_up_sync(kFull, rank, off, width);
            if (x >= off) rank += o;
        }
        if (x == width - 1 && i0 + q < s.n) all(q, rank);
        rank -= count;
        use(q, c, in, rank, count);
    }
}

// bits[word][block]: one bit a query of the chunk.
__device__ __forceinline__ void set_bits(const SelectShape& s, const int32_t* blocks, const BlockLists& l, uint32_t u,
                                         int64_t chunk, uint32_t* bits) {
    for (int x = threadIdx.x; x < s.nb * l.words; x += blockDim.x) bits[x] = 0;
    __syncthreads();
    const int w = threadIdx.x >> 5;          // a warp a word (the others have no queries)
    each_live(s, blocks, u, w < l.words ? (chunk * l.words + w) * 32 : s.n, l.width,
              [&](int q, const int (&c)[4], const bool (&in)[4], int, int) {
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                      if (in[j]) atomicOr(&bits[w * s.nb + c[j]], 1u << q);
              },
              [](int, int) {});
    __syncthreads();
}

__global__ void __launch_bounds__(kThreads)
count_lists_kernel(const __grid_constant__ SelectShape s, const int32_t* blocks, const __grid_constant__ BlockLists l) {
    extern __shared__ uint32_t bits[];       // [words][nb]
    ptx::griddep_launch_dependents();
    const uint32_t u = blockIdx.x / (uint32_t)l.chunks, chunk = blockIdx.x - u * l.chunks;
    set_bits(s, blocks, l, u, chunk, bits);
    ptx::griddep_wait();                     // (what runs before it is none of its inputs', but has to be over for the others)
    for (int c = threadIdx.x; c < s.nb; c += blockDim.x) {
        int n = 0;
        for (int w = 0; w < l.words; ++w) n += __popc(bits[w * s.nb + c]);
        l.counts[((int64_t)u * l.chunks + chunk) * s.nb + c] = n;
    }
}

struct Sums {
    int32_t entries, tiles;
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {a.entries + b.entries, a.tiles + b.tiles}; }

// Sums over the first kWarps warps: of the threads before this one, and (in *all) of all.
template <int kWarps>
__device__ __forceinline__ Sums before_and_all(Sums x, Sums* sums, Sums* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums run = x;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const Sums o = {__shfl_up_sync(kFull, run.entries, off), __shfl_up_sync(kFull, run.tiles, off)};
        if (lane >= off) run = run + o;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    Sums before = {run.entries - x.entries, run.tiles - x.tiles}, total = {0, 0};
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = before + total;
        total = total + sums[w];
    }
    __syncthreads();
    *all = total;
    return before;
}

// Counts of a unit's blocks c0 .. c0 + kBlocks - 1 into running sums over the chunks; returns the sum over all (to each
// run's thread of a block).
template <int kBlocks>
__device__ __forceinline__ int sum_chunks(const SelectShape& s, const BlockLists& l, int32_t* counts, int c0,
                                          int32_t (*runs)[kBlocks]) {
    constexpr int kRuns = kScanThreads / kBlocks;
    const int run = threadIdx.x / kBlocks, x = threadIdx.x % kBlocks, c = c0 + x, per = (l.chunks + kRuns - 1) / kRuns;
    const int k0 = min(run * per, l.chunks), k1 = min(k0 + per, l.chunks);
    int n = 0;
    if (c < s.nb) {
#pragma unroll 16
        for (int k = k0; k < k1; ++k) n += counts[(int64_t)k * s.nb + c];
    }
    runs[run][x] = n;
    __syncthreads();
    n = 0;
    int mine = 0;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
        if (r == run) mine = n;
        n += runs[r][x];
    }
    if (c < s.nb) {
#pragma unroll 16
        for (int k = k0; k < k1; ++k) {
            const int32_t y = counts[(int64_t)k * s.nb + c];
            counts[(int64_t)k * s.nb + c] = mine;
            mine += y;
        }
    }
    return n;
}

// Where the blocks' entries and tiles begin.  kWhole: a block of threads has all of a unit, and sums its chunks too;
// else base[c] has the number of block c's entries.
template <bool kWhole>
__global__ void __launch_bounds__(kScanThreads)
place_lists_kernel(const __grid_constant__ SelectShape s, const __grid_constant__ BlockLists l) {
    __shared__ Sums sums[kScanThreads / 32];
    __shared__ int32_t runs[kScanThreads / kScanBlocks][kScanBlocks];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t u = blockIdx.x;
    int32_t* counts = l.counts + u * l.chunks * s.nb;
    int32_t *base = l.base + u * (s.nb + 1), *tile_base = l.tile_base + u * (s.nb + 1);
    constexpr int kStep = kWhole ? kScanBlocks : kScanThreads;
    Sums done = {0, 0};
    for (int c0 = 0; c0 < s.nb; c0 += kStep) {
        const int c = c0 + threadIdx.x;
        int n;
        if (kWhole) n = sum_chunks<kScanBlocks>(s, l, counts, c0, runs);
        else n = c < s.nb ? base[c] : 0;
        const bool on = threadIdx.x < kStep && c < s.nb;     // (the first run's threads sum over the blocks)
        if (!on) n = 0;
        const int tiles = (int)(((int64_t)n * s.G + kTileRows - 1) / kTileRows);
        Sums all;
        const Sums before = done + before_and_all<kStep / 32>({n, tiles}, sums, &all);
        if (on) {
            base[c] = before.entries;
            tile_base[c] = before.tiles;
        }
        done = done + all;
    }
    if (threadIdx.x == 0) {
        base[s.nb] = done.entries;
        tile_base[s.nb] = done.tiles;
    }
}

// The chunks' sums of kPartBlocks blocks a block of threads.
__global__ void __launch_bounds__(kScanThreads)
sum_lists_kernel(const __grid_constant__ SelectShape s, const __grid_constant__ BlockLists l, int parts) {
    __shared__ int32_t runs[kScanThreads / kPartBlocks][kPartBlocks];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t u = blockIdx.x / (uint32_t)parts;
    const int c0 = (blockIdx.x - (uint32_t)u * parts) * kPartBlocks, c = c0 + threadIdx.x;
    const int n = sum_chunks<kPartBlocks>(s, l, l.counts + u * l.chunks * s.nb, c0, runs);
    if (threadIdx.x < kPartBlocks && c < s.nb) l.base[u * (s.nb + 1) + c] = n;
}

__global__ void __launch_bounds__(kThreads)
fill_lists_kernel(const __grid_constant__ SelectShape s, const int32_t* blocks, const __grid_constant__ BlockLists l) {
    extern __shared__ uint32_t bits[];       // [words][nb]; where each word's queries begin, [words][nb]; [nb]
    const uint32_t u = blockIdx.x / (uint32_t)l.chunks, chunk = blockIdx.x - u * l.chunks;
    set_bits(s, blocks, l, u, chunk, bits);  // (the lists of blocks are no earlier kernel's)
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    int32_t* begin = reinterpret_cast<int32_t*>(bits + s.nb * l.words);
    uint32_t* shift = bits + 2 * s.nb * l.words;             // from G times an entry's place to its rows' position
    const int32_t *base = l.base + (int64_t)u * (s.nb + 1), *tile_base = l.tile_base + (int64_t)u * (s.nb + 1);
    for (int c = threadIdx.x; c < s.nb; c += blockDim.x) {
        int at = base[c] + l.counts[((int64_t)u * l.chunks + chunk) * s.nb + c];
        shift[c] = (uint32_t)tile_base[c] * kTileRows - (uint32_t)base[c] * s.G;
        for (int w = 0; w < l.words; ++w) {
            begin[w * s.nb + c] = at;
            at += __popc(bits[w * s.nb + c]);
        }
    }
    __syncthreads();
    uint32_t* entries = l.entries + u * s.n * l.ranks;
    uint32_t* positions = l.positions + u * s.n * l.ranks;
    const int w = threadIdx.x >> 5;
    const int64_t i0 = w < l.words ? ((int64_t)chunk * l.words + w) * 32 : s.n;
    each_live(s, blocks, u, i0, l.width,
              [&](int q, const int (&c)[4], const bool (&in)[4], int rank, int count) {
                  uint32_t p[4];
                  uint32_t* to = positions + (i0 + q) * l.ranks + rank;
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                      if (!in[j]) continue;
                      const int at = begin[w * s.nb + c[j]] + __popc(bits[w * s.nb + c[j]] & ((1u << q) - 1));
                      entries[at] = (uint32_t)(i0 + q);
                      p[j] = (uint32_t)at * s.G + shift[c[j]];
                  }
                  if (count == 4 && (reinterpret_cast<uintptr_t>(to) & 15) == 0) {
                      *reinterpret_cast<uint4*>(to) = make_uint4(p[0], p[1], p[2], p[3]);
                  } else {
#pragma unroll
                      for (int j = 0; j < 4; ++j)
                          if (in[j]) *to++ = p[j];
                  }
              },
              [&](int q, int count) { l.live[u * s.n + i0 + q] = count; });
}

}  // namespace

size_t plan_block_lists(const SelectShape& s, char* ws, BlockLists* l) {
    const size_t units = (size_t)s.B * s.Hk;
    l->ranks = s.top < s.nb ? s.top : s.nb;
    l->width = 1;
    while (4 * l->width < s.top) l->width *= 2;
    l->words = 8;
    while (l->words > 1 && (int64_t)s.nb * l->words * 4 > kBitmapBytes) l->words /= 2;
    l->chunks = (int32_t)((s.n + 32 * l->words - 1) / (32 * l->words));
    const int64_t named = s.n * l->ranks;    // (query, block) pairs of a unit
    l->most_filled = (int32_t)(named < s.nb ? named : s.nb);
    l->most_tiles = l->most_filled + named * s.G / kTileRows;
    l->shares = 1;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = ws ? ws + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    l->entries = reinterpret_cast<uint32_t*>(take(units * named * 4));
    l->base = reinterpret_cast<int32_t*>(take(units * (s.nb + 1) * 4));
    l->tile_base = reinterpret_cast<int32_t*>(take(units * (s.nb + 1) * 4));
    l->live = reinterpret_cast<int32_t*>(take(units * s.n * 4));
    l->positions = reinterpret_cast<uint32_t*>(take(units * named * 4));
    l->counts = reinterpret_cast<int32_t*>(take(units * l->chunks * s.nb * 4));
    return at;
}

int launch_block_lists(const SelectShape& s, const int32_t* blocks, const BlockLists& l, bool beside, cudaStream_t stream) {
    static std::atomic<uint64_t> count_ready{0}, fill_ready{0};
    const int64_t units = s.B * s.Hk, grid = units * l.chunks;
    if (grid > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    cudaError_t err = allow_smem(count_lists_kernel, kBitmapBytes, count_ready);
    if (err == cudaSuccess) err = allow_smem(fill_lists_kernel, 3 * kBitmapBytes, fill_ready);
    if (err != cudaSuccess) return cuda_fail(err, "the block lists");
    const size_t smem = (size_t)s.nb * l.words * 4;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        if (beside) {
            err = launch_pdl(count_lists_kernel, dim3((unsigned)grid), dim3(kThreads), smem, stream, s, blocks, l);
        } else {
            count_lists_kernel<<<(unsigned)grid, kThreads, smem, stream>>>(s, blocks, l);
            err = cudaGetLastError();
        }
    }
    if (err == cudaSuccess) {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        // A unit of more blocks than that is shared out, where its chunks are many too (2 x 262144 queries: 2.85 ms
        // for the attention with one block of threads a unit, 1.39 so; one head's 2^20: 108 and 24).
        if (s.nb <= kScanBlocks || l.chunks < 16) {
            err = launch_pdl(place_lists_kernel<true>, dim3((unsigned)units), dim3(kScanThreads), 0, stream, s, l);
        } else {
            const int parts = (s.nb + kPartBlocks - 1) / kPartBlocks;
            if (units * parts > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
            err = launch_pdl(sum_lists_kernel, dim3((unsigned)(units * parts)), dim3(kScanThreads), 0, stream, s, l, parts);
            if (err == cudaSuccess) {
                LaunchScope second(DIFFUSER_KERNEL_AUX, stream);
                err = launch_pdl(place_lists_kernel<false>, dim3((unsigned)units), dim3(kScanThreads), 0, stream, s, l);
            }
        }
    }
    if (err == cudaSuccess) {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        err = launch_pdl(fill_lists_kernel, dim3((unsigned)grid), dim3(kThreads), 2 * smem + (size_t)s.nb * 4, stream, s, blocks, l);
    }
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "the block lists");
}

}  // namespace dfs
