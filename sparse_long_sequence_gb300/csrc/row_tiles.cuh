// Tiles of 128 gathered rows against a block of 64 keys on the tcgen05 tensor cores: what the
// attention over chosen blocks (selected_attention.cu) and its backward (selected_backward.cu) share.
//
// A tile in shared memory has rows of 128 bytes (64 bf16 values) under the 128-byte swizzle, 1024-byte
// aligned: as it lies it is a K-major operand whose rows are the product's rows (or columns) and, read
// MN-major, one whose rows are summed over.
#pragma once

#include "block_lists.h"
#include "dense_ptx.cuh"
#include "selected.h"

namespace dfs {
namespace tiles {

constexpr int kRowBytes = kHeadDim * 2;
constexpr int kTileBytes = kTileRows * kRowBytes;
constexpr int kKeyBytes = kBlockKeys * kRowBytes;

// Byte of 16-byte chunk `chunk` of a row.
__device__ __forceinline__ uint32_t place(int row, int chunk) { return row * kRowBytes + ((chunk ^ (row & 7)) << 4); }

// 16 bytes into shared memory; zeros, and nothing read, where `live` is false.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live ? 16 : 0) : "memory");
}
// The 64 keys (or values) at `from`, rows from `rows` on as zeros, by `threads` threads.
template <int kThreads>
__device__ __forceinline__ void copy_keys(uint32_t to, const __nv_bfloat16* from, int rows, int tid) {
#pragma unroll
    for (int x = tid; x < kBlockKeys * 8; x += kThreads) {
        const int r = x >> 3, c = x & 7;
        copy16(to + place(r, c), from + (r < rows ? r : 0) * kHeadDim + 8 * c, r < rows);
    }
}

// A lane's row of a tile.
struct Row {
    uint32_t at;                   // of [G][n]: head * n + query
    int32_t limit;                 // keys of the block that it sees (up to 64 or more); 0: there is no such row
};
// The entry of row `row` of the walk's block (any one of it where there is no such row).
__device__ __forceinline__ uint32_t entry_of(const Walk& w, const uint32_t* entries, int G, int row, uint32_t* head) {
    const uint32_t r = row < w.rows ? row : 0, e = G == 1 ? r : r / G;
    *head = r - e * G;
    return entries[w.first_entry + e];
}
__device__ __forceinline__ Row row_from(const SelectShape& s, int64_t b, int32_t key0, uint32_t entry, uint32_t head, bool live) {
    return {head * (uint32_t)s.n + entry, live ? row_limit(s, b, entry) - key0 : 0};
}
// Copies a warp's 32 rows (its lanes' own) of a tile from [G][n][64] at `from`.
__device__ __forceinline__ void copy_rows(uint32_t tile, const __nv_bfloat16* from, const Row& mine, int quarter, int lane) {
    const unsigned live = __ballot_sync(0xffffffffu, mine.limit > 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int r = 4 * j + (lane >> 3), c = lane & 7;
        const uint32_t at = __shfl_sync(0xffffffffu, mine.at, r);
        copy16(tile + place(32 * quarter + r, c), from + (int64_t)at * kHeadDim + 8 * c, live >> r & 1);
    }
}

// 32 bytes, a whole sector, in one store.
__device__ __forceinline__ void store32(float* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Partial sums of a tile, fp32 [128 rows][64], in the workspace as in shared memory: rows of 256 bytes, chunk c of
// 16 bytes in place c ^ (row & 7), so that the lanes of a warp, each with a row, fall in different banks.  A
// warp's 32 rows are one bulk copy: the copy engine takes them out while the warp goes on.  (Stores from registers
// fill the SM's queue to the memory, and everything behind them waits: 365 us where the whole kernel takes 123
// without them.)
constexpr int kSumsPitch = kHeadDim * 4;
constexpr int kSumsBytes = kTileRows * kSumsPitch;
// 32 of a row's 64 sums, to chunks 8 half ..
__device__ __forceinline__ void stage_sums(char* row, const uint32_t (&v)[32], int half, int lane) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(row + ((8 * half + c) ^ (lane & 7)) * 16) = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
}
// A warp's rows out, first to leave the L2 again: they are read once, after all of them are written, and the
// queries, keys and values are gathered many times meanwhile.
__device__ __forceinline__ void bulk_store_once(float* to, const char* from, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;" ::"l"(to),
                 "r"(ptx::smem_u32(from)), "r"(bytes), "l"(ptx::l2_evict_first())
                 : "memory");
}
// Four features of row `position` (tile 128 + row) of the partial sums: lane 0 .. 15's.
__device__ __forceinline__ float4 sums_at(const float* sums, uint32_t position, int lane) {
    return __ldcs(reinterpret_cast<const float4*>(sums) + (int64_t)position * 16 + (lane ^ (position & 7)));
}

}  // namespace tiles
}  // namespace dfs
