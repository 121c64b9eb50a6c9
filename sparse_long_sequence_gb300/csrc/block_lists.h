// The queries that list a key block, block by block (block_lists.cu).
#pragma once

#include "selected.h"

namespace dfs {

constexpr int kTileRows = 128;               // rows of a tile

// In device memory, for each unit (sequence and key head).  An entry is a query; a block's entries
// stand in rising order.  Entry e of a block stands for G rows, e G + h for head h of the group, and a block's rows make
// tiles of 128, the last one shorter.  A unit's tiles, block after block, go to `shares` blocks of
// threads in runs of equal length: share j has tiles [j N / shares, (j + 1) N / shares) of N (with
// fewer tiles than shares there are N shares).
struct BlockLists {
    uint32_t* entries;             // [units][n ranks]
    int32_t* base;                 // [units][nb + 1]: where a block's entries begin
    int32_t* tile_base;            // [units][nb + 1]: where its tiles do
    int32_t* live;                 // [units][n]: blocks of a query that count
    uint32_t* positions;           // [units][n][ranks]: for each of them, where head 0's row is: tile 128 + row of it
    int32_t* counts;               // [units][chunks][nb], while they are built
    int32_t ranks;                 // blocks of a query that count, at most: min(top, nb)
    int32_t shares;
    int32_t most_filled;           // blocks that have entries, at most
    int64_t most_tiles;            // tiles of a unit, at most
    int32_t words, chunks;         // queries of a chunk / 32; chunks
    int32_t width;                 // lanes that read a query's list
};

// Sizes, and the addresses in `ws` (null: sizes alone); returns the bytes.  `shares` is the caller's.
size_t plan_block_lists(const SelectShape& s, char* ws, BlockLists* l);
// Shares of a unit where `here` units have `resident` blocks of threads on each of 152 SMs: `rounds` times as
// many as run at once, and a tile at least for each.
constexpr int kMostRounds = 3;
inline int32_t tile_shares(const SelectShape& s, const BlockLists& l, int64_t here, int resident, int rounds) {
    const int64_t at_once = 152 * resident / here, tiles = l.most_tiles;
    const int64_t shares = (at_once < 1 ? 1 : at_once) * rounds;
    return (int32_t)(shares < tiles ? shares : tiles < 1 ? 1 : tiles);
}
// Where the units have alike lengths one round is enough unless there are 64 tiles or more to a block of threads, of
// which some take longer (16 x 16384 queries: 429 us with one round, 422 with three; 24 x 4096, 17 tiles each: 95 and
// 100).  Units of unlike lengths have shares of unlike lengths, which more of them even out, and each has its
// start (lengths from a quarter to all, 8 blocks a query: 2 x 12 units of 1024 queries, 4 tiles a block of threads,
// 28 us with one round and 32 with two; of 4096, 17 tiles, 53 and 53, with three 58; 8 x 12 of 2048, 34 tiles, 145, 135
// and 130; the backward of 4 x 12 of 4096, 50 tiles, 255, 228 and 228).
inline int tile_rounds(const SelectShape& s, const BlockLists& l, int64_t here, int resident) {
    const int64_t tiles = l.most_tiles * here / (152 * resident);
    if (!s.lengths) return tiles < 64 ? 1 : kMostRounds;
    return tiles < 8 ? 1 : tiles < 48 ? 2 : kMostRounds;
}
// The last kernel allows dependent launches.  `beside`: the launch before on the stream is the caller's own,
// allows dependent launches and writes nothing that the lists are made of.
int launch_block_lists(const SelectShape& s, const int32_t* blocks, const BlockLists& l, bool beside, cudaStream_t stream);

#ifdef __CUDACC__
__device__ __forceinline__ int32_t share_begin(int32_t tiles, int32_t share, int32_t shares) {
    return (int32_t)((uint64_t)(uint32_t)tiles * (uint32_t)share / (uint32_t)shares);
}
// the share that has tile t
__device__ __forceinline__ int32_t share_of_tile(int32_t tiles, int32_t t, int32_t shares) {
    return (int32_t)((((uint64_t)(uint32_t)t + 1) * (uint32_t)shares - 1) / (uint32_t)tiles);
}

// A walk over a unit's tiles.
struct Walk {
    const int32_t *base, *tile_base;         // the unit's
    int32_t block, begin, end;               // a key block, its tiles
    int32_t first_entry, rows;               // its entries, its rows

    // to the block that has tile t (warp-wide)
    __device__ __forceinline__ void find(const BlockLists& l, const SelectShape& s, int64_t u, int32_t t) {
        base = l.base + u * (s.nb + 1);
        tile_base = l.tile_base + u * (s.nb + 1);
        const int lane = threadIdx.x & 31;
        int lo = 0, n = s.nb;                // among blocks lo .. lo + n - 1: the last with tile_base <= t
        while (n > 1) {
            const int step = (n + 31) / 32, c = lo + lane * step;
            const unsigned m = __ballot_sync(0xffffffffu, lane * step < n && tile_base[c] <= t);
            const int k = 31 - __clz(m);     // (lane 0's always is)
            lo += k * step;
            n = min(step, n - k * step);
        }
        block = lo;
        begin = tile_base[lo];
        end = tile_base[lo + 1];
        load(s);
    }
    // on to tile t, the next one
    __device__ __forceinline__ void go(const SelectShape& s, int32_t t) {
        if (t < end) return;
        do {
            ++block;
            begin = end;
            end = tile_base[block + 1];
        } while (t >= end);
        load(s);
    }
    __device__ __forceinline__ void load(const SelectShape& s) {
        first_entry = base[block];
        rows = (base[block + 1] - first_entry) * s.G;
    }
};

// Row ((u - u0) n + i) G + h of a group of units that begins with u0 (fewer than 2^31 rows).
struct RowOf {
    uint32_t entry;                // (u - u0) n + i
    uint32_t unit, head;           // u - u0, h
    int64_t place;                 // the row of [B][Hq][n]
};
__device__ __forceinline__ RowOf row_of(const SelectShape& s, int64_t u0, uint32_t row) {
    const uint32_t entry = s.G == 1 ? row : row / s.G, h = row - entry * s.G;
    const uint32_t ul = entry / (uint32_t)s.n, i = entry - ul * (uint32_t)s.n;
    // unit u = b Hk + x: head (b Hk + x) G + h of B Hq
    return {entry, ul, h, ((u0 + ul) * s.G + h) * s.n + i};
}
#endif

}  // namespace dfs
