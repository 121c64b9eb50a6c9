// The queries that list a key block, block by block (block_lists.cu).
#pragma once

#include "selected.h"

namespace dfs {

// In device memory, for each unit (sequence and key head).  An entry is a query i and its rank
// among the query's blocks that count, i 64 + rank; a block's entries stand in rising order of i.
// Entry e of a block stands for G rows, e G + h for head h of the group; an item is up to
// `item_rows` rows of one block.
struct BlockLists {
    uint32_t* entries;             // [units][n ranks]
    int32_t* base;                 // [units][nb + 1]: where a block's entries begin
    int32_t* item_base;            // [units][nb + 1]: where its items do
    int4* items;                   // [units][most_items]: block, first row, rows, the block's first entry
    int32_t* live;                 // [units][n]: blocks of a query that count
    int32_t* counts;               // [units][chunks][nb], while they are built
    int32_t ranks;                 // blocks of a query that count, at most: min(top, nb)
    int32_t most_items, item_rows;
    int32_t words, chunks;         // queries of a chunk / 32; chunks
    int32_t width;                 // lanes that read a query's list
};

#ifdef __CUDACC__
struct ItemRows {
    int32_t block, first, rows;    // rows first .. first + rows - 1 of the block's
    const uint32_t* entries;       // the block's
};
// Item `at` of unit u; rows 0: there is none.
__device__ __forceinline__ ItemRows item_of(const BlockLists& l, const SelectShape& s, int64_t u, uint32_t at) {
    const int4 item = l.items[u * l.most_items + at];        // (whatever it holds where there is none)
    const bool live = (int32_t)at < l.item_base[u * (s.nb + 1) + s.nb];
    return {item.x, item.y, live ? item.z : 0, l.entries + u * s.n * l.ranks + (live ? item.w : 0)};
}
// Row ((u - u0) n + i) G + h of a group of units that begins with u0 (fewer than 2^31 rows).
struct RowOf {
    uint32_t entry;                // (u - u0) n + i
    int64_t place;                 // the row of [B][Hq][n]
};
__device__ __forceinline__ RowOf row_of(const SelectShape& s, int64_t u0, uint32_t row) {
    const uint32_t entry = s.G == 1 ? row : row / s.G, h = row - entry * s.G;
    const uint32_t ul = entry / (uint32_t)s.n, i = entry - ul * (uint32_t)s.n;
    // unit u = b Hk + x: head (b Hk + x) G + h of B Hq
    return {entry, ((u0 + ul) * s.G + h) * s.n + i};
}
#endif

// Rows of an item: four tiles of 128, fewer where there would be no two rounds of `resident` items
// an SM.
inline int32_t item_rows(const SelectShape& s, int resident) {
    const int64_t rows = s.B * s.Hq * s.n * (s.top < s.nb ? s.top : s.nb), wave = 152 * 2 * (int64_t)resident;
    return rows >= 512 * wave ? 512 : rows >= 256 * wave ? 256 : 128;
}

// Sizes, and the addresses in `ws` (null: sizes alone); returns the bytes.
size_t plan_block_lists(const SelectShape& s, int32_t item_rows, char* ws, BlockLists* l);
// The last kernel allows dependent launches.  `beside`: the launch before on the stream is the caller's own,
// allows dependent launches and writes nothing that the lists are made of.
int launch_block_lists(const SelectShape& s, const int32_t* blocks, const BlockLists& l, bool beside, cudaStream_t stream);

}  // namespace dfs
