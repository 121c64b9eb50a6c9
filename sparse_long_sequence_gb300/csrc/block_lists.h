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
    int2* items;                   // [units][most_items]: block, first row
    int32_t* live;                 // [units][n]: blocks of a query that count
    int32_t* counts;               // [units][chunks][nb], while they are built
    int32_t ranks;                 // blocks of a query that count, at most: min(top, nb)
    int32_t most_items, item_rows;
    int32_t words, chunks;         // queries of a chunk / 32; chunks
};

#ifdef __CUDACC__
struct ItemRows {
    int32_t block, first, rows;    // rows first .. first + rows - 1 of the block's
    const uint32_t* entries;       // the block's
};
// Item `at` of unit u; rows 0: there is none.
__device__ __forceinline__ ItemRows item_of(const BlockLists& l, const SelectShape& s, int64_t u, int32_t at) {
    ItemRows r{0, 0, 0, nullptr};
    if (at >= l.item_base[u * (s.nb + 1) + s.nb]) return r;
    const int2 item = l.items[u * l.most_items + at];
    const int32_t* base = l.base + u * (s.nb + 1) + item.x;
    r.block = item.x;
    r.first = item.y;
    r.rows = min(l.item_rows, (base[1] - base[0]) * s.G - item.y);
    r.entries = l.entries + u * s.n * l.ranks + base[0];
    return r;
}
#endif

// Sizes, and the addresses in `ws` (null: sizes alone); returns the bytes.
size_t plan_block_lists(const SelectShape& s, int32_t item_rows, char* ws, BlockLists* l);
int launch_block_lists(const SelectShape& s, const int32_t* blocks, const BlockLists& l, cudaStream_t stream);

}  // namespace dfs
