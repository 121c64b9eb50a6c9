// Internal declarations of the attention over chosen key blocks: the means of key blocks
// (block_means.cu), the choice of blocks for few queries (select_blocks.cu) and for many
// (select_tiles.cu; select_common.cuh has what both use), the attention (selected_attention.cu) and its
// backward pass (selected_backward.cu) on warp tiles (mma_tiles.cuh) and on tiles of gathered rows
// (row_tiles.cuh), the lists of queries that name a block (block_lists.cu), and their entry points
// (selected_abi.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "internal.h"

namespace dfs {

constexpr int kBlockKeys = 64;               // keys of a block
constexpr int kMaxTop = 64;                  // blocks that a query lists at most
constexpr int64_t kMaxKeys = 1 << 20;

// Queries against keys: n queries a head, Hq = G Hk heads, m keys, of which sequence b has lengths[b].
struct SelectShape {
    int64_t B, n, m;
    int32_t Hq, Hk, G, top, nb;              // nb = ceil(m / 64)
    bool causal;
    const int32_t* lengths;                  // [B] or null (m)
    const int32_t* starts;                   // [B] or null (length - n): position of query 0
};

#ifdef __CUDACC__
// Keys that query i of sequence b sees in the blocks that it lists: those below the result.
__device__ __forceinline__ int32_t row_limit(const SelectShape& s, int64_t b, int64_t i) {
    const int64_t len = s.lengths ? min(max((int64_t)s.lengths[b], (int64_t)0), s.m) : s.m;
    const int64_t p = (s.starts ? (int64_t)s.starts[b] : len - s.n) + i;
    if (p < 0 || p >= len) return 0;
    return (int32_t)(s.causal ? p + 1 : len);
}
// Unit u = b Hk + h of a launch (units are fewer than 2^31).
__device__ __forceinline__ uint32_t sequence_of(const SelectShape& s, int64_t u) { return (uint32_t)u / (uint32_t)s.Hk; }
__device__ __forceinline__ int32_t key_count(const SelectShape& s, int64_t b) {
    return s.lengths ? min(max(s.lengths[b], 0), (int32_t)s.m) : (int32_t)s.m;
}
#endif

int launch_block_means(const void* K, int64_t B, int64_t Hk, int64_t m, const int32_t* lengths, int64_t recent,
                       void* means, cudaStream_t stream);

// blocks [B][Hk][n][top]
int launch_select_blocks(const SelectShape& s, const void* Q, const void* means, int32_t sink, int32_t local,
                         int32_t* blocks, cudaStream_t stream);

struct SelectedArgs {
    SelectShape s;
    const __nv_bfloat16 *q, *k, *v;          // [B][Hq][n][64], [B][Hk][m][64]
    const int32_t* blocks;                   // [B][Hk][n][top]
    __nv_bfloat16* out;                      // [B][Hq][n][64]; backward: the forward's result
    float* lse;                              // [B][Hq][n] or null; backward: the forward's
    const __nv_bfloat16* dout;               // backward
    __nv_bfloat16 *dq, *dk, *dv;
};
size_t selected_workspace(const SelectShape& s);
int launch_selected(const SelectedArgs& a, char* ws, cudaStream_t stream);
size_t selected_backward_workspace(const SelectShape& s);
int launch_selected_backward(const SelectedArgs& a, char* ws, cudaStream_t stream);

}  // namespace dfs
