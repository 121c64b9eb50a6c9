// Gradients of the attention over chosen key blocks, block by block as the forward:
//   P_ij = exp(q_i.k_j / 8 - lse_i),  dS_ij = P_ij (dout_i.v_j - delta_i) / 8,  delta_i = dout_i.out_i,
//   dv_j = sum_i P_ij dout_i,  dk_j = sum_i dS_ij q_i,  dq_i = sum_j dS_ij k_j.
//
// The rows (a query of a head) that list a key block (block_lists.cu) make tiles of 128, and a block of
// eight warps walks over a run of tiles, their q and dout gathered into shared memory a tile ahead.  On
// tcgen05: S = Q K^T and dout V^T; then P and dS, two threads a row, go to shared memory as bf16, from
// where dS K gives the rows' dq and one product of 128 x 128,
//   [dout | Q]^T [P | dS] = [dv^T, .; ., dk^T],
// adds up dv and dk in tensor memory over a block's rows (its other two quarters are not used: 64-row
// accumulators would save half of a product that is a tenth of the time).  A (row, block) leaves 64 fp32
// sums of dq in the order of the tiles, which a second kernel joins in a fixed order.  dk and dv of a block
// whose tiles one block of threads has are written at once; a run of tiles that holds a part of a block leaves
// its sums to the second kernel.
//
// Bound by the latency of a tile's steps (copies, products, P and dS, products, dq out: about 6700 cycles with
// two blocks of threads an SM, which 115 KB of shared memory each allow), then by dq's partials.  16 x 16384 causal queries
// of 16 blocks: 652 us, of which delta takes 15, the lists 41, the tiles 410 and the join 190 (1.07 GB at 5.7 TB/s).
#include <atomic>

#include "block_lists.h"
#include "layer_ops.h"
#include "mma_tiles.cuh"
#include "row_tiles.cuh"
#include "selected.h"

namespace dfs {
namespace {

using namespace tiles;

constexpr float kScale = 0.125f;             // 1 / sqrt(64)
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kThreads = 256;
constexpr int kStage = 2 * kTileBytes;       // a tile's dout and queries
constexpr int kSmem = 2 * kKeyBytes + 2 * kStage + 2 * kTileBytes;       // keys, values; two stages; P and dS
constexpr uint32_t kColumns = 256;           // tensor memory: S (then dq), dout V^T, dv^T and dk^T
constexpr int kResident = 2;                 // blocks of threads an SM
constexpr size_t kGroupBytes = size_t(1536) << 20;       // partials of a group of units

struct Partials {
    float* dq;                               // [units][tiles] of [128][64] (row_tiles.cuh)
    float* dkv;                              // [units][shares][2][dv, dk][64 features][64 keys]: the share's part of a
                                             // block that begins before it, and of one that goes on after it
    const float2* stat;                      // [B][Hq][n]: lse in units of log 2, delta / 8
    int64_t u0;
    bool first;                              // the group after the lists (the others: after the joining kernel)
};

// stat = (lse in units of log 2, delta / 8): eight lanes a row.
__global__ void __launch_bounds__(256) selected_delta_kernel(const __grid_constant__ SelectedArgs a, int64_t rows, float2* stat) {
    ptx::griddep_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
    const int lane = threadIdx.x & 7;
    float d = 0.f;
    if (row < rows) {
        const uint4 x = reinterpret_cast<const uint4*>(a.out + row * kHeadDim)[lane];
        const uint4 y = reinterpret_cast<const uint4*>(a.dout + row * kHeadDim)[lane];
        const uint32_t p[4] = {x.x, x.y, x.z, x.w}, q[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            d = fmaf(__uint_as_float(p[j] << 16), __uint_as_float(q[j] << 16), d);
            d = fmaf(__uint_as_float(p[j] & 0xffff0000u), __uint_as_float(q[j] & 0xffff0000u), d);
        }
    }
    d += __shfl_xor_sync(kFull, d, 1);
    d += __shfl_xor_sync(kFull, d, 2);
    d += __shfl_xor_sync(kFull, d, 4);
    if (row < rows && lane == 0) stat[row] = make_float2(a.lse[row] * kLog2e, d * kScale);
}

__global__ void __launch_bounds__(kThreads, kResident)
selected_grads_kernel(const __grid_constant__ SelectedArgs a, const __grid_constant__ BlockLists l, const Partials out,
                      int* status) {
    extern __shared__ __align__(1024) char smem[];
    __shared__ uint64_t bars[3];             // S and dout V^T are there; dq is; dv and dk have taken the tile
    __shared__ uint32_t tmem_slot;
    const SelectShape& s = a.s;
    // A group starts while the one before is joined (which the lists are older than), and writes no partial
    // before that is over.
    if (out.first) ptx::griddep_wait();
    const uint32_t ul = blockIdx.x / (uint32_t)l.shares;
    const int32_t share = blockIdx.x - ul * l.shares;
    const int64_t u = out.u0 + ul, b = sequence_of(s, u);
    const int32_t tiles = l.tile_base[u * (s.nb + 1) + s.nb];
    const int32_t shares = min(l.shares, tiles);
    if (share >= shares) {
        ptx::griddep_wait();
        return;
    }
    const int32_t first = share_begin(tiles, share, shares), last = share_begin(tiles, share + 1, shares);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);      // (one value a warp)
    const int quarter = warp & 3, half = warp >> 2;          // rows 32 quarter .. and columns 32 half .. of a tile
    const uint32_t keys = ptx::smem_u32(smem), values = keys + kKeyBytes, stages = values + kKeyBytes;
    const uint32_t weights = stages + 2 * kStage;            // P, then dS
    const int64_t head0 = u * s.G * s.n;                     // row 0 of the unit's [G][n]
    // half 0 copies dout, half 1 the queries
    const __nv_bfloat16* from = (half ? a.q : a.dout) + head0 * kHeadDim;
    const uint32_t* entries = l.entries + u * s.n * l.ranks;
    const int32_t len = key_count(s, b);
    auto copy_block = [&](int32_t block) {
        const int64_t at = (u * s.m + (int64_t)block * kBlockKeys) * kHeadDim;
        const int rows = min(kBlockKeys, len - block * kBlockKeys);
        copy_keys<kThreads>(keys, a.k + at, rows, tid);
        copy_keys<kThreads>(values, a.v + at, rows, tid);
    };
    const int mine = 32 * quarter + lane;                    // this thread's row of a tile
    // tile x is worked on, the rows of x + 1 are known, the entries of x + 2 are being looked up
    Walk walk;
    walk.find(l, s, u, first);
    uint32_t head, entry;
    int32_t row = (first - walk.begin) * kTileRows + mine, block = walk.block, block_next;
    int32_t begin = walk.begin, end = walk.end, begin_next, end_next;        // their tiles
    entry = entry_of(walk, entries, s.G, row, &head);
    copy_block(block);
    int32_t count, count_next = walk.rows - (row - lane);    // rows from this warp's first on
    Row next = row_from(s, b, block * kBlockKeys, entry, head, row < walk.rows);
    copy_rows(stages + half * kTileBytes, from, next, quarter, lane);
    float2 stat, stat_next = out.stat[head0 + next.at];
    auto look = [&](int32_t x) {
        if (x >= last) return;
        walk.go(s, x);
        row = (x - walk.begin) * kTileRows + mine;
        entry = entry_of(walk, entries, s.G, row, &head);
    };
    look(first + 1);
    __syncwarp();
    if (warp == 0) ptx::tmem_alloc(&tmem_slot, kColumns);
    if (tid == 0) {
#pragma unroll
        for (int j = 0; j < 3; ++j) ptx::mbar_init(&bars[j], 1);
        ptx::fence_mbar_init();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot, col = tmem + ((uint32_t)(32 * quarter) << 16) + 32 * half;
    constexpr uint32_t kScores = ptx::mma_idesc_bf16(kTileRows, kBlockKeys, false, false);
    constexpr uint32_t kQueryGrad = ptx::mma_idesc_bf16(kTileRows, kHeadDim, false, true);
    constexpr uint32_t kKeyGrad = ptx::mma_idesc_bf16(2 * kHeadDim, 2 * kBlockKeys, true, true);
    const int64_t tile0 = (int64_t)ul * l.most_tiles;
    char* sums = smem + (weights - keys) + 32 * quarter * kSumsPitch;    // its rows' dq on their way out, two warps'
    uint32_t phase = 0;                      // of the barriers, and the stage
    bool fresh = true;                       // no tile of the block is in dv and dk yet

    for (int32_t x = first; x < last; ++x, phase ^= 1) {
        const uint32_t stage = stages + phase * kStage;
        ptx::cp_async_wait_all();
        ptx::fence_proxy_async_smem();
        __syncthreads();                     // the tile is there, and all have read the last dq
        if (warp == 0) {
            __syncwarp();
            ptx::tc_fence_after();
            const uint64_t dd = ptx::sw128_kmajor_desc(stage), qd = ptx::sw128_kmajor_desc(stage + kTileBytes);
            const uint64_t kd = ptx::sw128_kmajor_desc(keys), vd = ptx::sw128_kmajor_desc(values);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (ptx::elect_one()) ptx::mma_bf16_ss(tmem, qd + 2 * e, kd + 2 * e, kScores, e > 0);
                if (ptx::elect_one()) ptx::mma_bf16_ss(tmem + 64, dd + 2 * e, vd + 2 * e, kScores, e > 0);
            }
            if (ptx::elect_one()) ptx::mma_commit(&bars[0]);
        }
        __syncwarp();
        const int limit = next.limit - 32 * half;
        count = count_next;
        stat = stat_next;
        block_next = walk.block;
        begin_next = walk.begin;
        end_next = walk.end;
        if (x + 1 < last) {                  // (the other stage is free: dv and dk have taken it)
            next = row_from(s, b, block_next * kBlockKeys, entry, head, row < walk.rows);
            count_next = walk.rows - (row - lane);
            copy_rows(stages + (phase ^ 1) * kStage + half * kTileBytes, from, next, quarter, lane);
            stat_next = out.stat[head0 + next.at];
            look(x + 2);
        }
        uint32_t sc[32], dp[32];
        ptx::mbar_wait(&bars[0], phase, status);
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_ld32_issue(col, sc);
        ptx::tmem_ld32_issue(col + 64, dp);
        ptx::tmem_ld_wait32(sc);
        ptx::tmem_ld_wait32(dp);
        // sc and dp become P and dS, two bf16 a register, in their first halves.  (Rounded so, half a step of each term of
        // their sums, they put the gradients 2.8e-3 off in the 2-norm where the results' own rounding leaves 2.0e-3.  Low
        // parts beside them, as the forward has, would take 32 KB more: one block of threads an SM.)
        const bool whole = __all_sync(kFull, limit >= 32);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            float w[2], g[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[e] = exp2_fast(fmaf(__uint_as_float(sc[k + e]), kScale * kLog2e, -stat.x));
                g[e] = w[e] * (__uint_as_float(dp[k + e]) * kScale - stat.y);
                if (!whole && k + e >= limit) w[e] = g[e] = 0.f;
            }
            sc[k / 2] = pack(w[0], w[1]);
            dp[k / 2] = pack(g[0], g[1]);
        }
        if (lane == 0) ptx::bulk_wait_read<0>();             // the last dq has left by the place of P and dS
        __syncthreads();
        char* to = smem + (weights - keys);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t at = place(mine, 4 * half + c);
            *reinterpret_cast<uint4*>(to + at) = make_uint4(sc[4 * c], sc[4 * c + 1], sc[4 * c + 2], sc[4 * c + 3]);
            *reinterpret_cast<uint4*>(to + kTileBytes + at) = make_uint4(dp[4 * c], dp[4 * c + 1], dp[4 * c + 2], dp[4 * c + 3]);
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncthreads();                     // P and dS are whole
        if (warp == 0) {
            __syncwarp();
            ptx::tc_fence_after();
            const uint64_t sd = ptx::sw128_kmajor_desc(weights + kTileBytes), kd = ptx::sw128_mnmajor_desc(keys, kKeyBytes);
#pragma unroll
            for (int e = 0; e < 4; ++e) if (ptx::elect_one()) ptx::mma_bf16_ss(tmem, sd + 2 * e, kd + 128 * e, kQueryGrad, e > 0);
            if (ptx::elect_one()) ptx::mma_commit(&bars[1]);
            const uint64_t ad = ptx::sw128_mnmajor_desc(stage, kTileBytes), bd = ptx::sw128_mnmajor_desc(weights, kTileBytes);
#pragma unroll
            for (int e = 0; e < 8; ++e) if (ptx::elect_one()) ptx::mma_bf16_ss(tmem + 128, ad + 128 * e, bd + 128 * e, kKeyGrad, !fresh || e > 0);
            if (ptx::elect_one()) ptx::mma_commit(&bars[2]);
        }
        __syncwarp();
        if (x == first) ptx::griddep_wait();              // (the joining kernel is let in by the end alone)
        ptx::mbar_wait(&bars[1], phase, status);
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_ld32_issue(col, sc);
        ptx::tmem_ld_wait32(sc);
        ptx::mbar_wait(&bars[2], phase, status);             // P and dS are free: dq leaves by their place
        __syncwarp();
        stage_sums(sums + lane * kSumsPitch, sc, half, lane);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        ptx::named_barrier_sync(1 + quarter, 64);            // the rows' two warps
        if (half == 0 && lane == 0 && count > 0) {
            bulk_store_once(out.dq + ((tile0 + x) * kTileRows + 32 * quarter) * kHeadDim, sums, min(count, 32) * kSumsPitch);
            ptx::bulk_commit();
        }
        __syncwarp();
        fresh = x + 1 == last || block_next != block;
        if (fresh) {                         // the run's last tile of the block
            if (x + 1 < last) copy_block(block_next);        // (dq is there: keys and values are done with)
            __syncwarp();
            ptx::tc_fence_after();
            // lanes 0 .. 63: feature of dout, dv^T in the first 64 columns; 64 .. 127: feature of q, dk^T in the others
            ptx::tmem_ld32_issue(col + 128 + (quarter >> 1) * 64, sc);
            ptx::tmem_ld_wait32(sc);
            const int which = quarter >> 1, feature = mine & 63;
            if (begin >= first && end <= last) {             // all of the block: turned by the place of its last tile
                __nv_bfloat16* turned = reinterpret_cast<__nv_bfloat16*>(smem + (stage - keys) + which * kKeyBytes);
#pragma unroll
                for (int k = 0; k < 32; ++k) turned[(32 * half + k) * kHeadDim + feature] = __float2bfloat16_rn(__uint_as_float(sc[k]));
                __syncwarp();
                ptx::named_barrier_sync(5 + which, 128);
                const int rows = (int)min((int64_t)kBlockKeys, s.m - (int64_t)block * kBlockKeys);
                uint4* dst = reinterpret_cast<uint4*>((which ? a.dk : a.dv) + (u * s.m + (int64_t)block * kBlockKeys) * kHeadDim);
                const int x0 = 64 * (quarter & 1) + 32 * half + lane;        // of the four warps' threads
#pragma unroll
                for (int x = x0; x < kBlockKeys * 8; x += 128)
                    if (x < rows * 8) dst[x] = reinterpret_cast<const uint4*>(turned)[x];
            } else {
                const int64_t run = ((int64_t)blockIdx.x * 2 + (begin < first ? 0 : 1)) * 2 * kHeadDim;
                float* dst = out.dkv + (run + mine) * kBlockKeys + 32 * half;
#pragma unroll
                for (int j = 0; j < 4; ++j) store32(dst + 8 * j, sc + 8 * j);
            }
            block = block_next;
            begin = begin_next;
            end = end_next;
        }
        ptx::tc_fence_before();
    }
    if (lane == 0) ptx::bulk_wait<0>();
    __syncthreads();
    __syncwarp();
    if (warp == 0) ptx::tmem_dealloc(tmem, kColumns);
}

constexpr int kJoined = 4;                   // partials in flight

// dq of a row: the sum of its partials, sixteen lanes a row, sixteen rows a block of threads.
__device__ __forceinline__ void join_dq(const SelectedArgs& a, const BlockLists& l, const Partials& in, uint32_t row) {
    const SelectShape& s = a.s;
    const int lane = threadIdx.x & 15;
    const RowOf at = row_of(s, in.u0, row);
    const int count = l.live[in.u0 * s.n + at.entry];
    const uint32_t* position = l.positions + (in.u0 * s.n + at.entry) * l.ranks;
    const float* sums = in.dq + at.unit * l.most_tiles * (kSumsBytes / 4);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < count; x0 += kJoined) {            // a few partials at a time
        uint32_t p[kJoined];
        float4 v[kJoined];
#pragma unroll
        for (int x = 0; x < kJoined; ++x) p[x] = x0 + x < count ? position[x0 + x] + at.head : ~0u;
#pragma unroll
        for (int x = 0; x < kJoined; ++x) v[x] = x0 + x < count ? sums_at(sums, p[x], lane) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < kJoined; ++x) y = make_float4(y.x + v[x].x, y.y + v[x].y, y.z + v[x].z, y.w + v[x].w);
    }
    reinterpret_cast<uint2*>(a.dq + at.place * kHeadDim)[lane] = make_uint2(pack(y.x, y.y), pack(y.z, y.w));
}

// dk and dv of a key block: the sums of its runs', turned, sixteen keys a block of threads.
constexpr int kSplit = 4;
__device__ __forceinline__ void join_dkv(const SelectedArgs& a, const BlockLists& l, const Partials& in, uint32_t share) {
    __shared__ float sums[16][kHeadDim + 1];
    const SelectShape& s = a.s;
    const int split = share % (2 * kSplit), part = split % kSplit, which = split / kSplit;
    const uint32_t at = share / (2 * kSplit), ul = at / (uint32_t)s.nb;
    const int64_t u = in.u0 + ul;
    const int c = at - ul * s.nb, feature = threadIdx.x >> 2, four = threadIdx.x & 3;
    const int32_t* tile_base = l.tile_base + u * (s.nb + 1);
    const int32_t tiles = tile_base[s.nb], begin = tile_base[c], end = tile_base[c + 1];
    int from = 0, to = 0;                    // the shares that have its tiles
    if (begin < end) {
        from = share_of_tile(tiles, begin, min(l.shares, tiles));
        to = share_of_tile(tiles, end - 1, min(l.shares, tiles)) + 1;
        if (to == from + 1) return;          // (written already)
    }
    // the first share's part goes on after it, the others' begin before them
    const int64_t unit = (int64_t)ul * l.shares * 2;
    const float* src = in.dkv + ((unit * 2 + which) * kHeadDim + feature) * kBlockKeys + 16 * part + 4 * four;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = 0; x < to - from; ++x) {
        const int64_t run = 2 * (from + x) + (x == 0);
        const float4 p = *reinterpret_cast<const float4*>(src + run * 2 * kHeadDim * kBlockKeys);
        y = make_float4(y.x + p.x, y.y + p.y, y.z + p.z, y.w + p.w);
    }
    sums[4 * four][feature] = y.x;
    sums[4 * four + 1][feature] = y.y;
    sums[4 * four + 2][feature] = y.z;
    sums[4 * four + 3][feature] = y.w;
    __syncthreads();
    const int row = threadIdx.x >> 4, f = 4 * (threadIdx.x & 15);
    const int64_t key = (int64_t)c * kBlockKeys + 16 * part + row;
    if (key >= s.m) return;
    __nv_bfloat16* dst = (which ? a.dk : a.dv) + (u * s.m + key) * kHeadDim + f;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack(sums[row][f], sums[row][f + 1]), pack(sums[row][f + 2], sums[row][f + 3]));
}

__global__ void __launch_bounds__(256)
selected_join_grads_kernel(const __grid_constant__ SelectedArgs a, const __grid_constant__ BlockLists l, const Partials in,
                           uint32_t rows, uint32_t row_blocks) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    if (blockIdx.x >= row_blocks) return join_dkv(a, l, in, blockIdx.x - row_blocks);
    const uint32_t row = (row_blocks - 1 - blockIdx.x) * 16 + (threadIdx.x >> 4);      // (the last tiles' partials are in the L2)
    if (row < rows) join_dq(a, l, in, row);
}

struct Plan {
    BlockLists lists;
    int64_t group;                           // units whose partials are held at once
    size_t stat, dq, dkv, total;
};
Plan plan_backward(const SelectShape& s, char* ws) {
    Plan p;
    p.stat = plan_block_lists(s, ws, &p.lists);
    p.dq = p.stat + (s.B * s.Hq * s.n * 8 + 255) / 256 * 256;
    const int64_t units = s.B * s.Hk, dq = p.lists.most_tiles * kSumsBytes;
    const int64_t groups = (units * dq + (int64_t)kGroupBytes - 1) / (int64_t)kGroupBytes;
    p.group = groups < 1 ? units : groups < units ? (units + groups - 1) / groups : 1;
    // (room for any lengths, which a size query does not know)
    const int64_t most = tile_shares(s, p.lists, p.group, kResident, kMostRounds);
    p.lists.shares = tile_shares(s, p.lists, p.group, kResident, tile_rounds(s, p.lists, p.group, kResident));
    p.dkv = p.dq + p.group * dq;
    p.total = p.dkv + p.group * most * 2 * 2 * kBlockKeys * kHeadDim * 4;
    return p;
}

}  // namespace

size_t selected_backward_workspace(const SelectShape& s) {
    return s.B * s.n * s.m == 0 ? 0 : plan_backward(s, nullptr).total;
}

int launch_selected_backward(const SelectedArgs& a, char* ws, cudaStream_t stream) {
    const SelectShape& s = a.s;
    const Plan p = plan_backward(s, ws);
    static std::atomic<uint64_t> ready{0};
    int* status = nullptr;
    int st = ready_status(&status);
    if (st) return st;
    cudaError_t err = allow_smem(selected_grads_kernel, kSmem, ready);
    if (err != cudaSuccess) return cuda_fail(err, "selected_grads_kernel");
    const int64_t units = s.B * s.Hk, all = s.B * s.Hq * s.n;
    if ((all + 31) / 32 > INT32_MAX || p.group * p.lists.shares > INT32_MAX ||
        p.group * (s.n * s.G + s.nb * 2 * kSplit) > INT32_MAX)
        return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        selected_delta_kernel<<<(unsigned)((all + 31) / 32), 256, 0, stream>>>(a, all, reinterpret_cast<float2*>(ws + p.stat));
    }
    err = cudaGetLastError();
    if (err != cudaSuccess) return cuda_fail(err, "selected_delta_kernel");
    if ((st = launch_block_lists(s, a.blocks, p.lists, true, stream))) return st;
    for (int64_t u0 = 0; u0 < units && err == cudaSuccess; u0 += p.group) {
        const int64_t here = units - u0 < p.group ? units - u0 : p.group, rows = here * s.n * s.G;
        const Partials part{reinterpret_cast<float*>(ws + p.dq), reinterpret_cast<float*>(ws + p.dkv),
                            reinterpret_cast<const float2*>(ws + p.stat), u0, u0 == 0};
        {
            LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
            err = launch_pdl(selected_grads_kernel, dim3((unsigned)(here * p.lists.shares)), dim3(kThreads), kSmem, stream, a,
                             p.lists, part, status);
        }
        if (err == cudaSuccess) {
            LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
            const int64_t row_blocks = (rows + 15) / 16;
            err = launch_pdl(selected_join_grads_kernel, dim3((unsigned)(row_blocks + here * s.nb * 2 * kSplit)), dim3(256), 0,
                             stream, a, p.lists, part, (uint32_t)rows, (uint32_t)row_blocks);
        }
    }
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "selected_grads_kernel");
}

}  // namespace dfs
