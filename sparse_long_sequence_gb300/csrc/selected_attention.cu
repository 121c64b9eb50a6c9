// Attention over the key blocks that each query lists:
//   out_i = sum_j p_ij v_j,  p_ij = exp(q_i.k_j / 8 - lse_i),
// j over the visible keys of the listed blocks; a row without such keys is 0, its lse -infinity.
//
// Few queries: one block of threads for a query and up to eight heads of its group (the eight
// columns of the products).  Its warps take the listed blocks in turn, each with a running maximum
// and sum in registers, and join through shared memory.  A block's keys and values go from global
// memory into the products' registers.  Bound by the cache's bytes, or by a launch and the latency of two
// dependent loads (16 tokens, 16 heads of 4 key heads, 16 blocks of a cache of up to 65536 keys: 7.5 us; the bytes 2.5).
//
// Many queries: block by block.  The rows (a query of a head) that list a key block (block_lists.cu) make
// tiles of 128, and a block of four warps walks over a run of tiles: the rows' queries are gathered
// into shared memory a tile ahead, S = Q K^T and O = P V run on tcgen05 with P handed over through tensor
// memory in S's place (as two bf16 parts, mma_tiles.cuh: rounded to one it costs 2.2e-3 of the result in the 2-norm for
// the 1.7e-3 of its own rounding, and saves 11 us of 422), and each thread has one row's scores, maximum and sum,
// without exchanges.  Each (row, block)
// leaves a partial result in the order of the tiles: 64 fp32 sums, its maximum and its sum; a second kernel
// joins a row's partials.  Bound by the partials' way to HBM and back: 256 bytes for 8192 multiplications and
// additions of a row's scores and as many of its values.  16 x 16384 causal queries of 16 blocks: 422 us, of
// which the lists take 41, the tiles 216 (1.07 GB out at 5.0 TB/s) and the join 165 (6.5 TB/s).
#include <atomic>

#include "block_lists.h"
#include "layer_ops.h"
#include "mma_tiles.cuh"
#include "row_tiles.cuh"
#include "selected.h"

namespace dfs {
namespace {

using namespace tiles;

constexpr float kScale2 = 0.125f * 1.4426950408889634f;      // 1 / sqrt(64) in units of log 2
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kFewWarps = 16;

// The listed blocks that count: entry x of a query's list does if it is above all entries before it
// (which -1 is not) and has visible keys.  Warp-wide; bit x of the result.
__device__ __forceinline__ uint64_t live_slots(const int32_t* list, int top, int32_t limit, int lane) {
    uint64_t live = 0;
    int before = -1;
    for (int x0 = 0; x0 < top; x0 += 32) {
        const int x = x0 + lane;
        const int c = x < top ? list[x] : -1;
        int high = c;                                        // the largest up to this lane
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
            const int o = __shfl_up_sync(kFull, high, off);
            if (lane >= off) high = max(high, o);
        }
        int prev = __shfl_up_sync(kFull, high, 1);
        prev = max(lane ? prev : -1, before);
        const bool in = c > prev && (int64_t)c * kBlockKeys < limit;
        live |= (uint64_t)__ballot_sync(kFull, in) << x0;
        before = max(before, __shfl_sync(kFull, high, 31));
    }
    return live;
}

__global__ void __launch_bounds__(32 * kFewWarps) selected_few_kernel(const __grid_constant__ SelectedArgs a) {
    __shared__ float part[kFewWarps][8][kHeadDim];
    __shared__ float2 stat[kFewWarps][8];                    // maximum (of scores in units of log 2), sum
    const SelectShape& s = a.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int warps = blockDim.x >> 5, octets = (s.G + 7) / 8;
    const uint32_t row = octets == 1 ? blockIdx.x : blockIdx.x / octets;
    const int64_t u = s.n == 1 ? row : row / (uint32_t)s.n, i = row - u * s.n, b = sequence_of(s, u);
    const int h0 = (int)(blockIdx.x - row * octets) * 8, heads = min(8, s.G - h0);
    const int64_t first = (u * s.G + h0) * s.n + i;                // row of head h: + h n
    const int32_t limit = row_limit(s, b, i);
    const int32_t* list = a.blocks + (int64_t)row * s.top;

    uint32_t q[8];
    load_row(a.q + (first + g * s.n) * kHeadDim, g < heads, t, q);
    float o[4][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j >> 2][j & 3] = 0.f;
    uint64_t live = live_slots(list, s.top, limit, lane);
    for (int k = 0; live; ++k, live &= live - 1) {
        if (k % warps != warp) continue;
        const int32_t c = list[__ffsll((long long)live) - 1];
        const int64_t key0 = (int64_t)c * kBlockKeys;
        const int rows = min(kBlockKeys, (int)(limit - key0));
        uint32_t keys[8][8], values[8][8];
        load_keys(a.k + (u * s.m + key0) * kHeadDim, rows, lane, keys);
        load_keys(a.v + (u * s.m + key0) * kHeadDim, rows, lane, values);
        float x[4][4];
        score(keys, q, x);
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int M = 0; M < 4; ++M)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[M][j] = 16 * M + 8 * (j >> 1) + g < rows ? x[M][j] * kScale2 : -INFINITY;
                top[j & 1] = fmaxf(top[j & 1], x[M][j]);
            }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float now = fmaxf(m[e], column_max(top[e]));
            const float base = now == -INFINITY ? 0.f : now, shrink = exp2_fast(m[e] - base);
            float sum = 0.f;
#pragma unroll
            for (int M = 0; M < 4; ++M)
#pragma unroll
                for (int j = e; j < 4; j += 2) {
                    x[M][j] = exp2_fast(x[M][j] - base);
                    sum += x[M][j];
                }
            l[e] = l[e] * shrink + column_sum(sum);
            m[e] = now;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[j][e] *= shrink;
                o[j][e + 2] *= shrink;
            }
        }
        turn_values(values);
        weigh(values, x, o);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float* dst = &part[warp][2 * t + e][8 * g];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<float4*>(dst + 4 * j) = make_float4(o[2 * j][e], o[2 * j][e + 2], o[2 * j + 1][e], o[2 * j + 1][e + 2]);
        if (g == 0) stat[warp][2 * t + e] = make_float2(m[e], l[e]);
    }
    __syncthreads();
    for (int x = threadIdx.x; x < heads * 32; x += blockDim.x) {
        const int h = x >> 5, f = 2 * (x & 31);
        float top = -INFINITY;
        for (int w = 0; w < warps; ++w) top = fmaxf(top, stat[w][h].x);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f, y0 = 0.f, y1 = 0.f;
        for (int w = 0; w < warps; ++w) {
            const float e = exp2_fast(stat[w][h].x - base);
            sum += e * stat[w][h].y;
            y0 += e * part[w][h][place_of(f)];
            y1 += e * part[w][h][place_of(f + 1)];
        }
        const float r = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t at = first + h * s.n;
        *reinterpret_cast<uint32_t*>(a.out + at * kHeadDim + f) = pack(y0 * r, y1 * r);
        if (a.lse && f == 0) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

int launch_few(const SelectedArgs& a, cudaStream_t stream) {
    const SelectShape& s = a.s;
    const int64_t grid = s.B * s.Hk * s.n * ((s.G + 7) / 8);
    if (grid > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    // as many as fit an SM with another block of threads beside them, twice that where each has an SM to itself
    // (16 queries, 4 key heads, 16 blocks: 8.7 us with 8 warps)
    const int most = grid <= 152 ? kFewWarps : kFewWarps / 2, warps = s.top < most ? s.top : most;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        selected_few_kernel<<<(unsigned)grid, 32 * warps, 0, stream>>>(a);
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "selected_few_kernel");
}

constexpr int kTileThreads = 128;
constexpr int kTileSmem = 3 * kKeyBytes + kTileBytes + kSumsBytes;       // keys, two blocks' values, queries, sums
constexpr int kTileResident = 3;                             // blocks of threads an SM
constexpr uint32_t kTileColumns = 128;                       // tensor memory: S (then P) and O
constexpr size_t kGroupBytes = size_t(1280) << 20;           // partials of a group of units

// Partials of the units u0 .., [units][tiles].
struct Partials {
    float* sums;                             // [128][64] of a tile (row_tiles.cuh)
    float2* stat;                            // [128] of a tile: maximum (units of log 2), sum
    int64_t u0;
    bool first;                              // the group after the lists (the others: after a join)
};

__global__ void __launch_bounds__(kTileThreads, kTileResident)
selected_tiles_kernel(const __grid_constant__ SelectedArgs a, const __grid_constant__ BlockLists l, const Partials out,
                      int* status) {
    extern __shared__ __align__(1024) char smem[];
    __shared__ uint64_t bars[2];             // S is there; O is
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
    const uint32_t keys = ptx::smem_u32(smem), values = keys + kKeyBytes, queries = values + 2 * kKeyBytes;
    char* sums = smem + 3 * kKeyBytes + kTileBytes + 32 * warp * kSumsPitch; // this warp's rows on their way out
    const __nv_bfloat16* q0 = a.q + u * s.G * s.n * kHeadDim;
    const uint32_t* entries = l.entries + u * s.n * l.ranks;
    const int32_t len = key_count(s, b);
    auto copy_block = [&](int32_t block, uint32_t to_values) {
        const int64_t from = (u * s.m + (int64_t)block * kBlockKeys) * kHeadDim;
        const int rows = min(kBlockKeys, len - block * kBlockKeys);
        copy_keys<kTileThreads>(keys, a.k + from, rows, tid);
        copy_keys<kTileThreads>(to_values, a.v + from, rows, tid);
    };
    // tile x is worked on, the rows of x + 1 are known, the entries of x + 2 are being looked up
    Walk walk;
    walk.find(l, s, u, first);
    uint32_t head, entry;
    int32_t row = (first - walk.begin) * kTileRows + tid, block = walk.block, block_next;
    int32_t count = walk.rows - (row - lane), count_next;    // rows from this warp's first on
    entry = entry_of(walk, entries, s.G, row, &head);
    copy_block(block, values);
    Row now, next = row_from(s, b, block * kBlockKeys, entry, head, row < walk.rows);
    copy_rows(queries, q0, next, warp, lane);
    count_next = count;
    auto look = [&](int32_t x) {
        if (x >= last) return;
        walk.go(s, x);
        row = (x - walk.begin) * kTileRows + tid;
        entry = entry_of(walk, entries, s.G, row, &head);
    };
    look(first + 1);
    __syncwarp();
    if (warp == 0) ptx::tmem_alloc(&tmem_slot, kTileColumns);
    if (tid == 0) {
        ptx::mbar_init(&bars[0], 1);
        ptx::mbar_init(&bars[1], 1);
        ptx::fence_mbar_init();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot, mine = tmem + ((uint32_t)(32 * warp) << 16);
    constexpr uint32_t kScores = ptx::mma_idesc_bf16(kTileRows, kBlockKeys, false, false);
    constexpr uint32_t kSums = ptx::mma_idesc_bf16(kTileRows, kHeadDim, false, true);
    const int64_t tile0 = (int64_t)ul * l.most_tiles;
    uint32_t side = 0, phase = 0;            // which values; the barriers' phase

    for (int32_t x = first; x < last; ++x, phase ^= 1) {
        ptx::cp_async_wait_all();
        ptx::fence_proxy_async_smem();
        __syncthreads();                     // the tile is there, and all have read the last O
        if (warp == 0) {
            __syncwarp();
            ptx::tc_fence_after();
            const uint64_t qd = ptx::sw128_kmajor_desc(queries), kd = ptx::sw128_kmajor_desc(keys);
#pragma unroll
            for (int e = 0; e < 4; ++e) if (ptx::elect_one()) ptx::mma_bf16_ss(tmem, qd + 2 * e, kd + 2 * e, kScores, e > 0);
            if (ptx::elect_one()) ptx::mma_commit(&bars[0]);
        }
        __syncwarp();
        now = next;
        count = count_next;
        block_next = walk.block;
        next = row_from(s, b, block_next * kBlockKeys, entry, head, row < walk.rows);
        count_next = walk.rows - (row - lane);
        look(x + 2);
        uint32_t lo[32], hi[32];
        ptx::mbar_wait(&bars[0], phase, status);
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_ld32_issue(mine, lo);
        ptx::tmem_ld32_issue(mine + 32, hi);
        const uint32_t values_now = values + side * kKeyBytes;
        if (x + 1 < last) {                  // S is there: the queries' and the keys' places are free
            if (block_next != block) {
                side ^= 1;
                block = block_next;
                copy_block(block, values + side * kKeyBytes);
            }
            copy_rows(queries, q0, next, warp, lane);
        }
        ptx::tmem_ld_wait32(lo);
        ptx::tmem_ld_wait32(hi);
        float top = -INFINITY;
        if (__all_sync(kFull, now.limit >= kBlockKeys)) {
#pragma unroll
            for (int j = 0; j < 32; ++j) top = fmaxf(top, fmaxf(__uint_as_float(lo[j]), __uint_as_float(hi[j])));
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (j >= now.limit) lo[j] = 0xff800000u;     // -infinity
                if (j + 32 >= now.limit) hi[j] = 0xff800000u;
                top = fmaxf(top, fmaxf(__uint_as_float(lo[j]), __uint_as_float(hi[j])));
            }
        }
        top *= kScale2;
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        auto weights = [&](const uint32_t (&x)[32], uint32_t to) {   // to columns `to` .., and what their rounding leaves to 32 on
            uint32_t high[16], low[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float w0 = exp2_fast(fmaf(__uint_as_float(x[2 * j]), kScale2, -base));
                const float w1 = exp2_fast(fmaf(__uint_as_float(x[2 * j + 1]), kScale2, -base));
                sum += w0 + w1;
                split_weights(w0, w1, &high[j], &low[j]);
            }
            __syncwarp();
            ptx::tmem_st16x2(to, high, to + 32, low);
        };
        weights(lo, mine);
        weights(hi, mine + 16);
        ptx::tc_fence_before();
        __syncthreads();                     // P is whole
        if (warp == 0) {
            __syncwarp();
            ptx::tc_fence_after();
            const uint64_t vd = ptx::sw128_mnmajor_desc(values_now, kKeyBytes);
#pragma unroll
            for (int e = 0; e < 8; ++e)      // (the weights' high parts, then their low ones)
                if (ptx::elect_one()) ptx::mma_bf16_ts(tmem + 64, tmem + 8 * e, vd + 128 * (e & 3), kSums, e > 0);
            if (ptx::elect_one()) ptx::mma_commit(&bars[1]);
        }
        __syncwarp();
        if (x == first) ptx::griddep_wait();              // (the joining kernel is let in by the end alone: its blocks, waiting
                                                             // beside the last tiles, cost 60 us of 472 for 16 x 16384 queries)
        out.stat[(tile0 + x) * kTileRows + tid] = make_float2(top, sum);
        ptx::mbar_wait(&bars[1], phase, status);
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_ld32_issue(mine + 64, lo);
        ptx::tmem_ld32_issue(mine + 96, hi);
        ptx::tmem_ld_wait32(lo);
        ptx::tmem_ld_wait32(hi);
        ptx::tc_fence_before();
        if (lane == 0) ptx::bulk_wait_read<0>();             // the last rows have left
        __syncwarp();
        stage_sums(sums + lane * kSumsPitch, lo, 0, lane);
        stage_sums(sums + lane * kSumsPitch, hi, 1, lane);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && count > 0) {
            bulk_store_once(out.sums + ((tile0 + x) * kTileRows + 32 * warp) * kHeadDim, sums, min(count, 32) * kSumsPitch);
            ptx::bulk_commit();
        }
    }
    if (lane == 0) ptx::bulk_wait<0>();
    __syncthreads();
    __syncwarp();
    if (warp == 0) ptx::tmem_dealloc(tmem, kTileColumns);
}

constexpr int kJoined = 4;                   // partials in flight (16 x 16384 queries: 422 us, with 2 or 8 446 and 452)

// Sixteen lanes join a row's partials.
__global__ void __launch_bounds__(256)
selected_join_kernel(const __grid_constant__ SelectedArgs a, const __grid_constant__ BlockLists l, const Partials in,
                     uint32_t rows) {
    const SelectShape& s = a.s;
    const int lane = threadIdx.x & 15;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint32_t row = (gridDim.x - 1 - blockIdx.x) * 16 + (threadIdx.x >> 4);       // (the last tiles' partials are in the L2)
    if (row >= rows) return;
    const RowOf at = row_of(s, in.u0, row);
    const int count = l.live[in.u0 * s.n + at.entry];
    const uint32_t* position = l.positions + (in.u0 * s.n + at.entry) * l.ranks;
    const float* sums = in.sums + at.unit * l.most_tiles * (kSumsBytes / 4);
    const float2* stat = in.stat + at.unit * l.most_tiles * kTileRows;
    // a few partials at a time, under a running maximum
    float top = -INFINITY, sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < count; x0 += kJoined) {
        uint32_t p[kJoined];
        float4 v[kJoined];
        float2 st[kJoined];
#pragma unroll
        for (int x = 0; x < kJoined; ++x) p[x] = x0 + x < count ? position[x0 + x] + at.head : ~0u;
#pragma unroll
        for (int x = 0; x < kJoined; ++x) {
            const bool on = x0 + x < count;
            v[x] = on ? sums_at(sums, p[x], lane) : make_float4(0.f, 0.f, 0.f, 0.f);
            st[x] = on ? stat[p[x]] : make_float2(-INFINITY, 0.f);
        }
        float now = top;
#pragma unroll
        for (int x = 0; x < kJoined; ++x) now = fmaxf(now, st[x].x);
        const float base = now == -INFINITY ? 0.f : now, shrink = exp2_fast(top - base);
        sum *= shrink;
        y = make_float4(y.x * shrink, y.y * shrink, y.z * shrink, y.w * shrink);
#pragma unroll
        for (int x = 0; x < kJoined; ++x) {
            const float w = exp2_fast(st[x].x - base);
            sum += w * st[x].y;
            y.x += w * v[x].x;
            y.y += w * v[x].y;
            y.z += w * v[x].z;
            y.w += w * v[x].w;
        }
        top = now;
    }
    const float r = sum == 0.f ? 0.f : 1.f / sum;            // (a NaN among the scores is one in the sum)
    reinterpret_cast<uint2*>(a.out + at.place * kHeadDim)[lane] = make_uint2(pack(y.x * r, y.y * r), pack(y.z * r, y.w * r));
    if (a.lse && lane == 0) a.lse[at.place] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

struct Plan {
    BlockLists lists;
    int64_t group;                           // units whose partials are held at once
    size_t sums, stat, total;
};
Plan plan_tiles(const SelectShape& s, char* ws) {
    Plan p;
    p.sums = plan_block_lists(s, ws, &p.lists);
    const int64_t units = s.B * s.Hk;
    const int64_t groups = (units * p.lists.most_tiles * kSumsBytes + (int64_t)kGroupBytes - 1) / (int64_t)kGroupBytes;
    p.group = groups < 1 ? units : groups < units ? (units + groups - 1) / groups : 1;
    p.stat = p.sums + p.group * p.lists.most_tiles * kSumsBytes;
    p.total = p.stat + p.group * p.lists.most_tiles * kTileRows * 8;
    p.lists.shares = tile_shares(s, p.lists, p.group, kTileResident, tile_rounds(s, p.lists, p.group, kTileResident));
    return p;
}

int launch_tiles(const SelectedArgs& a, char* ws, cudaStream_t stream) {
    const SelectShape& s = a.s;
    const Plan p = plan_tiles(s, ws);
    static std::atomic<uint64_t> ready{0};
    int* status = nullptr;
    int st = ready_status(&status);
    if (st) return st;
    cudaError_t err = allow_smem(selected_tiles_kernel, kTileSmem, ready);
    if (err != cudaSuccess) return cuda_fail(err, "selected_tiles_kernel");
    if (p.group * p.lists.shares > INT32_MAX || p.group * s.n * s.G > INT32_MAX)
        return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    if ((st = launch_block_lists(s, a.blocks, p.lists, false, stream))) return st;
    const int64_t units = s.B * s.Hk;
    for (int64_t u0 = 0; u0 < units && err == cudaSuccess; u0 += p.group) {
        const int64_t here = units - u0 < p.group ? units - u0 : p.group, rows = here * s.n * s.G;
        const Partials part{reinterpret_cast<float*>(ws + p.sums), reinterpret_cast<float2*>(ws + p.stat), u0, u0 == 0};
        {
            LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
            err = launch_pdl(selected_tiles_kernel, dim3((unsigned)(here * p.lists.shares)), dim3(kTileThreads), kTileSmem,
                             stream, a, p.lists, part, status);
        }
        if (err == cudaSuccess) {
            LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
            err = launch_pdl(selected_join_kernel, dim3((unsigned)((rows + 15) / 16)), dim3(256), 0, stream, a, p.lists, part,
                             (uint32_t)rows);
        }
    }
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "selected_tiles_kernel");
}

// By query, a warp reads 16 KB of a block's keys and values for a query and up to eight heads, 3 us a thousand.  By block,
// a tile takes as long whether it has a row or 128, 9 us a thousand; its rows' partials 1 us for 25000, and the lists
// and the launches 12 more than a launch.  So what decides is how many queries a listed block has, which is at most
// the queries of one sequence and key head: many sequences' single tokens never share one, however many they are.
// (By query and by block, 16 blocks a query, 4 heads, us: 512 and 2048 single tokens of caches of 16384 keys 32 and 132,
// 111 and 371; 512 with 8 tokens each 197 and 421, with 32 of 4096 keys 619 and 308.  One sequence's 256 queries of
// 4096 keys 12 and 22; 640, 8 heads, 28 and 29; 4 heads of 256 queries, one a group, 39 and 23.)
bool by_query(const SelectShape& s) {
    if (s.m == 0) return true;
    BlockLists l;
    plan_block_lists(s, nullptr, &l);
    const int64_t listed = s.B * s.Hk * s.n * l.ranks;       // (query, block) pairs
    return listed * ((s.G + 7) / 8) <= 4000 + 3 * s.B * s.Hk * l.most_tiles + listed * s.G / 75;
}

}  // namespace

size_t selected_workspace(const SelectShape& s) { return by_query(s) || s.B * s.n == 0 ? 0 : plan_tiles(s, nullptr).total; }

int launch_selected(const SelectedArgs& a, char* ws, cudaStream_t stream) {
    return by_query(a.s) ? launch_few(a, stream) : launch_tiles(a, ws, stream);
}

}  // namespace dfs
