// Attention over the key blocks that each query lists:
//   out_i = sum_j p_ij v_j,  p_ij = exp(q_i.k_j / 8 - lse_i),
// j over the visible keys of the listed blocks; a row without such keys is 0, its lse -infinity.
//
// Few queries: one block of threads for a query and up to eight heads of its group (the eight
// columns of the products).  Its warps take the listed blocks in turn, each with a running maximum
// and sum in registers, and join through shared memory.  A block's keys and values go from global
// memory into the products' registers.  Bound by the cache's bytes, or by a launch.
#include <atomic>

#include "block_lists.h"
#include "mma_tiles.cuh"
#include "selected.h"

namespace dfs {
namespace {

using namespace tiles;

constexpr float kScale2 = 0.125f * 1.4426950408889634f;      // 1 / sqrt(64) in units of log 2
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kFewWarps = 8;

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
        const float r = limit && top != -INFINITY ? 1.f / sum : 0.f;
        const int64_t at = first + h * s.n;
        *reinterpret_cast<uint32_t*>(a.out + at * kHeadDim + f) = pack(y0 * r, y1 * r);
        if (a.lse && f == 0) a.lse[at] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

int launch_few(const SelectedArgs& a, cudaStream_t stream) {
    const SelectShape& s = a.s;
    const int64_t grid = s.B * s.Hk * s.n * ((s.G + 7) / 8);
    if (grid > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    const int warps = s.top < kFewWarps ? s.top : kFewWarps;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        selected_few_kernel<<<(unsigned)grid, 32 * warps, 0, stream>>>(a);
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "selected_few_kernel");
}

constexpr int kItemRows = 256;
constexpr int kItemWarps = 4;
constexpr size_t kGroupBytes = 64 << 20;     // partials of a group of units

// Partials of the units u0 .. : slot x = ((u - u0) n + i) G + h) ranks + rank.
struct Partials {
    float* sums;                             // [slots][64], features by place_of
    float2* stat;                            // [slots]: maximum (units of log 2), sum
    int64_t u0;
};

// 32 bytes, a whole sector, in one store.
__device__ __forceinline__ void store32(float* p, float a, float b, float c, float d, float e, float f, float g, float h) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(a), "f"(b), "f"(c), "f"(d), "f"(e),
                 "f"(f), "f"(g), "f"(h)
                 : "memory");
}

__global__ void __launch_bounds__(32 * kItemWarps, 2)
selected_items_kernel(const __grid_constant__ SelectedArgs a, const __grid_constant__ BlockLists l, const Partials out) {
    const SelectShape& s = a.s;
    const uint32_t ul = blockIdx.x / (uint32_t)l.most_items;
    const int64_t u = out.u0 + ul, b = sequence_of(s, u);
    const ItemRows item = item_of(l, s, u, blockIdx.x - ul * l.most_items);
    if (!item.rows) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int32_t key0 = item.block * kBlockKeys;
    const int rows = min(kBlockKeys, key_count(s, b) - key0);
    uint32_t keys[8][8], values[8][8];
    load_keys(a.k + (u * s.m + key0) * kHeadDim, rows, lane, keys);
    load_keys(a.v + (u * s.m + key0) * kHeadDim, rows, lane, values);
    turn_values(values);
    const __nv_bfloat16* q0 = a.q + u * s.G * s.n * kHeadDim;
    const int64_t slot0 = (int64_t)ul * s.n * s.G * l.ranks;

    // rows r0 + g and r0 + 8 + g of this lane: their entries two steps ahead, their queries one
    struct Rows {
        uint32_t entry[2], head[2];
    };
    auto look = [&](int r0) {
        Rows x;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = r0 + 8 * j + g;
            const uint32_t r = item.first + (row < item.rows ? row : 0), e = s.G == 1 ? r : r / s.G;
            x.head[j] = r - e * s.G;
            x.entry[j] = item.entries[e];
        }
        return x;
    };
    auto fetch = [&](const Rows& x, int r0, uint32_t (&q)[2][8]) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            load_row(q0 + ((int64_t)x.head[j] * s.n + (x.entry[j] >> 6)) * kHeadDim, r0 + 8 * j + g < item.rows, t, q[j]);
    };
    constexpr int kStep = 16 * kItemWarps;
    Rows now = look(16 * warp), next = look(16 * warp + kStep);
    uint32_t q[2][8];
    fetch(now, 16 * warp, q);
    for (int r0 = 16 * warp; r0 < item.rows; r0 += kStep) {
        float x[2][4][4];
        uint32_t mine[2];
        int sees[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t i = now.entry[j] >> 6;
            const bool live = r0 + 8 * j + g < item.rows;
            mine[j] = live ? (i * s.G + now.head[j]) * l.ranks + (now.entry[j] & 63) : ~0u;
            sees[j] = live ? row_limit(s, b, i) - key0 : 0;
            score(keys, q[j], x[j]);
        }
        now = next;
        fetch(now, r0 + kStep, q);
        next = look(r0 + 2 * kStep);
        const bool whole = __all_sync(kFull, min(sees[0], sees[1]) >= kBlockKeys);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!whole) {
                const int limit[2] = {__shfl_sync(kFull, sees[j], 8 * t), __shfl_sync(kFull, sees[j], 8 * t + 4)};
#pragma unroll
                for (int M = 0; M < 4; ++M)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (16 * M + 8 * (c >> 1) + g >= limit[c & 1]) x[j][M][c] = -INFINITY;
            }
            float m[2], sum[2] = {0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m[c] = fmaxf(x[j][0][c], x[j][0][c + 2]);
#pragma unroll
                for (int M = 1; M < 4; ++M) m[c] = fmaxf(m[c], fmaxf(x[j][M][c], x[j][M][c + 2]));
                m[c] = column_max(m[c]) * kScale2;
                const float base = m[c] == -INFINITY ? 0.f : m[c];
#pragma unroll
                for (int M = 0; M < 4; ++M)
#pragma unroll
                    for (int k = c; k < 4; k += 2) {
                        x[j][M][k] = exp2_fast(fmaf(x[j][M][k], kScale2, -base));
                        sum[c] += x[j][M][k];
                    }
            }
            float o[4][4];
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k >> 2][k & 3] = 0.f;
            weigh(values, x[j], o);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                sum[c] = column_sum(sum[c]);
                const uint32_t slot = __shfl_sync(kFull, mine[j], 8 * t + 4 * c);
                if (slot == ~0u) continue;
                store32(out.sums + (slot0 + slot) * kHeadDim + 8 * g, o[0][c], o[0][c + 2], o[1][c], o[1][c + 2], o[2][c],
                        o[2][c + 2], o[3][c], o[3][c + 2]);
                if (g == 0) out.stat[slot0 + slot] = make_float2(m[c], sum[c]);
            }
        }
    }
}

constexpr int kJoined = 8;                   // partials in flight

// Sixteen lanes join a row's partials.
__global__ void __launch_bounds__(256)
selected_join_kernel(const __grid_constant__ SelectedArgs a, const __grid_constant__ BlockLists l, const Partials in,
                     uint32_t rows) {
    const SelectShape& s = a.s;
    const int lane = threadIdx.x & 15;
    const unsigned half = 0xffffu << (threadIdx.x & 16);
    const uint32_t row = blockIdx.x * 16 + (threadIdx.x >> 4);
    if (row >= rows) return;
    const RowOf at = row_of(s, in.u0, row);
    const int count = l.live[in.u0 * s.n + at.entry];
    const float2* stat = in.stat + (int64_t)row * l.ranks;
    const float4* part = reinterpret_cast<const float4*>(in.sums + (int64_t)row * l.ranks * kHeadDim) + lane;
    // eight partials at a time, under a running maximum
    float top = -INFINITY, sum = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < count; x0 += kJoined) {
        float4 p[kJoined];
        float2 st[kJoined];
#pragma unroll
        for (int x = 0; x < kJoined; ++x) {
            const bool on = x0 + x < count;
            p[x] = on ? part[(x0 + x) * 16] : make_float4(0.f, 0.f, 0.f, 0.f);
            st[x] = on ? stat[x0 + x] : make_float2(-INFINITY, 0.f);
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
            y.x += w * p[x].x;
            y.y += w * p[x].y;
            y.z += w * p[x].z;
            y.w += w * p[x].w;
        }
        top = now;
    }
    const float r = top != -INFINITY ? 1.f / sum : 0.f;
    // this lane has features 2k + e of an eight, k = 0 .. 3, its neighbour two lanes on the other e
    const int g = lane >> 1, e = g & 1;
    const float z[4] = {y.x * r, y.y * r, y.z * r, y.w * r};
    const float got0 = __shfl_xor_sync(half, e ? z[0] : z[2], 2), got1 = __shfl_xor_sync(half, e ? z[1] : z[3], 2);
    const uint2 w = e ? make_uint2(pack(got0, z[2]), pack(got1, z[3])) : make_uint2(pack(z[0], got0), pack(z[1], got1));
    *reinterpret_cast<uint2*>(a.out + at.place * kHeadDim + 32 * (lane & 1) + 8 * (g >> 1) + 4 * e) = w;
    if (a.lse && lane == 0) a.lse[at.place] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * kLn2;
}

struct Plan {
    BlockLists lists;
    int64_t group;                           // units whose partials are held at once
    size_t sums, stat, total;
};
Plan plan_items(const SelectShape& s, char* ws) {
    Plan p;
    p.sums = plan_block_lists(s, kItemRows, ws, &p.lists);
    const int64_t units = s.B * s.Hk, slots = s.n * s.G * p.lists.ranks;
    p.group = slots ? (int64_t)(kGroupBytes / (slots * 264)) : 1;
    p.group = p.group < 1 ? 1 : p.group > units ? units : p.group;
    p.stat = p.sums + p.group * slots * kHeadDim * 4;
    p.total = p.stat + (p.group * slots * 8 + 255) / 256 * 256;
    return p;
}

int launch_items(const SelectedArgs& a, char* ws, cudaStream_t stream) {
    const SelectShape& s = a.s;
    const Plan p = plan_items(s, ws);
    int st = launch_block_lists(s, a.blocks, p.lists, stream);
    if (st) return st;
    const int64_t units = s.B * s.Hk;
    for (int64_t u0 = 0; u0 < units; u0 += p.group) {
        const int64_t here = units - u0 < p.group ? units - u0 : p.group, rows = here * s.n * s.G;
        const Partials part{reinterpret_cast<float*>(ws + p.sums), reinterpret_cast<float2*>(ws + p.stat), u0};
        if (here * p.lists.most_items > INT32_MAX || rows > INT32_MAX)
            return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
        {
            LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
            selected_items_kernel<<<(unsigned)(here * p.lists.most_items), 32 * kItemWarps, 0, stream>>>(a, p.lists, part);
        }
        {
            LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
            selected_join_kernel<<<(unsigned)((rows + 15) / 16), 256, 0, stream>>>(a, p.lists, part, (uint32_t)rows);
        }
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "selected_items_kernel");
}

// Few queries: what the lists, the partials and their joining would cost outweighs reading a block's
// keys once for each query that lists it.
bool by_query(const SelectShape& s) { return s.m == 0 || s.B * s.Hk * s.n * s.top <= 8192; }

}  // namespace

size_t selected_workspace(const SelectShape& s) { return by_query(s) || s.B * s.n == 0 ? 0 : plan_items(s, nullptr).total; }

int launch_selected(const SelectedArgs& a, char* ws, cudaStream_t stream) {
    return by_query(a.s) ? launch_few(a, stream) : launch_items(a, ws, stream);
}

}  // namespace dfs
