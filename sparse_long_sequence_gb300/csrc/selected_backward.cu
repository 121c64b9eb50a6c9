// Gradients of the attention over chosen key blocks, block by block as the forward:
//   P_ij = exp(q_i.k_j / 8 - lse_i),  dS_ij = P_ij (dout_i.v_j - delta_i) / 8,  delta_i = dout_i.out_i,
//   dv_j = sum_i P_ij dout_i,  dk_j = sum_i dS_ij q_i,  dq_i = sum_j dS_ij k_j.
//
// A block of four warps takes up to 512 rows that list a key block (block_lists.cu), 32 at a time, their
// queries and dout gathered into shared memory two steps ahead of use.  Each warp holds 16 of the 64 keys
// (as the left operand of the scores and of dout.v) and their 16 x 64 sums of dk and dv in registers over
// all the rows, so that P and dS go from one product's result straight into the next one's left operand;
// dS also goes through shared memory, after which each warp has 16 features of the rows' dq.  A (row,
// block) leaves 64 fp32 sums of dq, an item its sums of dk and dv, and two kernels join them in a fixed
// order.  The units go in groups whose partials stay in the L2.
#include <atomic>

#include "block_lists.h"
#include "layer_ops.h"
#include "mma_tiles.cuh"
#include "selected.h"
#include "sm100_ptx.cuh"

namespace dfs {
namespace {

using namespace tiles;

constexpr float kScale = 0.125f;             // 1 / sqrt(64)
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kItemRows = 512;
constexpr int kThreads = 128;
constexpr int kTile = 32;                    // rows of a step
constexpr int kRowBytes = kHeadDim * 2;
constexpr int kTurnStride = 80;              // bytes of a key's 32 dS values, apart by banks
constexpr size_t kGroupBytes = 96 << 20;     // partials of a group of units

struct Partials {
    float* dq;                               // [slots][64], slot ((u - u0) n + i) G + h) ranks + rank
    float* dkv;                              // [items][2][64][64]
    const float2* stat;                      // [B][Hq][n]: lse in units of log 2, delta
    int64_t u0;
};

__device__ __forceinline__ void ldmatrix(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void ldmatrix_turned(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
// 16 bytes into shared memory; zeros where `live` is false (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

// Byte of 16-byte chunk `chunk` of a row of 128 bytes; the chunks of eight rows fall in eight bank groups.
__device__ __forceinline__ uint32_t place(int row, int chunk) { return row * kRowBytes + ((chunk ^ (row & 7)) << 4); }

// stat = (lse in units of log 2, delta): eight lanes a row.
__global__ void __launch_bounds__(256) selected_delta_kernel(const __grid_constant__ SelectedArgs a, int64_t rows, float2* stat) {
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
    if (row < rows && lane == 0) stat[row] = make_float2(a.lse[row] * kLog2e, d);
}

__global__ void __launch_bounds__(kThreads, 3)
selected_grads_kernel(const __grid_constant__ SelectedArgs a, const __grid_constant__ BlockLists l, const Partials out) {
    __shared__ __align__(128) char rows_smem[2][2][kTile * kRowBytes];       // [stage][queries, dout]; first the keys, values
    __shared__ __align__(128) char turn_smem[kBlockKeys * kTurnStride];      // dS [key][row]
    __shared__ float2 stat_smem[2][kTile];
    __shared__ int2 meta_smem[2][kTile];                                     // visible keys of the block, slot
    const SelectShape& s = a.s;
    const uint32_t ul = blockIdx.x / (uint32_t)l.most_items;
    const int64_t u = out.u0 + ul, b = sequence_of(s, u);
    const ItemRows item = item_of(l, s, u, blockIdx.x - ul * l.most_items);
    if (!item.rows) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int32_t key0 = item.block * kBlockKeys;
    const int keys = min(kBlockKeys, key_count(s, b) - key0);
    const int64_t head0 = u * s.G;
    const uint32_t smem = ptx::smem_u32(rows_smem), turned = ptx::smem_u32(turn_smem);

    // the keys' and values' operands, by way of the rows' buffers
    {
        const __nv_bfloat16 *k = a.k + (u * s.m + key0) * kHeadDim, *v = a.v + (u * s.m + key0) * kHeadDim;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int x = tid + kThreads * j, r = x >> 3, c = x & 7;
            const int64_t from = (int64_t)(r < keys ? r : 0) * kHeadDim + 8 * c;
            copy16(smem + place(r, c), k + from, r < keys);
            copy16(smem + 2 * kTile * kRowBytes + place(r, c), v + from, r < keys);
        }
        copies_commit();
        copies_wait<0>();
        __syncthreads();
    }
    uint32_t ka[4][4], va[4][4];             // keys 16 warp ..: left operands, by 16 features
    uint32_t kb[4][4];                       // 16 features from 16 warp: right operand, by 16 keys
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int r = 16 * warp + (lane & 15), c = 2 * e + (lane >> 4);
        ldmatrix(smem + place(r, c), ka[e]);
        ldmatrix(smem + 2 * kTile * kRowBytes + place(r, c), va[e]);
        ldmatrix_turned(smem + place(16 * e + (lane & 15), 2 * warp + (lane >> 4)), kb[e]);
    }
    __syncthreads();

    // rows of step x: this thread's two entries, and their copies
    const int steps = (item.rows + kTile - 1) / kTile;
    auto entry_of = [&](int row, uint32_t* h) -> uint32_t {                  // of a row of the item
        const uint32_t r = item.first + (row < item.rows ? row : 0), e = s.G == 1 ? r : r / s.G;
        *h = r - e * s.G;
        return item.entries[e];
    };
    uint32_t entry[2], head[2];
    auto look = [&](int x) {
#pragma unroll
        for (int j = 0; j < 2; ++j) entry[j] = entry_of(x * kTile + 16 * j + (tid >> 3), &head[j]);
    };
    auto fetch = [&](int x) {                // copies step x, whose entries have been looked up
        const int stage = x & 1;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 16 * j + (tid >> 3), c = tid & 7;
            const bool live = x * kTile + r < item.rows;
            const uint32_t i = entry[j] >> 6;
            const int64_t row = (head0 + head[j]) * s.n + i;
            const uint32_t to = smem + stage * 2 * kTile * kRowBytes + place(r, c);
            copy16(to, a.q + row * kHeadDim + 8 * c, live);
            copy16(to + kTile * kRowBytes, a.dout + row * kHeadDim + 8 * c, live);
            if (c == 0) {
                copy8(ptx::smem_u32(&stat_smem[stage][r]), out.stat + row);
                meta_smem[stage][r] = live ? make_int2(row_limit(s, b, i) - key0, (i * s.G + head[j]) * l.ranks + (entry[j] & 63))
                                           : make_int2(0, -1);
            }
        }
        copies_commit();
    };
    look(0);
    fetch(0);
    if (steps > 1) look(1);

    float dk[8][4], dv[8][4];
#pragma unroll
    for (int j = 0; j < 32; ++j) dk[j >> 2][j & 3] = dv[j >> 2][j & 3] = 0.f;
    const int64_t slot0 = (int64_t)ul * s.n * s.G * l.ranks;

    for (int x = 0; x < steps; ++x) {
        copies_wait<0>();
        __syncthreads();                     // step x has arrived; all are done with step x - 1
        if (x + 1 < steps) {
            fetch(x + 1);
            if (x + 2 < steps) look(x + 2);
        }
        const int stage = x & 1;
        const uint32_t qs = smem + stage * 2 * kTile * kRowBytes, ds = qs + kTile * kRowBytes;
#pragma unroll
        for (int half = 0; half < 2; ++half) {               // 16 rows
            uint32_t pa[4], sa[4];                           // P and dS as left operands
#pragma unroll
            for (int eight = 0; eight < 2; ++eight) {
                const int r0 = 16 * half + 8 * eight;
                float sc[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int f = 0; f < 2; ++f) {                // 32 features
                    uint32_t qb[4], db[4];
                    const uint32_t at = place(r0 + (lane & 7), 4 * f + (lane >> 3));
                    ldmatrix(qs + at, qb);
                    ldmatrix(ds + at, db);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t(&k4)[4] = ka[2 * f + e];
                        const uint32_t(&v4)[4] = va[2 * f + e];
                        mma(sc, k4[0], k4[1], k4[2], k4[3], qb[2 * e], qb[2 * e + 1]);
                        mma(dp, v4[0], v4[1], v4[2], v4[3], db[2 * e], db[2 * e + 1]);
                    }
                }
                // results: keys g, g + 8 of the warp's; rows r0 + 2t, + 1
                float p[4], d[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = r0 + 2 * t + (j & 1), key = 16 * warp + g + 8 * (j >> 1);
                    const float2 st = stat_smem[stage][r];
                    const bool on = key < meta_smem[stage][r].x;
                    p[j] = on ? exp2_fast(sc[j] * (kScale * kLog2e) - st.x) : 0.f;
                    d[j] = on ? p[j] * (dp[j] - st.y) * kScale : 0.f;
                }
                pa[2 * eight] = pack(p[0], p[1]);
                pa[2 * eight + 1] = pack(p[2], p[3]);
                sa[2 * eight] = pack(d[0], d[1]);
                sa[2 * eight + 1] = pack(d[2], d[3]);
                char* to = turn_smem + (16 * warp + g) * kTurnStride + (r0 + 2 * t) * 2;
                *reinterpret_cast<uint32_t*>(to) = sa[2 * eight];
                *reinterpret_cast<uint32_t*>(to + 8 * kTurnStride) = sa[2 * eight + 1];
            }
#pragma unroll
            for (int f = 0; f < 4; ++f) {                    // 16 features
                uint32_t qb[4], db[4];
                const uint32_t at = place(16 * half + (lane & 15), 2 * f + (lane >> 4));
                ldmatrix_turned(qs + at, qb);
                ldmatrix_turned(ds + at, db);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mma(dk[2 * f + e], sa[0], sa[1], sa[2], sa[3], qb[2 * e], qb[2 * e + 1]);
                    mma(dv[2 * f + e], pa[0], pa[1], pa[2], pa[3], db[2 * e], db[2 * e + 1]);
                }
            }
        }
        __syncthreads();                     // dS is whole
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float dq[2][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) dq[j >> 2][j & 3] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {                    // 16 keys
                uint32_t da[4];
                // matrices: keys 0-7 by rows 0-7, keys 0-7 by rows 8-15, keys 8-15 by rows 0-7, by rows 8-15
                ldmatrix_turned(turned + (16 * e + (lane & 7) + 8 * (lane >> 4)) * kTurnStride + 32 * half + 16 * (lane >> 3 & 1), da);
                mma(dq[0], da[0], da[1], da[2], da[3], kb[e][0], kb[e][1]);
                mma(dq[1], da[0], da[1], da[2], da[3], kb[e][2], kb[e][3]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int slot = meta_smem[stage][16 * half + g + 8 * j].y;
                if (slot < 0) continue;
                float* dst = out.dq + (slot0 + slot) * kHeadDim + 16 * warp + 2 * t;
                *reinterpret_cast<float2*>(dst) = make_float2(dq[0][2 * j], dq[0][2 * j + 1]);
                *reinterpret_cast<float2*>(dst + 8) = make_float2(dq[1][2 * j], dq[1][2 * j + 1]);
            }
        }
    }
    float* dst = out.dkv + (int64_t)blockIdx.x * (2 * kBlockKeys * kHeadDim) +
                 (16 * warp + g) * kHeadDim + 2 * t;
#pragma unroll
    for (int f = 0; f < 8; ++f)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float* at = dst + 8 * j * kHeadDim + 8 * f;
            *reinterpret_cast<float2*>(at) = make_float2(dk[f][2 * j], dk[f][2 * j + 1]);
            *reinterpret_cast<float2*>(at + kBlockKeys * kHeadDim) = make_float2(dv[f][2 * j], dv[f][2 * j + 1]);
        }
}

// dq of a row: the sum of its partials, sixteen lanes a row.
__global__ void __launch_bounds__(256)
selected_dq_kernel(const __grid_constant__ SelectedArgs a, const __grid_constant__ BlockLists l, const Partials in, uint32_t rows) {
    const SelectShape& s = a.s;
    const int lane = threadIdx.x & 15;
    const uint32_t row = blockIdx.x * 16 + (threadIdx.x >> 4);
    if (row >= rows) return;
    const RowOf at = row_of(s, in.u0, row);
    const int count = l.live[in.u0 * s.n + at.entry];
    const float4* part = reinterpret_cast<const float4*>(in.dq + (int64_t)row * l.ranks * kHeadDim) + lane;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = 0; x < count; ++x) {
        const float4 p = part[x * 16];
        y = make_float4(y.x + p.x, y.y + p.y, y.z + p.z, y.w + p.w);
    }
    reinterpret_cast<uint2*>(a.dq + at.place * kHeadDim)[lane] = make_uint2(pack(y.x, y.y), pack(y.z, y.w));
}

// dk and dv of a key block: the sums of its items', by sixteen rows of keys; eight items in flight.
constexpr int kSplit = 4;
__global__ void __launch_bounds__(256)
selected_dkv_kernel(const __grid_constant__ SelectedArgs a, const __grid_constant__ BlockLists l, const Partials in) {
    const SelectShape& s = a.s;
    const int split = blockIdx.x % (2 * kSplit), part = split % kSplit, which = split / kSplit;
    const uint32_t at = blockIdx.x / (2 * kSplit), ul = at / (uint32_t)s.nb;
    const int64_t u = in.u0 + ul;
    const int c = at - ul * s.nb;
    const int32_t* base = l.item_base + u * (s.nb + 1) + c;
    const int from = base[0], to = base[1];
    const int64_t key = (int64_t)c * kBlockKeys + 16 * part + (threadIdx.x >> 4);
    if (key >= s.m) return;
    const float4* src = reinterpret_cast<const float4*>(in.dkv) +
                        (((int64_t)ul * l.most_items + from) * 2 + which) * 1024 + 256 * part + threadIdx.x;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int x = 0; x < to - from; ++x) {
        const float4 p = src[(int64_t)x * 2048];
        y = make_float4(y.x + p.x, y.y + p.y, y.z + p.z, y.w + p.w);
    }
    __nv_bfloat16* dst = (which ? a.dv : a.dk) + (u * s.m + key) * kHeadDim;
    reinterpret_cast<uint2*>(dst)[threadIdx.x & 15] = make_uint2(pack(y.x, y.y), pack(y.z, y.w));
}

struct Plan {
    BlockLists lists;
    int64_t group;                           // units whose partials are held at once
    size_t stat, dq, dkv, total;
};
Plan plan_backward(const SelectShape& s, char* ws) {
    Plan p;
    p.stat = plan_block_lists(s, kItemRows, ws, &p.lists);
    p.dq = p.stat + (s.B * s.Hq * s.n * 8 + 255) / 256 * 256;
    const int64_t units = s.B * s.Hk;
    const size_t dq = (size_t)s.n * s.G * p.lists.ranks * kHeadDim * 4;
    const size_t dkv = (size_t)p.lists.most_items * 2 * kBlockKeys * kHeadDim * 4;
    p.group = (int64_t)(kGroupBytes / (dq + dkv));
    p.group = p.group < 1 ? 1 : p.group > units ? units : p.group;
    p.dkv = p.dq + p.group * dq;
    p.total = p.dkv + p.group * dkv;
    return p;
}

}  // namespace

size_t selected_backward_workspace(const SelectShape& s) {
    return s.B * s.n * s.m == 0 ? 0 : plan_backward(s, nullptr).total;
}

int launch_selected_backward(const SelectedArgs& a, char* ws, cudaStream_t stream) {
    const SelectShape& s = a.s;
    const Plan p = plan_backward(s, ws);
    int st = launch_block_lists(s, a.blocks, p.lists, stream);
    if (st) return st;
    const int64_t units = s.B * s.Hk, all = s.B * s.Hq * s.n;
    if ((all + 31) / 32 > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        selected_delta_kernel<<<(unsigned)((all + 31) / 32), 256, 0, stream>>>(a, all, reinterpret_cast<float2*>(ws + p.stat));
    }
    for (int64_t u0 = 0; u0 < units; u0 += p.group) {
        const int64_t here = units - u0 < p.group ? units - u0 : p.group, rows = here * s.n * s.G;
        const Partials part{reinterpret_cast<float*>(ws + p.dq), reinterpret_cast<float*>(ws + p.dkv),
                            reinterpret_cast<const float2*>(ws + p.stat), u0};
        if (here * p.lists.most_items > INT32_MAX || rows > INT32_MAX || here * s.nb * 2 * kSplit > INT32_MAX)
            return fail(DIFFUSER_ERR_OVERFLOW, "too many queries");
        {
            LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
            selected_grads_kernel<<<(unsigned)(here * p.lists.most_items), kThreads, 0, stream>>>(a, p.lists, part);
        }
        {
            LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
            selected_dq_kernel<<<(unsigned)((rows + 15) / 16), 256, 0, stream>>>(a, p.lists, part, (uint32_t)rows);
        }
        {
            LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
            selected_dkv_kernel<<<(unsigned)(here * s.nb * 2 * kSplit), 256, 0, stream>>>(a, p.lists, part);
        }
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "selected_grads_kernel");
}

}  // namespace dfs
