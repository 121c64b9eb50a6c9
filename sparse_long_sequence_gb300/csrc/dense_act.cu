// The elementwise half of the dense products' backward passes.
//
//   dense   dP[t][f] = dY[t][f] act'(P[t][f]),  db[f] = sum_t dP[t][f]
//   gated   dP[t][f] = dH[t][f] act'(g) u,  dP[t][F + f] = dH[t][f] act(g),
//           g = P[t][f], u = P[t][F + f]
// dP is the operand of the two tensor-core products that follow, so it is rounded to
// bf16 here; the bias gradient is summed in fp32 from the unrounded values, over a
// block's rows and then over the blocks in a fixed order.
// Bound by memory: every array is read or written once, 16 bytes a lane.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "activations.cuh"
#include "layer_ops.h"

namespace dfs {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 8;                          // columns of a lane (16 bytes)
constexpr int kAhead = 4;                        // rows of a warp whose loads are in flight together
constexpr int kBlockCols = 32 * kPer;            // columns of a block; its warps take rows in turn

__device__ __forceinline__ void widen8(const uint4& r, float (&v)[kPer]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 round8(const float (&v)[kPer]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }

// block (x, y): columns 256 x .. +255, rows [y chunk, (y + 1) chunk).  The column sums go to
// `partial`, or, rounded, to `colsum` where one block has all the rows; both null: none asked for.
template <int kAct>
__global__ void __launch_bounds__(kThreads)
act_backward_kernel(const __nv_bfloat16* dY, const __nv_bfloat16* P, int64_t rows, int32_t F, int64_t chunk,
                    __nv_bfloat16* dP, float* partial, __nv_bfloat16* colsum) {
    __shared__ float sums[kWarps][kBlockCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = (int)blockIdx.x * kBlockCols + lane * kPer;
    const int64_t r1 = min(rows, ((int64_t)blockIdx.y + 1) * chunk);
    float sum[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum[j] = 0.f;
    if (c < F) {
        for (int64_t r0 = (int64_t)blockIdx.y * chunk + warp; r0 < r1; r0 += kWarps * kAhead) {
            uint4 dy[kAhead], pr[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int64_t r = r0 + k * kWarps;
                if (r < r1) {
                    dy[k] = load8(dY + r * F + c);
                    if constexpr (kAct != DIFFUSER_ACT_NONE) pr[k] = load8(P + r * F + c);
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int64_t r = r0 + k * kWarps;
                if (r >= r1) break;
                float d[kPer];
                widen8(dy[k], d);
                if constexpr (kAct != DIFFUSER_ACT_NONE) {
                    float p[kPer];
                    widen8(pr[k], p);
#pragma unroll
                    for (int j = 0; j < kPer; ++j) d[j] *= act::value_slope<kAct>(p[j]).y;
                    *reinterpret_cast<uint4*>(dP + r * F + c) = round8(d);
                }
#pragma unroll
                for (int j = 0; j < kPer; ++j) sum[j] += d[j];
            }
        }
    }
    if (!partial && !colsum) return;
#pragma unroll
    for (int j = 0; j < kPer; ++j) sums[warp][lane * kPer + j] = sum[j];
    __syncthreads();
    const int col = (int)blockIdx.x * kBlockCols + (int)threadIdx.x;
    if (col >= F) return;
    float t = 0.f;
    for (int w = 0; w < kWarps; ++w) t += sums[w][threadIdx.x];
    if (colsum) colsum[col] = __float2bfloat16_rn(t);
    else partial[(int64_t)blockIdx.y * F + col] = t;
}

// column sums over the chunks: 32 columns a block, its 32 warps take every 32nd chunk
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32) colsum_kernel(const float* partial, int64_t chunks, int32_t F, __nv_bfloat16* out) {
    __shared__ float sums[kSumWarps][32];
    ptx::griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = (int)blockIdx.x * 32 + lane;
    float t = 0.f;
    if (col < F) {
#pragma unroll 8
        for (int64_t k = warp; k < chunks; k += kSumWarps) t += partial[k * F + col];
    }
    sums[warp][lane] = t;
    __syncthreads();
    if (warp || col >= F) return;
    t = 0.f;
    for (int w = 0; w < kSumWarps; ++w) t += sums[w][lane];
    out[col] = __float2bfloat16_rn(t);
}

template <int kAct>
__global__ void __launch_bounds__(kThreads)
gated_backward_kernel(const __nv_bfloat16* dH, const __nv_bfloat16* P, int64_t items, int32_t F8, __nv_bfloat16* dP) {
    const int64_t F = (int64_t)F8 * kPer, step = (int64_t)gridDim.x * kThreads;
    for (int64_t e0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; e0 < items; e0 += 2 * step) {
        uint4 dh[2], pg[2], pu[2];
        int64_t at[2];                                // of the gate's element; dH's is r F + c
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t e = e0 + k * step;
            if (e >= items) break;
            const int64_t r = e / F8, c = (e - r * F8) * kPer;
            at[k] = r * 2 * F + c;
            dh[k] = load8(dH + r * F + c);
            pg[k] = load8(P + at[k]);
            pu[k] = load8(P + at[k] + F);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (e0 + k * step >= items) break;
            float d[kPer], g[kPer], u[kPer];
            widen8(dh[k], d);
            widen8(pg[k], g);
            widen8(pu[k], u);
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const float2 vs = act::value_slope<kAct>(g[j]);
                const float h = d[j];
                d[j] = h * u[j] * vs.y;
                u[j] = h * vs.x;
            }
            *reinterpret_cast<uint4*>(dP + at[k]) = round8(d);
            *reinterpret_cast<uint4*>(dP + at[k] + F) = round8(u);
        }
    }
}

// one instantiation per activation
template <template <int> class Launch, class... Args>
void by_activation(int32_t act, Args... args) {
    switch (act) {
        case DIFFUSER_ACT_RELU: Launch<DIFFUSER_ACT_RELU>::go(args...); break;
        case DIFFUSER_ACT_GELU: Launch<DIFFUSER_ACT_GELU>::go(args...); break;
        case DIFFUSER_ACT_GELU_TANH: Launch<DIFFUSER_ACT_GELU_TANH>::go(args...); break;
        case DIFFUSER_ACT_SILU: Launch<DIFFUSER_ACT_SILU>::go(args...); break;
        default: Launch<DIFFUSER_ACT_NONE>::go(args...); break;
    }
}
template <int kAct>
struct DenseBackward {
    static void go(dim3 grid, cudaStream_t s, const __nv_bfloat16* dY, const __nv_bfloat16* P, int64_t rows, int32_t F,
                   int64_t chunk, __nv_bfloat16* dP, float* partial, __nv_bfloat16* colsum) {
        act_backward_kernel<kAct><<<grid, kThreads, 0, s>>>(dY, P, rows, F, chunk, dP, partial, colsum);
    }
};
template <int kAct>
struct GatedBackward {
    static void go(dim3 grid, cudaStream_t s, const __nv_bfloat16* dH, const __nv_bfloat16* P, int64_t items, int32_t F8,
                   __nv_bfloat16* dP) {
        gated_backward_kernel<kAct><<<grid, kThreads, 0, s>>>(dH, P, items, F8, dP);
    }
};

// The most blocks of a pass: 152 SMs hold three at once (five without an activation, 48
// registers; 69 to 80 with one), so 2.7 rounds of them, taken for HBM rate rather than whole rounds
// (gated silu 16384 x 2816: 70 us, 97 % of the measured copy).
constexpr int64_t kManyBlocks = 152 * 8;

// Up to 64 rows one block has them all and finishes the column sums itself: a launch less
// (2.5 us on the host), while its 8 rows a warp take no longer than a launch (at 128 rows: 3 us more).
constexpr int64_t kOneChunk = 64;

int64_t chunk_rows(int64_t rows, int32_t F) {
    if (rows <= kOneChunk) return kOneChunk;
    const int64_t col_blocks = (F + kBlockCols - 1) / kBlockCols;
    const int64_t want = (kManyBlocks + col_blocks - 1) / col_blocks;
    const int64_t per = (rows + want - 1) / want;
    // at least two rows a warp, and at most 65535 chunks (the grid's y extent)
    const int64_t least = rows / 65535 + 1;
    const int64_t c = per < 2 * kWarps ? 2 * kWarps : per;
    return c < least ? least : c;
}

}  // namespace

int64_t act_chunks(int64_t rows, int32_t F) {
    if (rows <= 0) return 0;
    const int64_t c = chunk_rows(rows, F);
    return (rows + c - 1) / c;
}

int launch_colsum(const BiasSums& b, cudaStream_t stream) {
    cudaError_t err;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        err = launch_pdl(colsum_kernel, dim3((unsigned)((b.F + 31) / 32)), dim3(kSumWarps * 32), 0, stream, b.partial,
                         b.chunks, b.F, b.out);
    }
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "colsum_kernel");
}

int launch_act_backward(const void* dY, const void* P, int64_t rows, int32_t F, int32_t act, void* dP, void* colsum,
                        float* partial, BiasSums* sums, cudaStream_t stream) {
    const int64_t chunk = chunk_rows(rows, F), chunks = act_chunks(rows, F);
    const dim3 grid((unsigned)((F + kBlockCols - 1) / kBlockCols), (unsigned)chunks);
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        by_activation<DenseBackward>(act, grid, stream, static_cast<const __nv_bfloat16*>(dY),
                                     static_cast<const __nv_bfloat16*>(P), rows, F, chunk,
                                     static_cast<__nv_bfloat16*>(dP), colsum && chunks > 1 ? partial : nullptr,
                                     static_cast<__nv_bfloat16*>(chunks > 1 ? nullptr : colsum));
    }
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return cuda_fail(err, "act_backward_kernel");
    *sums = BiasSums{};
    if (colsum && chunks > 1) *sums = {partial, chunks, F, static_cast<__nv_bfloat16*>(colsum)};
    return DIFFUSER_OK;
}

int launch_gated_backward(const void* dH, const void* P, int64_t rows, int32_t F, int32_t act, void* dP,
                          cudaStream_t stream) {
    const int64_t items = rows * (F / kPer);
    int64_t blocks = (items + kThreads - 1) / kThreads;
    if (blocks > kManyBlocks) blocks = kManyBlocks;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        by_activation<GatedBackward>(act, dim3((unsigned)blocks), stream, static_cast<const __nv_bfloat16*>(dH),
                                     static_cast<const __nv_bfloat16*>(P), items, F / kPer,
                                     static_cast<__nv_bfloat16*>(dP));
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "gated_backward_kernel");
}

}  // namespace dfs
