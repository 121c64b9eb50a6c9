// The whole backward of a dense or gated product of at most 4 tokens in one launch:
//   dP = dY act'(P)  (gated: [dH act'(g) u | dH act(g)]),
//   dX[t][d] = sum_f dP[t][f] W[f][d],  dW[f][d] = sum_t dP[t][f] X[t][d],  db[f] = sum_t dP[t][f].
//
// With so few tokens the weights' bytes bound it (W read once, dW written once): 64 columns
// of W and dW a cluster of 8 CTAs, each CTA an eighth of their rows.  A CTA computes dP of
// 512 rows at a time into shared memory, in fp32: it is no tensor-core operand here and is
// never rounded.  Then eight lanes take a row's 64 columns, 16 bytes each, and both
// products' terms come from the one pass over the row: dX adds up in registers, dW's row is
// finished.  dX is joined over a warp's four rows, the warps and the cluster's CTAs (through
// their shared memory), always in the same order.  No workspace.
// One launch where the tensor-core path takes two.  With the activation and a bias, on the
// GPU: 1 token, 512 x 512: 3.6 us in place of 7.6; 4 tokens, 1024 x 4096: 10.3 in place of 15.6.
// 8 tokens need 176 registers, one CTA an SM: 1024 x 4096 took 25.5 us.
// The grid follows D alone, 8 CTAs for 64 columns, each with an eighth of the rows, so narrow D with
// many rows leaves most SMs idle: 4 tokens, 64 x 4096: 9.2 us; 64 x 65536: 99 (79 with one token),
// where 5 tokens on the tensor cores take 12.3 and 49.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "activations.cuh"
#include "dense_ptx.cuh"
#include "layer_ops.h"
#include "packed.cuh"

namespace dfs {
namespace {

using namespace packed;

constexpr int kThreads = 256;
static_assert(kFewBackward == 4, "instantiations");
constexpr int kWarps = kThreads / 32;
constexpr int kCols = 64;                    // columns of a cluster: 8 lanes of 8
constexpr int kSplit = 8;                    // CTAs of a cluster
constexpr int kChunk = 512;                  // rows of dP in shared memory
constexpr int kGroups = kThreads / 8;        // rows at once

struct FewBackArgs {
    const __nv_bfloat16 *x, *w, *dy, *pre;   // [T][D], [cols][D], [T][F], [T][cols] (null: no activation)
    __nv_bfloat16 *dx, *dw, *db;             // each may be null
    int32_t T, D, F, cols;                   // cols: F, or 2 F when gated
    int32_t act;
};

__device__ __forceinline__ void widen(const uint4& r, F2 (&v)[4]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = f2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
}
__device__ __forceinline__ uint4 narrow(const F2 (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = un(v[j]);
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// dP of rows fb .. fb + rows - 1 into shared memory, all of a row's loads in flight together.
template <int kT, bool kGated, int kAct>
__device__ __forceinline__ void fill(const FewBackArgs& a, int fb, int rows, bool sums, float (&dp)[kT][kChunk]) {
    for (int r = threadIdx.x; r < rows; r += kThreads) {
        const int f = fb + r, c = kGated && f >= a.F ? f - a.F : f;
        __nv_bfloat16 d[kT], p[kT], u[kT];
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            d[t] = p[t] = u[t] = __float2bfloat16_rn(0.f);
            if (t >= a.T) continue;
            d[t] = a.dy[(int64_t)t * a.F + c];
            if (kGated || kAct != DIFFUSER_ACT_NONE) p[t] = a.pre[(int64_t)t * a.cols + c];
            if (kGated && f < a.F) u[t] = a.pre[(int64_t)t * a.cols + a.F + c];
        }
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            float v = __bfloat162float(d[t]);
            if (kGated || kAct != DIFFUSER_ACT_NONE) {
                const float2 vs = act::value_slope<kAct>(__bfloat162float(p[t]));
                v *= kGated ? (f < a.F ? __bfloat162float(u[t]) * vs.y : vs.x) : vs.y;
            }
            if (t >= a.T) v = 0.f;
            dp[t][r] = v;
            sum += v;
        }
        if (sums) a.db[f] = __float2bfloat16_rn(sum);
    }
}

// kT: tokens, rounded up to 1, 2 or 4 (dP and X of the missing ones are 0)
template <int kT, bool kGated>
__global__ void __launch_bounds__(kThreads) few_backward_kernel(const FewBackArgs a) {
    __shared__ float dp[kT][kChunk];
    __shared__ float part[kWarps][kT][kCols];
    __shared__ __align__(16) float mine[kT][kCols];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = (int)ptx::cluster_ctarank();
    const int slab = (int)blockIdx.x / kSplit;
    const int c = slab * kCols + (tid & 7) * 8;              // D is a multiple of 8: in or out together
    const bool in = c < a.D;
    const int f0 = (int)((int64_t)a.cols * split / kSplit), f1 = (int)((int64_t)a.cols * (split + 1) / kSplit);

    F2 x[kT][4], acc[kT][4];
#pragma unroll
    for (int t = 0; t < kT; ++t) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (in && a.dw && t < a.T) r = *reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.D + c);
        widen(r, x[t]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = both(0.f);
    }

    for (int fb = f0; fb < f1; fb += kChunk) {
        const int rows = min(kChunk, f1 - fb);
        const bool sums = a.db && slab == 0;
        switch (a.act) {
            case DIFFUSER_ACT_RELU: fill<kT, kGated, DIFFUSER_ACT_RELU>(a, fb, rows, sums, dp); break;
            case DIFFUSER_ACT_GELU: fill<kT, kGated, DIFFUSER_ACT_GELU>(a, fb, rows, sums, dp); break;
            case DIFFUSER_ACT_GELU_TANH: fill<kT, kGated, DIFFUSER_ACT_GELU_TANH>(a, fb, rows, sums, dp); break;
            case DIFFUSER_ACT_SILU: fill<kT, kGated, DIFFUSER_ACT_SILU>(a, fb, rows, sums, dp); break;
            default: fill<kT, kGated, DIFFUSER_ACT_NONE>(a, fb, rows, sums, dp); break;
        }
        __syncthreads();
        if (in) {
#pragma unroll 4
            for (int r = tid >> 3; r < rows; r += kGroups) {
                const int64_t at = (int64_t)(fb + r) * a.D + c;
                F2 w[4], g[4];
                if (a.dx) widen(*reinterpret_cast<const uint4*>(a.w + at), w);
#pragma unroll
                for (int j = 0; j < 4; ++j) g[j] = both(0.f);
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    const F2 d = both(dp[t][r]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (a.dx) acc[t][j] = fma(w[j], d, acc[t][j]);
                        g[j] = fma(x[t][j], d, g[j]);
                    }
                }
                if (a.dw) *reinterpret_cast<uint4*>(a.dw + at) = narrow(g);
            }
        }
        __syncthreads();
    }
    if (!a.dx) return;                                       // (all of the cluster's threads)

    // the warp's four rows, the warps, the CTAs
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float2 v = un(acc[t][j]);
            v.x += __shfl_xor_sync(0xffffffffu, v.x, 8);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, 8);
            v.x += __shfl_xor_sync(0xffffffffu, v.x, 16);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, 16);
            if (lane < 8) *reinterpret_cast<float2*>(&part[warp][t][lane * 8 + 2 * j]) = v;
        }
    __syncthreads();
    for (int e = tid; e < kT * kCols; e += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) s += part[k][e / kCols][e % kCols];
        mine[e / kCols][e % kCols] = s;
    }
    ptx::cluster_sync();
    // pairs of columns, an eighth of them a CTA
    for (int e = split * kThreads + tid; e < a.T * kCols / 2; e += kSplit * kThreads) {
        const int t = e / (kCols / 2), cc = e % (kCols / 2) * 2, d = slab * kCols + cc;
        if (d >= a.D) continue;
        const uint32_t at = ptx::smem_u32(&mine[t][cc]);
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kSplit; ++k) {
            const float2 v = ptx::ld_cluster_f2(ptx::map_rank(at, (uint32_t)k));
            s.x += v.x;
            s.y += v.y;
        }
        *reinterpret_cast<__nv_bfloat162*>(a.dx + (int64_t)t * a.D + d) = __floats2bfloat162_rn(s.x, s.y);
    }
    ptx::cluster_sync();                                     // nobody leaves while its sums are read
}

template <int kT, bool kGated>
int launch_as(const FewBackArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(kSplit * ((a.D + kCols - 1) / kCols)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSplit;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t err;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        err = cudaLaunchKernelEx(&cfg, few_backward_kernel<kT, kGated>, a);
    }
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "few_backward_kernel");
}

template <bool kGated>
int launch_for(const FewBackArgs& a, cudaStream_t stream) {
    if (a.T == 1) return launch_as<1, kGated>(a, stream);
    if (a.T == 2) return launch_as<2, kGated>(a, stream);
    return launch_as<4, kGated>(a, stream);
}

}  // namespace

int launch_few_backward(const void* X, const void* W, const void* dY, const void* pre, int64_t T, int32_t D, int32_t F,
                        int32_t act, bool gated, void* dX, void* dW, void* dbias, cudaStream_t stream) {
    FewBackArgs a{};
    a.x = static_cast<const __nv_bfloat16*>(X);
    a.w = static_cast<const __nv_bfloat16*>(W);
    a.dy = static_cast<const __nv_bfloat16*>(dY);
    a.pre = static_cast<const __nv_bfloat16*>(pre);
    a.dx = static_cast<__nv_bfloat16*>(dX);
    a.dw = static_cast<__nv_bfloat16*>(dW);
    a.db = static_cast<__nv_bfloat16*>(dbias);
    a.T = (int32_t)T;
    a.D = D;
    a.F = F;
    a.cols = gated ? 2 * F : F;
    a.act = act;
    return gated ? launch_for<true>(a, stream) : launch_for<false>(a, stream);
}

}  // namespace dfs
