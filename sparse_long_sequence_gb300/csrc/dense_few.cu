// Forward products of a few tokens (a decoding step, a short batch): the weights' bytes
// bound them.
//
// Y[t][f] = sum_k W[f][k] X[t][k] in tiles of 128 features x bn tokens.  Features are the
// MMA's 128 rows and tokens its columns, so a step of few tokens pads to 16 columns and not
// to 128 rows, and a warp's 32 accumulator lanes are neighbouring features of one token.
// Gated: 64 gate rows and 64 up rows of the weights a tile.
//
// K is split over the CTAs of a cluster: CTA s of S takes K steps [s kb/S, (s+1) kb/S)
// through a TMA ring into tcgen05 MMAs (fp32 accumulators in tensor memory), writes its
// partial tile to its own shared memory, and after a cluster barrier every CTA sums its share
// of the elements over the S partials in rank order (the result does not depend on timing),
// applies the epilogue and stores.  One launch, no workspace, no atomics.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>

#include "activations.cuh"
#include "band_common.cuh"
#include "dense_ptx.cuh"
#include "dense_tma.h"
#include "layer_ops.h"

namespace dfs {
namespace {

constexpr int kTI = 128;                         // tile rows (i)
constexpr int kTK = 64;                          // K step: 64 bf16, one 128-byte row
constexpr int kABytes = kTI * kTK * 2;           // 16 KB
constexpr int kMaxStages = 5;                  // 18 or 20 KB each: two CTAs an SM
constexpr int kThreads = 256;                    // warp 0 loads, warp 1 multiplies, all reduce
constexpr int kMaxSplit = 4;

constexpr int kMaxSmem = 1024 + kMaxStages * (kABytes + 32 * kTK * 2);

struct FewArgs {
    int32_t I, J;              // result extents (gated: I = F, the tile has 64 gate and 64 up rows)
    int32_t k_blocks;          // K steps of 64 in all
    int32_t i_tiles;
    int32_t splits;            // CTAs of a cluster, each with its part of K
    int32_t bn, stages, tmem_cols;
    __nv_bfloat16* out;        // [J][I]
    __nv_bfloat16* pre;        // [J][I] ([J][2 I] gated) or null
    const __nv_bfloat16* bias;       // [I] or null
    const __nv_bfloat16* residual;   // [J][I] or null
    int32_t act;
    int* status;
};

__device__ __forceinline__ float2 bf16x2(const __nv_bfloat16* p) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void put_bf16x2(__nv_bfloat16* p, float x, float y) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
}

template <bool kGated>
__global__ void __launch_bounds__(kThreads)
dense_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, FewArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[1];
    __shared__ uint32_t tmem_slot;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int splits = a.splits, split = (int)ptx::cluster_ctarank();
    const int tile = (int)blockIdx.x / splits;
    constexpr int kRowsI = kGated ? kTI / 2 : kTI;                   // result features of a tile
    const int i0 = (tile % a.i_tiles) * kRowsI, j0 = (tile / a.i_tiles) * a.bn;
    const int kb0 = (int)((int64_t)a.k_blocks * split / splits);
    const int kb1 = (int)((int64_t)a.k_blocks * (split + 1) / splits);
    const int b_bytes = a.bn * kTK * 2, stage_bytes = kABytes + b_bytes;

    if (warp == 1) ptx::tmem_alloc(&tmem_slot, (uint32_t)a.tmem_cols);
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) { ptx::mbar_init(&full[s], 1); ptx::mbar_init(&empty[s], 1); }
        ptx::mbar_init(acc_full, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmA);
        ptx::prefetch_tensormap(&tmB);
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == 0) {
        for (int kb = kb0, g = 0; kb < kb1; ++kb, ++g) {
            const int s = g % a.stages;
            if (g >= a.stages) ptx::mbar_wait(&empty[s], ((g / a.stages) - 1) & 1, a.status);
            __syncwarp();
            if (ptx::elect_one()) {
                uint8_t* sa = smem + s * stage_bytes;
                uint8_t* sb = sa + kABytes;
                ptx::mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes);
                if constexpr (kGated) {
                    ptx::tma_load_3d(sa, &tmA, &full[s], kb * kTK, i0, 0);       // 64 gate rows, 64 up rows
                } else {
                    ptx::tma_load_2d(sa, &tmA, &full[s], kb * kTK, i0);
                }
                ptx::tma_load_2d(sb, &tmB, &full[s], kb * kTK, j0);
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = ptx::mma_idesc_bf16(kTI, (uint32_t)a.bn, false, false);
        const uint64_t ad0 = ptx::sw128_kmajor_desc(ptx::smem_u32(smem));
        const uint64_t bd0 = ptx::sw128_kmajor_desc(ptx::smem_u32(smem) + kABytes);
        for (int kb = kb0, g = 0; kb < kb1; ++kb, ++g) {
            const int s = g % a.stages;
            ptx::mbar_wait(&full[s], (g / a.stages) & 1, a.status);
            __syncwarp();
            ptx::tc_fence_after();
            const uint64_t ad = ad0 + (uint64_t)(s * (stage_bytes >> 4));
            const uint64_t bd = bd0 + (uint64_t)(s * (stage_bytes >> 4));
#pragma unroll
            for (int ks = 0; ks < kTK / 16; ++ks)
                if (ptx::elect_one())
                    ptx::mma_bf16_ss(tmem, ad + 2 * ks, bd + 2 * ks, idesc, g > 0 || ks > 0);
            if (ptx::elect_one()) ptx::mma_commit(&empty[s]);
        }
        if (ptx::elect_one()) ptx::mma_commit(acc_full);
        // drain: the last commits land before the CTA exits
        const int steps = kb1 - kb0;
        for (int s = 0; s < a.stages; ++s) {
            const int uses = (steps - s + a.stages - 1) / a.stages;
            if (uses > 0) ptx::mbar_wait(&empty[s], (uses - 1) & 1, a.status);
        }
    }
    __syncwarp();
    // the MMAs have read every stage and written the accumulator
    ptx::mbar_wait(acc_full, 0, a.status);
    __syncwarp();
    ptx::tc_fence_after();

    // partial tile -> shared memory [j][128] fp32 (the ring is free)
    float* part = reinterpret_cast<float*>(smem);
    {
        const int quad = warp & 3;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        for (int c0 = (warp >> 2) * 16; c0 < a.bn; c0 += 32) {
            float v[16];
            __syncwarp();
            ptx::tmem_ld16(tmem + lane_base + c0, v);
#pragma unroll
            for (int c = 0; c < 16; ++c) part[(c0 + c) * kTI + quad * 32 + lane] = v[c];
        }
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, (uint32_t)a.tmem_cols);
    }

    // this CTA's share of the element pairs (two neighbouring features)
    const int live_j = min(a.bn, a.J - j0);
    constexpr int kPairs = kRowsI / 2;
    uint32_t peer[kMaxSplit];
#pragma unroll
    for (int s = 0; s < kMaxSplit; ++s) peer[s] = s < splits ? ptx::map_rank(ptx::smem_u32(part), (uint32_t)s) : 0;
    for (int e = split * kThreads + threadIdx.x; e < live_j * kPairs; e += splits * kThreads) {
        const int j = e / kPairs, ii = (e % kPairs) * 2, i = i0 + ii;
        if (i >= a.I) continue;                       // I is even: a pair is in or out
        const uint32_t at = (uint32_t)(j * kTI + ii) * 4;
        float2 v = make_float2(0.f, 0.f), w = make_float2(0.f, 0.f);
#pragma unroll
        for (int s = 0; s < kMaxSplit; ++s) {
            if (s >= splits) break;
            const float2 x = ptx::ld_cluster_f2(peer[s] + at);
            v.x += x.x; v.y += x.y;
            if constexpr (kGated) {
                const float2 y = ptx::ld_cluster_f2(peer[s] + at + 4 * kRowsI);
                w.x += y.x; w.y += y.y;
            }
        }
        const int64_t row = j0 + j;
        if constexpr (kGated) {
            if (a.pre) {
                put_bf16x2(a.pre + row * 2 * a.I + i, v.x, v.y);
                put_bf16x2(a.pre + row * 2 * a.I + a.I + i, w.x, w.y);
            }
            v = make_float2(act::value_of(a.act, v.x) * w.x, act::value_of(a.act, v.y) * w.y);
        } else {
            if (a.bias) {
                const float2 b = bf16x2(a.bias + i);
                v.x += b.x; v.y += b.y;
            }
            if (a.pre) put_bf16x2(a.pre + row * a.I + i, v.x, v.y);
            if (a.act) v = make_float2(act::value_of(a.act, v.x), act::value_of(a.act, v.y));
            if (a.residual) {
                const float2 r = bf16x2(a.residual + row * a.I + i);
                v.x += r.x; v.y += r.y;
            }
        }
        put_bf16x2(a.out + row * a.I + i, v.x, v.y);
    }
    ptx::cluster_sync();                              // nobody leaves while its partials are read
}

template <bool kGated>
int launch_few_as(const CUtensorMap& tmA, const CUtensorMap& tmB, const FewArgs& a, int64_t tiles,
                    cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const int stage_bytes = kABytes + a.bn * kTK * 2;
    const int ring = a.stages * stage_bytes, part = a.bn * kTI * 4;
    const int smem = 1024 + (ring > part ? ring : part);
    cudaError_t err = allow_smem(dense_few_kernel<kGated>, kMaxSmem, done);
    if (err != cudaSuccess) return cuda_fail(err, "cudaFuncSetAttribute(dense few kernel)");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * a.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        err = cudaLaunchKernelEx(&cfg, dense_few_kernel<kGated>, tmA, tmB, a);
    }
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "dense_few_kernel");
}

}  // namespace

// bn: 16 up to 16 tokens, 32 above (the accumulator's columns; two tiles of 32 take 64 tokens
// faster than one of 64: 5.2 and 6.3 us, gated, 512 -> 512).  splits: as many as leave every
// CTA two K steps and the grid within two CTAs an SM, at most 4: a cluster of 8 costs more to
// start than it saves (512 x 512 to 768 x 2048, 16 tokens: 5.4 to 6.6 us with 8, 5.1 to 5.4 with
// 4, 6.9 to 8.0 with 1).
int launch_dense_few(const DenseArgs& d, cudaStream_t stream) {
    FewArgs a{};
    const int64_t F = d.gated ? d.cols / 2 : d.cols;
    const int rows_i = d.gated ? kTI / 2 : kTI;
    a.I = (int32_t)F;
    a.J = (int32_t)d.rows;
    a.k_blocks = (d.inner + kTK - 1) / kTK;
    a.i_tiles = (int32_t)((F + rows_i - 1) / rows_i);
    a.bn = d.rows <= 16 ? 16 : 32;
    a.tmem_cols = 32;
    const int64_t tiles = (int64_t)a.i_tiles * ((d.rows + a.bn - 1) / a.bn);
    if (tiles > INT32_MAX / kMaxSplit) return fail(DIFFUSER_ERR_OVERFLOW, "dense product too large");
    a.splits = 1;
    while (a.splits < kMaxSplit && tiles * a.splits * 2 <= 2 * 152 && a.k_blocks >= 4 * a.splits) a.splits *= 2;
    const int steps = (a.k_blocks + a.splits - 1) / a.splits;
    a.stages = steps < kMaxStages ? steps : kMaxStages;
    a.out = static_cast<__nv_bfloat16*>(d.out);
    a.pre = static_cast<__nv_bfloat16*>(d.pre);
    a.bias = static_cast<const __nv_bfloat16*>(d.bias);
    a.residual = static_cast<const __nv_bfloat16*>(d.residual);
    a.act = d.act;
    a.status = d.status;
    CUtensorMap tmA, tmB;
    int st = d.gated ? map_halves(&tmA, d.b, d.inner, F, kTK, kTI / 2, 2) : map_matrix(&tmA, d.b, d.inner, F, kTK, kTI);
    if (!st) st = map_matrix(&tmB, d.a, d.inner, d.rows, kTK, a.bn);
    if (st) return st;
    return d.gated ? launch_few_as<true>(tmA, tmB, a, tiles, stream) : launch_few_as<false>(tmA, tmB, a, tiles, stream);
}

}  // namespace dfs
