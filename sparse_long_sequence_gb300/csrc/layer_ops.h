// Internal declarations of the operators around the module: the per-head norms
// with the position rotation and the rotation alone (qk_norm_rope.cu), the dense product with its
// epilogue and the gated product (dense_pick.cu, dense_pair.cu, dense_few.cu, dense_act.cu), and their entry
// points (layer_ops_abi.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include <cstdint>

#include "internal.h"

namespace dfs {

// Status block of the projections and dense products on the current device
// (abi.cu): the block's device address and its page-locked host mirror.
struct ProjStatus {
    int* d = nullptr;
    int* h = nullptr;
};
int projection_status(ProjStatus* out);
// its device word, or DIFFUSER_ERR_DEVICE where a kernel has reported a failure (layer_ops_abi.cu)
int ready_status(int** word);
int check_workspace_bytes(size_t need, void* ws, size_t ws_bytes);

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) once per kernel and device.
// `done` is the kernel's own word, one bit per device.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return err;
}

// ---- norms and rotation (qk_norm_rope.cu) ------------------------------------
struct QkArgs {
    const void *q, *k;              // [B][Hq][n][64], [B][Hk][n][64]
    const void *dqo, *dko;          // backward: gradients of the results
    void *qo, *ko;                  // results (forward) or gradients dQ, dK
    const void *wq, *wk;            // [64] or null (ones)
    const int64_t* pos;             // [B][n] or null
    int64_t pos0;                   // added to every position
    int64_t tokens;                 // B n
    int64_t n;
    int32_t Hq, Hk;
    int32_t rot;                    // rotated features: 0, 16, 32, 48, 64
    float eps;
    float magnitude;                // the rotation alone: factor of the turned features
    float* partial;                 // backward: [blocks][64] sums of the weights' gradients, or null
    // turns per position of pair i, in units of 2^-64, and what is left of it, of 2^-128
    uint64_t freq[kHeadDim / 2], freq_low[kHeadDim / 2];
};
int launch_qk_norm_rope(const QkArgs& a, int32_t dtype, bool interleaved, cudaStream_t stream);
// the rotation alone (q, k, qo, ko, pos and the turns); `back` turns the other way
int launch_rope(const QkArgs& a, int32_t dtype, bool interleaved, bool back, cudaStream_t stream);
// blocks of the backward kernel (rows of `partial`)
int64_t qk_backward_blocks(int64_t tokens, int64_t Hq, int64_t Hk);
int launch_qk_norm_rope_backward(const QkArgs& a, int32_t dtype, bool interleaved, void* dwq, void* dwk,
                                 cudaStream_t stream);

// ---- dense products (dense_pick.cu chooses the kernel) -----------------------------------------
// Which product: Y[t][f] = sum_k X[t][k] W[f][k] (forward),
// dX[t][k] = sum_f dP[t][f] W[f][k], dW[f][k] = sum_t dP[t][f] X[t][k].
enum DenseForm { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };

struct DenseArgs {
    const void* a;                  // left matrix: X (forward), dP (both gradients)
    const void* b;                  // right matrix: W (forward, input gradient), X (weight gradient)
    int64_t rows;                   // tokens T
    int32_t inner;                  // D: width of X and of W's rows
    int32_t cols;                   // width of dP; rows of W (2 F for the gated product)
    void* out;                      // bf16; forward [T][cols] or [T][F] (gated), dX [T][D], dW [cols][D]
    void* pre;                      // forward: bf16 [T][cols] or null
    const void* bias;               // forward: bf16 [cols] or null
    const void* residual;           // forward: bf16 [T][cols] or null
    int32_t act;                    // forward: diffuser_activation
    bool gated;                     // forward: out = act(P[:, :F]) * P[:, F:], F = cols / 2
    int* status;
};
// forward of a few tokens (dense_few.cu)
int launch_dense_few(const DenseArgs& a, cudaStream_t stream);
// CTA pairs, 256 x bn tiles, bn 128 or 256 (gated: 256); splits 1: persistent, 2 or 4: K split
// over that many pairs of a cluster (dense_pair.cu)
int launch_dense_pair(DenseForm form, const DenseArgs& a, int bn, int splits, cudaStream_t stream);
// clusters of 2 `splits` CTAs of the split kernel that run at once on the current device
int dense_pair_clusters(int splits);
// A bias gradient's fp32 partial sums [chunks][F] and where their sums go (null: nowhere)
struct BiasSums {
    const float* partial;
    int64_t chunks;
    int32_t F;
    __nv_bfloat16* out;
};
int launch_colsum(const BiasSums& b, cudaStream_t stream);                   // dense_act.cu
// both gradients in one launch (dense_pair.cu), and the K steps of its busiest CTA pair
int launch_dense_grads(const DenseArgs& x, const DenseArgs& w, const BiasSums& bias, int bn, cudaStream_t stream);
int64_t dense_grads_steps(const DenseArgs& x, int bn);
// picks the kernel (dense_pick.cu); the gradients: x for dX and w for dW, of one product
int launch_gradients(const DenseArgs& x, const DenseArgs& w, const BiasSums& bias, cudaStream_t stream);
int launch_dense(DenseForm form, const DenseArgs& a, cudaStream_t stream);

// The whole backward of up to kFewBackward tokens in one launch (dense_few_backward.cu); null
// results are left out.
constexpr int64_t kFewBackward = 4;
int launch_few_backward(const void* X, const void* W, const void* dY, const void* pre, int64_t T, int32_t D, int32_t F,
                        int32_t act, bool gated, void* dX, void* dW, void* dbias, cudaStream_t stream);

// ---- the activations' backward (dense_act.cu) --------------------------------
// dP[t][f] = dY[t][f] act'(P[t][f]); colsum (or null): bf16 [F], the column sums of dP in fp32:
// written where the rows are one chunk, else left in `partial` ([act_chunks][F]) and described in
// *sums for the caller to finish.  dP may be null with act none (dP is dY itself).
int64_t act_chunks(int64_t rows, int32_t F);
int launch_act_backward(const void* dY, const void* P, int64_t rows, int32_t F, int32_t act, void* dP,
                        void* colsum, float* partial, BiasSums* sums, cudaStream_t stream);
// gated: P [T][2F]; dP[t][f] = dH act'(g) u, dP[t][F + f] = dH act(g)
int launch_gated_backward(const void* dH, const void* P, int64_t rows, int32_t F, int32_t act, void* dP,
                          cudaStream_t stream);

}  // namespace dfs
