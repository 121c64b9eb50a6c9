// Dense products with many output tiles: a persistent kernel of CTA pairs.
//
// Computes C[i][j] = sum_k A[i][k] B[j][k] in tiles of 256 (i) x kBn (j), j being the
// contiguous index of the result:
//   forward      A = X (K-major), B = W (K-major)            C = P [T][F]
//   input grad   A = dP (K-major), B = W (j-major)           C = dX [T][D]
//   weight grad  A = dP (i-major), B = X (j-major)           C = dW [F][D]
// Operands stay in their row-major layout: where the summed index is not the contiguous
// one, the 64 x 64 boxes load as they are and the MMA reads them MN-major.
//
// The two CTAs of a cluster work on one tile (tcgen05 cta_group::2, M = 256): each loads
// its 128 rows of A and half of B's rows, so B crosses shared memory once per pair and
// not once per CTA, and one thread of CTA 0 issues the MMAs for both.  Each CTA holds its
// 128 x kBn fp32 accumulator in tensor memory, twice, so that a tile's epilogue overlaps
// the next tile's MMAs.
//
// Warps of a CTA: 0 loads (TMA, a ring of K steps of 64), 1 multiplies (CTA 0 only), the others
// are the epilogue, each alone on its 32 accumulator lanes and some of the tile's columns, in blocks of
// 32: tensor memory -> registers (bias, activation, residual) -> a swizzled 2 KB buffer of
// its own (used in turn) -> TMA store, which drops what lies outside the result.  Warps
// wait for no other warp: with 128 x 64 blocks shared by four warps the forward 512 -> 2048 of
// 32768 tokens with gelu and kept pre-activations took 132 us.  The residual arrives by TMA in
// the buffer the result leaves from.  Gated: B's rows are 128 gate rows (CTA 0) and 128 up rows
// (CTA 1), so columns c and 128 + c of an accumulator lane are g and u of one element.
// Every barrier wait is bounded and records a status instead of hanging.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>

#include "activations.cuh"
#include "dense_ptx.cuh"
#include "dense_tma.h"
#include "layer_ops.h"

namespace dfs {
namespace {

constexpr int kTI = 256;                          // tile rows of a pair, 128 a CTA
constexpr int kTK = 64;                           // K step: 64 bf16, one 128-byte row
constexpr int kBox = 64 * kTK * 2;                // an MN-major box: 64 x 64, 8 KB
constexpr int kABytes = 128 * kTK * 2;            // 16 KB a CTA
constexpr int kThreads = 320;
constexpr int kEpiWarp0 = 2;
constexpr int kBlock = 32;                        // an epilogue step: 32 rows x 32 columns of a warp
constexpr int kBufBytes = 32 * kBlock * 2;        // 2 KB
constexpr int kEpiBytes = 32 * kBufBytes;          // the epilogue warps' buffers: 2 of 16, 4 of 8
constexpr int kBarBytes = 1024;                   // barriers and the tensor memory's address
constexpr int kGroupTiles = 8;                    // i tiles walked together (L2 reuse of both operands)

constexpr int b_bytes(int bn) { return bn / 2 * kTK * 2; }
constexpr int stage_count(int bn) {
    return (227 * 1024 - 1024 - kBarBytes - kEpiBytes) / (kABytes + b_bytes(bn));
}
constexpr int smem_bytes(int bn) {
    return 1024 + stage_count(bn) * (kABytes + b_bytes(bn)) + kEpiBytes + kBarBytes;
}
static_assert(stage_count(256) == 5 && smem_bytes(256) <= 227 * 1024, "shared memory per CTA");
static_assert(stage_count(128) == 6 && smem_bytes(128) <= 227 * 1024, "shared memory per CTA");

struct PairArgs {
    int32_t I, J;              // result extents (gated: J = F)
    int32_t k_blocks;
    int32_t i_tiles, j_tiles;
    int32_t act;
    bool pre, residual;        // their maps are valid
    const __nv_bfloat16* bias;
    int* status;
};

struct Tile { int i0, j0; };
// tile t: groups of kGroupTiles i tiles, i fastest inside a group
__device__ __forceinline__ Tile tile_at(const PairArgs& a, int t, int width) {
    const int per = kGroupTiles * a.j_tiles;
    const int grp = t / per, in = t - grp * per;
    const int rows = min(kGroupTiles, a.i_tiles - grp * kGroupTiles);
    return {(grp * kGroupTiles + in % rows) * kTI, in / rows * width};
}

// 32 neighbouring columns of a lane's row as 16 packed pairs.  (tcgen05.ld is a warp's instruction,
// and lane 0 comes from issuing copies.)
using packed::F2;
__device__ __forceinline__ void load_acc(uint32_t taddr, F2 (&v)[16]) {
    uint32_t r[32];
    __syncwarp();
    ptx::tmem_ld32_issue(taddr, r);
    ptx::tmem_ld_wait32(r);
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] = packed::f2(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1]));
}
// v = act(v) (the activation is uniform over the launch)
__device__ __forceinline__ void activate(int which, F2 (&v)[16]) {
#define DFS_EACH(A) case A: _Pragma("unroll") for (int c = 0; c < 16; ++c) v[c] = act::value2<A>(v[c]); break;
    switch (which) {
        DFS_EACH(DIFFUSER_ACT_RELU)
        DFS_EACH(DIFFUSER_ACT_GELU)
        DFS_EACH(DIFFUSER_ACT_GELU_TANH)
        DFS_EACH(DIFFUSER_ACT_SILU)
        default: break;
    }
#undef DFS_EACH
}
// into the lane's row of a swizzled buffer (64-byte rows: 16-byte piece q at q ^ ((row / 2) % 4),
// so that eight neighbouring rows' writes fall in eight bank groups)
__device__ __forceinline__ void put_row(uint8_t* row, int sw, const F2 (&v)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t w[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const float2 x = packed::un(v[4 * q + p]);
            const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
            w[p] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(row + ((q ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// eight bf16 values added to v[0..3]
__device__ __forceinline__ void add8(F2* v, const uint4& r) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int p = 0; p < 4; ++p)
        v[p] = packed::add(v[p], packed::f2(__uint_as_float(w[p] << 16), __uint_as_float(w[p] & 0xffff0000u)));
}

// ---- the roles both kernels share -------------------------------------------------
template <bool kAMn, bool kBMn, bool kGated, int kBn>
struct Roles {
    static constexpr int kStages = stage_count(kBn);
    static constexpr int kBBytes = b_bytes(kBn);
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kWidth = kGated ? kBn / 2 : kBn;     // result columns of a tile

    // One K step of a tile (rows from ai, columns from bj: this CTA's shares) into stage s; `lead`
    // is the cluster rank of the pair's first CTA, whose full barrier both CTAs' copies report to.
    static __device__ __forceinline__ void load(uint8_t* smem, uint64_t* full, int s, const CUtensorMap* tmA,
                                                const CUtensorMap* tmB, int ai, int bj, int kb, int rank, int lead) {
        uint8_t* sa = smem + s * kStageBytes;
        uint8_t* sb = sa + kABytes;
        const uint32_t bar = ptx::map_rank(ptx::smem_u32(&full[s]), (uint32_t)lead);
        if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
        if constexpr (kAMn) {
            ptx::pair_load_2d(sa, tmA, bar, ai, kb * kTK);
            ptx::pair_load_2d(sa + kBox, tmA, bar, ai + 64, kb * kTK);
        } else {
            ptx::pair_load_2d(sa, tmA, bar, kb * kTK, ai);
        }
        if constexpr (kGated) {
            ptx::pair_load_3d(sb, tmB, bar, kb * kTK, bj, rank);
        } else if constexpr (kBMn) {
#pragma unroll
            for (int c = 0; c < kBn / 2; c += 64) ptx::pair_load_2d(sb + c / 64 * kBox, tmB, bar, bj + c, kb * kTK);
        } else {
            ptx::pair_load_2d(sb, tmB, bar, kb * kTK, bj);
        }
    }
    // first row and column of this CTA's shares of the operands
    static __device__ __forceinline__ int a_row(const Tile& t, int rank) { return t.i0 + 128 * rank; }
    static __device__ __forceinline__ int b_row(const Tile& t, int rank) { return t.j0 + (kGated ? 0 : kBn / 2 * rank); }

    // The MMAs of stage s (one thread of the pair's first CTA), then the commit that frees it.
    static __device__ __forceinline__ void multiply(uint32_t dacc, uint32_t sa0, int s, bool first, uint64_t* empty,
                                                    uint16_t pair_mask) {
        constexpr uint32_t idesc = ptx::mma_idesc_bf16(kTI, kBn, kAMn, kBMn);
        const uint32_t sa = sa0 + s * kStageBytes, sb = sa + kABytes;
        const uint64_t ad = kAMn ? ptx::sw128_mnmajor_desc(sa, kBox) : ptx::sw128_kmajor_desc(sa);
        const uint64_t bd = kBMn ? ptx::sw128_mnmajor_desc(sb, kBox) : ptx::sw128_kmajor_desc(sb);
#pragma unroll
        for (int ks = 0; ks < kTK / 16; ++ks)
            ptx::pair_mma_bf16(dacc, ad + (kAMn ? 128 : 2) * ks, bd + (kBMn ? 128 : 2) * ks, idesc, !first || ks > 0);
        ptx::pair_commit(&empty[s], pair_mask);
    }
    // after g steps: wait until the last commits have landed (before the CTA exits)
    static __device__ __forceinline__ void drain(uint64_t* empty, int g, int* status) {
        for (int s = 0; s < kStages; ++s) {
            const int uses = (g - s + kStages - 1) / kStages;
            if (uses > 0) ptx::mbar_wait(&empty[s], (uses - 1) & 1, status);
        }
    }
};

// kEpilogue: bias, activation, residual and kept pre-activations may be asked for; gated has one.
// 16 epilogue warps then, as the accumulators' arithmetic outlasts the MMAs of a short K: with
// 8 the forward 512 -> 2048 of 32768 tokens, gelu and kept pre-activations, took 99 us.
constexpr int epi_warps(bool epilogue) { return epilogue ? 16 : 8; }
constexpr int pair_threads(bool epilogue) { return 32 * (kEpiWarp0 + epi_warps(epilogue)); }

template <bool kAMn, bool kBMn, bool kGated, int kBn, bool kEpilogue>
__global__ void __launch_bounds__(pair_threads(kEpilogue), 1)
dense_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmPre,
                  const __grid_constant__ CUtensorMap tmRes, const __grid_constant__ PairArgs a) {
    using R = Roles<kAMn, kBMn, kGated, kBn>;
    constexpr int kStages = R::kStages, kWidth = R::kWidth;
    constexpr int kEpiWarps = epi_warps(kEpilogue), kBufs = kEpiBytes / kBufBytes / kEpiWarps;
    constexpr int kEpiCols = kWidth / (kEpiWarps / 4);        // columns of an epilogue warp
    constexpr int kBlocks = kEpiCols / kBlock;
    static_assert(kBlocks >= 1 && kBlocks <= kBufs, "a tile's residual blocks have a buffer each");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* bufs = smem + kStages * R::kStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(bufs + kEpiBytes);   // [kStages] (CTA 0's are used)
    uint64_t* empty = full + kStages;                          // [kStages]
    uint64_t* acc_full = empty + kStages;                      // [2]
    uint64_t* acc_empty = acc_full + 2;                        // [2] (CTA 0's are used)
    uint64_t* res_full = acc_empty + 2;                        // [kEpiWarps][kBufs]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + kEpiWarps * kBufs);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)ptx::cluster_ctarank();
    const int pairs = (int)gridDim.x / 2, pair = (int)blockIdx.x / 2;
    const int total = a.i_tiles * a.j_tiles;
    const int my_tiles = pair < total ? (total - 1 - pair) / pairs + 1 : 0;

    if (warp == 1) ptx::pair_tmem_alloc(tmem_slot, 512);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) { ptx::mbar_init(&full[s], 1); ptx::mbar_init(&empty[s], 1); }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(&acc_full[s], 1);
            ptx::mbar_init(&acc_empty[s], 2 * kEpiWarps);
        }
        for (int s = 0; s < kEpiWarps * kBufs; ++s) ptx::mbar_init(&res_full[s], 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmA);
        ptx::prefetch_tensormap(&tmB);
        ptx::prefetch_tensormap(&tmOut);
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::griddep_wait();                                       // (dP, after the activations' kernel)

    if (warp == 0) {
        // (the whole warp runs the loop; the elected lane issues the copies)
        int g = 0;
        for (int lt = 0; lt < my_tiles; ++lt) {
            const Tile tl = tile_at(a, pair + lt * pairs, kWidth);
            for (int kb = 0; kb < a.k_blocks; ++kb, ++g) {
                const int s = g % kStages;
                if (g >= kStages) ptx::mbar_wait(&empty[s], ((g / kStages) - 1) & 1, a.status);
                __syncwarp();
                if (ptx::elect_one())
                    R::load(smem, full, s, &tmA, &tmB, R::a_row(tl, rank), R::b_row(tl, rank), kb, rank, 0);
            }
        }
        R::drain(empty, g, a.status);
    } else if (warp == 1) {
        if (rank == 0) {
            int g = 0;
            for (int lt = 0; lt < my_tiles; ++lt) {
                const int buf = lt & 1;
                // both CTAs' epilogues have read this accumulator's previous tile
                if (lt >= 2) ptx::mbar_wait(&acc_empty[buf], ((lt / 2) - 1) & 1, a.status);
                __syncwarp();
                ptx::tc_fence_after();
                for (int kb = 0; kb < a.k_blocks; ++kb, ++g) {
                    const int s = g % kStages;
                    ptx::mbar_wait(&full[s], (g / kStages) & 1, a.status);
                    __syncwarp();
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) R::multiply(tmem + buf * kBn, ptx::smem_u32(smem), s, kb == 0, empty, 3);
                }
                if (ptx::elect_one()) ptx::pair_commit(&acc_full[buf], 3);
            }
        }
    } else {
        const int grp = (warp - kEpiWarp0) >> 2, quad = warp & 3;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        uint8_t* wbuf = bufs + (warp - kEpiWarp0) * kBufs * kBufBytes;
        const int row_at = lane * 64, sw = (lane >> 1) & 3;    // a lane's row of a buffer and its swizzle
        uint64_t* rbar = res_full + (warp - kEpiWarp0) * kBufs;
        const uint32_t acc_empty0 = ptx::map_rank(ptx::smem_u32(acc_empty), 0);
        const bool lead = lane == 0;                           // issues the warp's copies
        int u = 0;                                             // the warp's stores so far; buffer u % kBufs
        uint32_t rphase = 0;                                   // bit b: parity of buffer b's next residual
        for (int lt = 0; lt < my_tiles; ++lt) {
            const Tile tl = tile_at(a, pair + lt * pairs, kWidth);
            const int buf = lt & 1;
            const int row0 = tl.i0 + 128 * rank + 32 * quad;
            const int c_first = tl.j0 + grp * kEpiCols;
            // blocks with something to store
            const int live = row0 < a.I ? max(0, min(kBlocks, (a.J - c_first + kBlock - 1) / kBlock)) : 0;
            auto fetch_residual = [&](int k, int b) {
                ptx::mbar_arrive_expect_tx(&rbar[b], kBufBytes);
                ptx::tma_load_2d(wbuf + b * kBufBytes, &tmRes, &rbar[b], c_first + k * kBlock, row0);
            };
            if (kEpilogue && a.residual && !a.pre && lead && live) {
                // every block's residual into the buffer its result will leave from
                ptx::bulk_wait_read<0>();
                for (int k = 0; k < live; ++k) fetch_residual(k, (u + k) % kBufs);
            }
            ptx::mbar_wait(&acc_full[buf], (lt / 2) & 1, a.status);
            __syncwarp();
            ptx::tc_fence_after();
            const uint32_t acc = tmem + lane_base + buf * kBn + grp * kEpiCols;
            // the accumulator is read: the MMAs of the tile after next may overwrite it
            auto release = [&]() {
                ptx::tc_fence_before();
                __syncwarp();
                if (lead) ptx::mbar_arrive_cluster(acc_empty0 + 8 * buf);
            };
            if (!live) release();
            for (int k = 0; k < live; ++k) {
                const int col = c_first + k * kBlock;
                // one store: wait until its buffer's last one has left, write the rows, hand over
                auto put = [&](const CUtensorMap& map, int part, const F2 (&v)[16]) {
                    uint8_t* b = wbuf + u % kBufs * kBufBytes;
                    if (lead) ptx::bulk_wait_read<kBufs - 1>();
                    __syncwarp();
                    put_row(b + row_at, sw, v);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lead) {
                        if (part >= 0) ptx::tma_store_3d(&map, b, col, part, row0);
                        else ptx::tma_store_2d(&map, b, col, row0);
                        ptx::bulk_commit();
                    }
                    ++u;
                };
                if (kEpilogue && a.residual && a.pre && lead) {
                    ptx::bulk_wait_read<0>();
                    fetch_residual(k, (u + 1) % kBufs);
                }
                F2 v[16];
                load_acc(acc + k * kBlock, v);
                if constexpr (kGated) {
                    // (u is read again after the activation: both at once would not fit 96 registers)
                    F2 w[16];
                    if (a.pre) {
                        put(tmPre, 0, v);
                        load_acc(acc + kBn / 2 + k * kBlock, w);
                        put(tmPre, 1, w);
                    }
                    activate(a.act, v);
                    load_acc(acc + kBn / 2 + k * kBlock, w);
                    if (k + 1 == live) release();
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] = packed::mul(v[c], w[c]);
                } else {
                    if (k + 1 == live) release();
                    if constexpr (kEpilogue) {
                        if (a.bias) {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                if (col + 8 * q < a.J)
                                    add8(v + 4 * q, __ldg(reinterpret_cast<const uint4*>(a.bias + col + 8 * q)));
                        }
                        if (a.pre) put(tmPre, -1, v);
                        activate(a.act, v);
                        if (a.residual) {
                            const int b = u % kBufs;
                            ptx::mbar_wait(&rbar[b], (rphase >> b) & 1, a.status);
                            rphase ^= 1u << b;
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                add8(v + 4 * q, *reinterpret_cast<const uint4*>(wbuf + b * kBufBytes + row_at + ((q ^ sw) << 4)));
                        }
                    }
                }
                put(tmOut, -1, v);
            }
        }
        if (lead) ptx::bulk_wait<0>();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::pair_tmem_dealloc(tmem, 512);
    }
}

// ---- both gradients of a product in one launch --------------------------------------
// dX = dP W and dW = dP^T X need nothing of each other, and neither's tiles fill a whole number
// of waves.  One persistent kernel runs both: a pair takes its share of the longer tiles (K
// steps) first, then of the shorter ones, dealt on the host so that all pairs finish nearly
// together.  Neighbouring pairs work on neighbouring tiles (j fastest) at the same time and read
// the same rows of dP from the L2; with a pair's tiles one after the other the gated backward
// 16384 x 1024 x 2816 read 964 MB from memory and not 458.
struct GradDeal {
    int32_t longer;            // 0: dX has the longer tiles, 1: dW
    int32_t a_pairs;           // pairs with one long tile more
    int32_t longs;             // long tiles of the others
    int32_t a_shorts, a_rest;  // short tiles of the first a_pairs pairs, one more for a_rest of them
    int32_t b_shorts, b_rest;  // and of the others
};
struct GradArgs {
    PairArgs p[2];             // dX, dW
    GradDeal deal;
    BiasSums bias;             // partial sums of the bias gradient to finish (null: none)
};
// counts of a pair's long and short tiles
__device__ __forceinline__ int long_tiles(const GradDeal& d, int pair) { return d.longs + (pair < d.a_pairs); }
__device__ __forceinline__ int short_tiles(const GradDeal& d, int pair) {
    return pair < d.a_pairs ? d.a_shorts + (pair < d.a_rest) : d.b_shorts + (pair - d.a_pairs < d.b_rest);
}
// a pair's k-th long tile (all pairs in rounds) and short tile (the a pairs' rounds, then the b pairs')
__device__ __forceinline__ int long_tile(int pairs, int pair, int k) { return k * pairs + pair; }
__device__ __forceinline__ int short_tile(const GradDeal& d, int pairs, int pair, int k) {
    if (pair < d.a_pairs) return k * d.a_pairs + pair;
    return d.a_pairs * d.a_shorts + d.a_rest + k * (pairs - d.a_pairs) + pair - d.a_pairs;
}

template <int kBn>
__global__ void __launch_bounds__(pair_threads(false), 1)
dense_grads_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmB0,
                   const __grid_constant__ CUtensorMap tmOut0, const __grid_constant__ CUtensorMap tmA1,
                   const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmOut1,
                   const __grid_constant__ GradArgs g) {
    using X = Roles<false, true, false, kBn>;
    using W = Roles<true, true, false, kBn>;
    constexpr int kStages = X::kStages;
    constexpr int kEpiWarps = epi_warps(false), kBufs = kEpiBytes / kBufBytes / kEpiWarps;
    constexpr int kEpiCols = kBn / (kEpiWarps / 4), kBlocks = kEpiCols / kBlock;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* bufs = smem + kStages * X::kStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(bufs + kEpiBytes);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)ptx::cluster_ctarank();
    const int pairs = (int)gridDim.x / 2, pair = (int)blockIdx.x / 2;
    const int my_longs = long_tiles(g.deal, pair), my_tiles = my_longs + short_tiles(g.deal, pair);
    int* const status = g.p[0].status;
    // tile lt of this pair: whose it is (0 dX, 1 dW) and where
    auto kind_of = [&](int lt) { return lt < my_longs ? g.deal.longer : 1 - g.deal.longer; };
    auto tile_of = [&](int lt, int kind) {
        const int t = lt < my_longs ? long_tile(pairs, pair, lt) : short_tile(g.deal, pairs, pair, lt - my_longs);
        const int jt = g.p[kind].j_tiles;
        return Tile{t / jt * kTI, t % jt * kBn};
    };

    if (warp == 1) ptx::pair_tmem_alloc(tmem_slot, 512);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) { ptx::mbar_init(&full[s], 1); ptx::mbar_init(&empty[s], 1); }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(&acc_full[s], 1);
            ptx::mbar_init(&acc_empty[s], 2 * kEpiWarps);
        }
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmA0);
        ptx::prefetch_tensormap(&tmB0);
        ptx::prefetch_tensormap(&tmA1);
        ptx::prefetch_tensormap(&tmB1);
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::griddep_wait();                                       // dP and the bias's partial sums are there

    if (warp == 0) {
        int n = 0;
        for (int lt = 0; lt < my_tiles; ++lt) {
            const int kind = kind_of(lt), kbs = g.p[kind].k_blocks;
            const Tile tl = tile_of(lt, kind);
            const int ai = X::a_row(tl, rank), bj = X::b_row(tl, rank);
            for (int kb = 0; kb < kbs; ++kb, ++n) {
                const int s = n % kStages;
                if (n >= kStages) ptx::mbar_wait(&empty[s], ((n / kStages) - 1) & 1, status);
                __syncwarp();
                if (ptx::elect_one()) {
                    if (kind == 0) X::load(smem, full, s, &tmA0, &tmB0, ai, bj, kb, rank, 0);
                    else W::load(smem, full, s, &tmA1, &tmB1, ai, bj, kb, rank, 0);
                }
            }
        }
        X::drain(empty, n, status);
    } else if (warp == 1) {
        if (rank == 0) {
            int n = 0;
            for (int lt = 0; lt < my_tiles; ++lt) {
                const int buf = lt & 1, kind = kind_of(lt), kbs = g.p[kind].k_blocks;
                // both CTAs' epilogues have read this accumulator's previous tile
                if (lt >= 2) ptx::mbar_wait(&acc_empty[buf], ((lt / 2) - 1) & 1, status);
                __syncwarp();
                ptx::tc_fence_after();
                for (int kb = 0; kb < kbs; ++kb, ++n) {
                    const int s = n % kStages;
                    ptx::mbar_wait(&full[s], (n / kStages) & 1, status);
                    __syncwarp();
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
                        if (kind == 0) X::multiply(tmem + buf * kBn, ptx::smem_u32(smem), s, kb == 0, empty, 3);
                        else W::multiply(tmem + buf * kBn, ptx::smem_u32(smem), s, kb == 0, empty, 3);
                    }
                }
                if (ptx::elect_one()) ptx::pair_commit(&acc_full[buf], 3);
            }
        }
    } else {
        const int grp = (warp - kEpiWarp0) >> 2, quad = warp & 3;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        uint8_t* wbuf = bufs + (warp - kEpiWarp0) * kBufs * kBufBytes;
        const int row_at = lane * 64, sw = (lane >> 1) & 3;
        const uint32_t acc_empty0 = ptx::map_rank(ptx::smem_u32(acc_empty), 0);
        const bool lead = lane == 0;
        if (g.bias.out) {
            // until the first accumulator is full: the bias gradient, 32 columns a CTA at a time, every
            // eighth partial sum a warp
            float* sums = reinterpret_cast<float*>(bufs);
            const int w = warp - kEpiWarp0;
            for (int c0 = (int)blockIdx.x * 32; c0 < g.bias.F; c0 += (int)gridDim.x * 32) {
                const int col = c0 + lane;
                float t = 0.f;
                if (col < g.bias.F) {
#pragma unroll 8
                    for (int64_t k = w; k < g.bias.chunks; k += kEpiWarps) t += g.bias.partial[k * g.bias.F + col];
                }
                sums[w * 32 + lane] = t;
                __syncwarp();                                  // (the last columns' lanes and the others)
                ptx::named_barrier_sync(1, 32 * kEpiWarps);
                if (w == 0 && col < g.bias.F) {
                    t = 0.f;
#pragma unroll
                    for (int k = 0; k < kEpiWarps; ++k) t += sums[k * 32 + lane];
                    g.bias.out[col] = __float2bfloat16_rn(t);
                }
                __syncwarp();
                ptx::named_barrier_sync(1, 32 * kEpiWarps);
            }
        }
        int u = 0;                                             // the warp's stores so far; buffer u % kBufs
        for (int lt = 0; lt < my_tiles; ++lt) {
            const int buf = lt & 1, kind = kind_of(lt);
            const Tile tl = tile_of(lt, kind);
            const int row0 = tl.i0 + 128 * rank + 32 * quad, c_first = tl.j0 + grp * kEpiCols;
            const int live =
                row0 < g.p[kind].I ? max(0, min(kBlocks, (g.p[kind].J - c_first + kBlock - 1) / kBlock)) : 0;
            ptx::mbar_wait(&acc_full[buf], (lt / 2) & 1, status);
            __syncwarp();
            ptx::tc_fence_after();
            const uint32_t acc = tmem + lane_base + buf * kBn + grp * kEpiCols;
            for (int k = 0; k < live; ++k, ++u) {
                F2 v[16];
                load_acc(acc + k * kBlock, v);
                uint8_t* b = wbuf + u % kBufs * kBufBytes;
                if (lead) ptx::bulk_wait_read<kBufs - 1>();
                __syncwarp();
                put_row(b + row_at, sw, v);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lead) {
                    ptx::tma_store_2d(kind == 0 ? &tmOut0 : &tmOut1, b, c_first + k * kBlock, row0);
                    ptx::bulk_commit();
                }
            }
            // the accumulator is read: the MMAs of the tile after next may overwrite it
            ptx::tc_fence_before();
            __syncwarp();
            if (lead) ptx::mbar_arrive_cluster(acc_empty0 + 8 * buf);
        }
        if (lead) ptx::bulk_wait<0>();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::pair_tmem_dealloc(tmem, 512);
    }
}

// ---- few tiles, many K steps: K split over the pairs of a cluster -------------------
// One tile a cluster of 2 S CTAs; pair s takes K steps [s kb/S, (s+1) kb/S).  Every CTA then
// lays its 128 x kBn partial accumulator into its own shared memory (the ring is free; rows
// padded by 16 bytes so that neither the rows' writes nor the row reads conflict), and after a
// cluster barrier CTA (s, rank) sums rows [s 128/S, (s+1) 128/S) of its half of the tile over
// the S partials in rank order, a warp a row, and stores 8 bytes a lane.
__device__ __forceinline__ float4 widen4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4& v) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}
__device__ __forceinline__ float4 act4(int which, const float4& v) {
    return make_float4(act::value_of(which, v.x), act::value_of(which, v.y), act::value_of(which, v.z),
                       act::value_of(which, v.w));
}
__device__ __forceinline__ void add4(float4& a, const float4& b) {
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
}

struct Results {               // row-major [I][J]; pre [I][2 J] when gated
    __nv_bfloat16* out;
    __nv_bfloat16* pre;
    const __nv_bfloat16* residual;
};

template <bool kAMn, bool kBMn, bool kGated, int kBn, int kSplits>
__global__ void __launch_bounds__(kThreads, 1)
dense_pair_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ PairArgs a, const __grid_constant__ Results r) {
    using R = Roles<kAMn, kBMn, kGated, kBn>;
    constexpr int kStages = R::kStages;
    constexpr int kRowBytes = kBn * 4 + 16;
    static_assert(128 * kRowBytes <= kStages * R::kStageBytes, "the partial tile fits the ring");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * R::kStageBytes);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int crank = (int)ptx::cluster_ctarank(), split = crank >> 1, rank = crank & 1;
    const uint16_t pair_mask = (uint16_t)(3u << (2 * split));
    const Tile tl = tile_at(a, (int)blockIdx.x / (2 * kSplits), R::kWidth);
    const int kb0 = (int)((int64_t)a.k_blocks * split / kSplits);
    const int kb1 = (int)((int64_t)a.k_blocks * (split + 1) / kSplits);

    if (warp == 1) ptx::pair_tmem_alloc(tmem_slot, kBn);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) { ptx::mbar_init(&full[s], 1); ptx::mbar_init(&empty[s], 1); }
        ptx::mbar_init(acc_full, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&tmA);
        ptx::prefetch_tensormap(&tmB);
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    ptx::griddep_wait();

    if (warp == 0) {
        int g = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
            const int s = g % kStages;
            if (g >= kStages) ptx::mbar_wait(&empty[s], ((g / kStages) - 1) & 1, a.status);
            __syncwarp();
            if (ptx::elect_one())
                R::load(smem, full, s, &tmA, &tmB, R::a_row(tl, rank), R::b_row(tl, rank), kb, rank, 2 * split);
        }
        R::drain(empty, g, a.status);
    } else if (warp == 1 && rank == 0) {
        int g = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
            const int s = g % kStages;
            ptx::mbar_wait(&full[s], (g / kStages) & 1, a.status);
            __syncwarp();
            ptx::tc_fence_after();
            if (ptx::elect_one()) R::multiply(tmem, ptx::smem_u32(smem), s, kb == kb0, empty, pair_mask);
        }
        if (ptx::elect_one()) ptx::pair_commit(acc_full, pair_mask);
    }
    __syncwarp();
    if (warp >= kEpiWarp0) {
        // the pair's MMAs have read every stage of both CTAs and written the accumulators
        ptx::mbar_wait(acc_full, 0, a.status);
        __syncwarp();
        ptx::tc_fence_after();
        const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        uint8_t* row = smem + (quad * 32 + lane) * kRowBytes;
#pragma unroll 1
        for (int c0 = half * kBn / 2; c0 < (half + 1) * kBn / 2; c0 += 32) {
            float v[32];
            __syncwarp();
            ptx::tmem_ld32(tmem + lane_base + c0, v);
#pragma unroll
            for (int c = 0; c < 32; c += 4)
                *reinterpret_cast<float4*>(row + (c0 + c) * 4) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
        }
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::pair_tmem_dealloc(tmem, kBn);
    }

    constexpr int kRows = 128 / kSplits;
    uint32_t peer[kSplits];
#pragma unroll
    for (int s = 0; s < kSplits; ++s) peer[s] = ptx::map_rank(ptx::smem_u32(smem), (uint32_t)(2 * s + rank));
    auto total = [&](int row, int col) {
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int s = 0; s < kSplits; ++s) add4(t, ptx::ld_cluster_f4(peer[s] + row * kRowBytes + col * 4));
        return t;
    };
    for (int k = warp; k < kRows; k += kThreads / 32) {
        const int row = split * kRows + k;
        const int64_t i = (int64_t)tl.i0 + 128 * rank + row;
        if (i >= a.I) break;
#pragma unroll
        for (int c0 = 0; c0 < R::kWidth; c0 += 128) {
            const int c = c0 + 4 * lane, j = tl.j0 + c;
            if (j >= a.J) continue;                    // J is a multiple of 8: four columns are in or out
            float4 v = total(row, c);
            if constexpr (kGated) {
                const float4 u = total(row, kBn / 2 + c);
                if (r.pre) {
                    store4(r.pre + i * 2 * a.J + j, v);
                    store4(r.pre + i * 2 * a.J + a.J + j, u);
                }
                v = act4(a.act, v);
                v = make_float4(v.x * u.x, v.y * u.y, v.z * u.z, v.w * u.w);
            } else {
                if (a.bias) add4(v, widen4(a.bias + j));
                if (r.pre) store4(r.pre + i * a.J + j, v);
                if (a.act) v = act4(a.act, v);
                if (r.residual) add4(v, widen4(r.residual + i * a.J + j));
            }
            store4(r.out + i * a.J + j, v);
        }
    }
    ptx::cluster_sync();                               // nobody leaves while its partial is read
}

// Clusters of `ctas` CTAs that run at once on the current device (0 on failure).
template <class Kernel>
int resident_clusters(Kernel kernel, int ctas, int threads, int smem) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
}

// early: the kernel may start while the one before it on the stream ends (griddep_wait)
template <class Kernel, class... Args>
int launch_clusters(Kernel kernel, int ctas, int64_t clusters, int threads, int smem, bool early, cudaStream_t stream,
                    const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas * clusters));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 2 : 1;
    cudaError_t err;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        err = cudaLaunchKernelEx(&cfg, kernel, args...);
    }
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "dense pair kernel");
}

template <bool kAMn, bool kBMn, bool kGated, int kBn>
int launch_pair_as(const CUtensorMap (&tm)[5], const PairArgs& a, cudaStream_t stream) {
    constexpr bool kEpilogue = !kBMn;             // the gradients have none
    constexpr int kAll = pair_threads(kEpilogue);
    auto kernel = dense_pair_kernel<kAMn, kBMn, kGated, kBn, kEpilogue>;
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> fit[64];
    const cudaError_t err = allow_smem(kernel, smem_bytes(kBn), done);
    if (err != cudaSuccess) return cuda_fail(err, "cudaFuncSetAttribute(dense pair kernel)");
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    int pairs = fit[dev & 63].load();
    if (!pairs) {
        pairs = resident_clusters(kernel, 2, kAll, smem_bytes(kBn));
        if (pairs < 1) return fail(DIFFUSER_ERR_CUDA, "no CTA pair of the dense product fits the device");
        fit[dev & 63].store(pairs);
    }
    const int64_t tiles = (int64_t)a.i_tiles * a.j_tiles;
    return launch_clusters(kernel, 2, tiles < pairs ? tiles : pairs, kAll, smem_bytes(kBn), kBMn, stream, tm[0], tm[1],
                           tm[2], tm[3], tm[4], a);
}

template <bool kAMn, bool kBMn, bool kGated, int kBn, int kSplits>
int launch_split_as(const CUtensorMap (&tm)[5], const PairArgs& a, const Results& r, cudaStream_t stream) {
    auto kernel = dense_pair_split_kernel<kAMn, kBMn, kGated, kBn, kSplits>;
    static std::atomic<uint64_t> done{0};
    constexpr int kSmem = 1024 + stage_count(kBn) * (kABytes + b_bytes(kBn)) + kBarBytes;
    const cudaError_t err = allow_smem(kernel, kSmem, done);
    if (err != cudaSuccess) return cuda_fail(err, "cudaFuncSetAttribute(dense pair split kernel)");
    return launch_clusters(kernel, 2 * kSplits, (int64_t)a.i_tiles * a.j_tiles, kThreads, kSmem, kBMn, stream, tm[0], tm[1],
                           a, r);
}

template <bool kAMn, bool kBMn, bool kGated, int kBn>
int launch_as(const CUtensorMap (&tm)[5], const PairArgs& a, const Results& r, int splits, cudaStream_t stream) {
    if (splits == 4) return launch_split_as<kAMn, kBMn, kGated, kBn, 4>(tm, a, r, stream);
    if (splits == 2) return launch_split_as<kAMn, kBMn, kGated, kBn, 2>(tm, a, r, stream);
    return launch_pair_as<kAMn, kBMn, kGated, kBn>(tm, a, stream);
}

}  // namespace

int dense_pair_clusters(int splits) {
    static std::atomic<int> fit[3][64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    std::atomic<int>& f = fit[splits >> 1][dev & 63];
    int n = f.load();
    if (!n) {
        constexpr int kSmem = 1024 + stage_count(256) * (kABytes + b_bytes(256)) + kBarBytes;
        if (splits == 4) {
            static std::atomic<uint64_t> done{0};
            auto kernel = dense_pair_split_kernel<false, false, false, 256, 4>;
            if (allow_smem(kernel, kSmem, done) == cudaSuccess) n = resident_clusters(kernel, 8, kThreads, kSmem);
        } else if (splits == 2) {
            static std::atomic<uint64_t> done{0};
            auto kernel = dense_pair_split_kernel<false, false, false, 256, 2>;
            if (allow_smem(kernel, kSmem, done) == cudaSuccess) n = resident_clusters(kernel, 4, kThreads, kSmem);
        } else {
            static std::atomic<uint64_t> done{0};
            auto kernel = dense_pair_kernel<false, false, false, 256, true>;
            if (allow_smem(kernel, smem_bytes(256), done) == cudaSuccess) n = resident_clusters(kernel, 2, pair_threads(true), smem_bytes(256));
        }
        if (n < 1) n = 1;
        f.store(n);
    }
    return n;
}

namespace {

// extents, K steps and tiles of a product; OVERFLOW where tile indexes would not fit
int plan_pair(DenseForm form, const DenseArgs& d, int bn, PairArgs* a) {
    const bool gated = form == kForward && d.gated;
    int64_t I, J, K;
    if (form == kForward) { I = d.rows; J = gated ? d.cols / 2 : d.cols; K = d.inner; }
    else if (form == kInputGrad) { I = d.rows; J = d.inner; K = d.cols; }
    else { I = d.cols; J = d.inner; K = d.rows; }
    const int width = gated ? bn / 2 : bn;
    const int64_t it = (I + kTI - 1) / kTI, jt = (J + width - 1) / width;
    if (it * jt > INT32_MAX / 8) return fail(DIFFUSER_ERR_OVERFLOW, "dense product too large");
    *a = PairArgs{};
    a->I = (int32_t)I;
    a->J = (int32_t)J;
    a->k_blocks = (int32_t)((K + kTK - 1) / kTK);
    a->i_tiles = (int32_t)it;
    a->j_tiles = (int32_t)jt;
    a->status = d.status;
    return DIFFUSER_OK;
}

// the operands' maps
int map_operands(DenseForm form, const DenseArgs& d, int bn, CUtensorMap* A, CUtensorMap* B) {
    int st;
    if (form == kWeightGrad) st = map_matrix(A, d.a, d.cols, d.rows, 64, kTK);
    else st = map_matrix(A, d.a, form == kForward ? d.inner : d.cols, d.rows, kTK, 128);
    if (st) return st;
    if (form == kForward) {
        return d.gated ? map_halves(B, d.b, d.inner, d.cols / 2, kTK, 128, 1)
                       : map_matrix(B, d.b, d.inner, d.cols, kTK, bn / 2);
    }
    return map_matrix(B, d.b, d.inner, form == kInputGrad ? d.cols : d.rows, 64, kTK);
}

// Deals `longs` tiles of `long_steps` and `shorts` of `short_steps` to the pairs; returns the
// largest load in steps.
int64_t deal_tiles(int64_t longs, int64_t long_steps, int64_t shorts, int64_t short_steps, int pairs, GradDeal* d) {
    d->longs = (int32_t)(longs / pairs);
    d->a_pairs = (int32_t)(longs % pairs);
    const int64_t na = d->a_pairs, nb = pairs - na;
    const int64_t load_b = d->longs * long_steps, load_a = load_b + long_steps;
    // short tiles go to the least loaded: first the b pairs, up to the a pairs' load, then all evenly
    int64_t b = (long_steps + short_steps - 1) / short_steps, to_b = na ? nb * b : 0;
    if (!na) {
        to_b = shorts;
    } else if (to_b >= shorts) {
        to_b = shorts;
    } else {
        const int64_t rest = shorts - to_b;
        to_b += rest / pairs * nb;
        // the last, incomplete round: the b pairs when they stand lower, else the a pairs first
        const int64_t last = rest % pairs, level_b = load_b + b * short_steps;
        const int64_t first = level_b <= load_a ? nb : na;
        const int64_t to_first = last < first ? last : first;
        to_b += level_b <= load_a ? to_first : last - to_first;
    }
    const int64_t to_a = shorts - to_b;
    d->b_shorts = (int32_t)(to_b / nb);
    d->b_rest = (int32_t)(to_b % nb);
    d->a_shorts = na ? (int32_t)(to_a / na) : 0;
    d->a_rest = na ? (int32_t)(to_a % na) : 0;
    const int64_t most_b = load_b + (d->b_shorts + (d->b_rest ? 1 : 0)) * short_steps;
    const int64_t most_a = na ? load_a + (d->a_shorts + (d->a_rest ? 1 : 0)) * short_steps : 0;
    return most_a > most_b ? most_a : most_b;
}

GradDeal deal_grads(const PairArgs& x, const PairArgs& w, int pairs, int64_t* most) {
    GradDeal d{};
    const int64_t tx = (int64_t)x.i_tiles * x.j_tiles, tw = (int64_t)w.i_tiles * w.j_tiles;
    d.longer = w.k_blocks >= x.k_blocks;
    *most = d.longer ? deal_tiles(tw, w.k_blocks, tx, x.k_blocks, pairs, &d)
                     : deal_tiles(tx, x.k_blocks, tw, w.k_blocks, pairs, &d);
    return d;
}

template <int kBn>
int launch_grads_as(const CUtensorMap (&tm)[6], GradArgs g, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    auto kernel = dense_grads_kernel<kBn>;
    const cudaError_t err = allow_smem(kernel, smem_bytes(kBn), done);
    if (err != cudaSuccess) return cuda_fail(err, "cudaFuncSetAttribute(dense gradients kernel)");
    const int64_t tiles =
        (int64_t)g.p[0].i_tiles * g.p[0].j_tiles + (int64_t)g.p[1].i_tiles * g.p[1].j_tiles;
    int64_t pairs = dense_pair_clusters(1), most = 0;
    if (tiles < pairs) pairs = tiles;
    g.deal = deal_grads(g.p[0], g.p[1], (int)pairs, &most);
    return launch_clusters(kernel, 2, pairs, pair_threads(false), smem_bytes(kBn), true, stream, tm[0], tm[1], tm[2],
                           tm[3], tm[4], tm[5], g);
}

}  // namespace

int64_t dense_grads_steps(const DenseArgs& x, int bn) {
    PairArgs px, pw;
    if (plan_pair(kInputGrad, x, bn, &px) || plan_pair(kWeightGrad, x, bn, &pw)) return INT64_MAX;
    int64_t most = 0;
    deal_grads(px, pw, dense_pair_clusters(1), &most);
    return most;
}

int launch_dense_grads(const DenseArgs& x, const DenseArgs& w, const BiasSums& bias, int bn, cudaStream_t stream) {
    GradArgs g{};
    g.bias = bias;
    CUtensorMap tm[6] = {};                        // dX: A, B, result; dW: A, B, result
    int st = plan_pair(kInputGrad, x, bn, &g.p[0]);
    if (!st) st = plan_pair(kWeightGrad, w, bn, &g.p[1]);
    if (!st) st = map_operands(kInputGrad, x, bn, &tm[0], &tm[1]);
    if (!st) st = map_matrix(&tm[2], x.out, g.p[0].J, g.p[0].I, kBlock, 32);
    if (!st) st = map_operands(kWeightGrad, w, bn, &tm[3], &tm[4]);
    if (!st) st = map_matrix(&tm[5], w.out, g.p[1].J, g.p[1].I, kBlock, 32);
    if (st) return st;
    return bn == 256 ? launch_grads_as<256>(tm, g, stream) : launch_grads_as<128>(tm, g, stream);
}

int launch_dense_pair(DenseForm form, const DenseArgs& d, int bn, int splits, cudaStream_t stream) {
    const bool gated = form == kForward && d.gated;
    PairArgs a;
    int st = plan_pair(form, d, bn, &a);
    if (st) return st;
    while (splits > a.k_blocks) splits /= 2;       // every pair has a K step
    a.act = d.act;
    a.pre = d.pre != nullptr;
    a.residual = d.residual != nullptr;
    a.bias = static_cast<const __nv_bfloat16*>(d.bias);
    const Results r{static_cast<__nv_bfloat16*>(d.out), static_cast<__nv_bfloat16*>(d.pre),
                    static_cast<const __nv_bfloat16*>(d.residual)};
    CUtensorMap tm[5] = {};                        // A, B, result, pre, residual
    st = map_operands(form, d, bn, &tm[0], &tm[1]);
    if (splits == 1) {
        if (!st) st = map_matrix(&tm[2], d.out, a.J, a.I, kBlock, 32);
        if (!st && a.pre)
            st = gated ? map_column_halves(&tm[3], d.pre, a.J, a.I, kBlock, 32) : map_matrix(&tm[3], d.pre, a.J, a.I, kBlock, 32);
        if (!st && a.residual) st = map_matrix(&tm[4], d.residual, a.J, a.I, kBlock, 32);
    }
    if (st) return st;
    if (gated) return launch_as<false, false, true, 256>(tm, a, r, splits, stream);
    if (form == kForward)
        return bn == 256 ? launch_as<false, false, false, 256>(tm, a, r, splits, stream)
                         : launch_as<false, false, false, 128>(tm, a, r, splits, stream);
    if (form == kInputGrad)
        return bn == 256 ? launch_as<false, true, false, 256>(tm, a, r, splits, stream)
                         : launch_as<false, true, false, 128>(tm, a, r, splits, stream);
    return bn == 256 ? launch_as<true, true, false, 256>(tm, a, r, splits, stream)
                     : launch_as<true, true, false, 128>(tm, a, r, splits, stream);
}

}  // namespace dfs
