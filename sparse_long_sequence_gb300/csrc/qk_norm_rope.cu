// Per-head root-mean-square norms of queries and keys with the position rotation
// in the same pass, forward and backward.
//
// A row x of 64 features (one token of one head) gives
//   y = R(p) (r x w),  r = (mean x^2 + eps)^-1/2,
// R(p) turning feature pair i by the angle p theta^(-2i/rot).  Backward, for
// dy: g = R(-p) dy, dn = g w, xh = r x:
//   dx = r (dn - xh mean(dn xh)),  dw = sum over rows of g xh.
//
// Eight lanes hold a row (8 features each, one or two 16-byte loads), a warp four
// consecutive tokens of a head, and goes on over heads with the tokens' cosines
// and sines kept in registers: they depend on the token alone.  The angle is
// exact integer arithmetic: theta^(-2i/rot) / (2 pi), in units of 2^-64 turns,
// times the position modulo 2^64 leaves the fraction of a turn, so far positions
// lose nothing (a float product would be off by p 2^-24 radians).
// Bound by HBM: every row is read and written once (backward: two reads).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "layer_ops.h"
#include "sm100_ptx.cuh"

namespace dfs {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowLanes = 8;                 // lanes of a row
constexpr int kPer = kHeadDim / kRowLanes;   // features of a lane
constexpr int kTok = 32 / kRowLanes;         // tokens of a warp
constexpr unsigned kFull = 0xffffffffu;

template <class T> struct Io;
template <> struct Io<float> {
    struct Raw { float4 a, b; };
    static __device__ __forceinline__ Raw load(const float* p) {
        return {*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4)};
    }
    static __device__ __forceinline__ void widen(const Raw& r, float (&v)[kPer]) {
        v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
        v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&v)[kPer]) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
    static __device__ __forceinline__ float round(float x) { return x; }
};
template <> struct Io<__nv_bfloat16> {
    using Raw = uint4;
    static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) {
        return *reinterpret_cast<const uint4*>(p);
    }
    static __device__ __forceinline__ void widen(const Raw& r, float (&v)[kPer]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[kPer]) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ __nv_bfloat16 round(float x) { return __float2bfloat16_rn(x); }
};

// Sum over the 8 lanes of a row.
__device__ __forceinline__ float row_sum(float s) {
    s += __shfl_xor_sync(kFull, s, 1);
    s += __shfl_xor_sync(kFull, s, 2);
    s += __shfl_xor_sync(kFull, s, 4);
    return s;
}

// Cosines and sines of a lane's 8 features; a feature's turned value is
// x cos + partner sin (the sine negated for the first of a pair; 1 and 0 past rot).
template <bool kInterleaved>
struct Turn {
    float c[kInterleaved ? kPer / 2 : kPer], s[kInterleaved ? kPer / 2 : kPer];
    int src;                                 // split halves: lane that holds the partners

    __device__ __forceinline__ void set(const uint64_t* freq, int rot, int64_t pos, int lane) {
        const int t = lane & (kRowLanes - 1);
        const bool turned = t * kPer < rot;
        const int half = rot / (2 * kPer);   // lanes of a half
        const bool second = t >= half;
        src = turned ? (second ? lane - half : lane + half) : lane;
        constexpr int count = kInterleaved ? kPer / 2 : kPer;
        const int i0 = kInterleaved ? t * (kPer / 2) : (second ? t - half : t) * kPer;
#pragma unroll
        for (int j = 0; j < count; ++j) {
            c[j] = 1.f;
            s[j] = 0.f;
            if (turned) {
                // the fraction of a turn, in [-1/2, 1/2), times 2: sincospi's unit
                const uint64_t phase = (uint64_t)pos * freq[i0 + j];
                const float halfturns = (float)(int32_t)(phase >> 32) * 4.656612873077393e-10f;   // 2^-31
                sincospif(halfturns, &s[j], &c[j]);
                if (!kInterleaved && !second) s[j] = -s[j];
            }
        }
    }
    // kSign +1: R(p), -1: R(-p)
    template <int kSign>
    __device__ __forceinline__ void apply(float (&v)[kPer]) const {
        if constexpr (kInterleaved) {
#pragma unroll
            for (int j = 0; j < kPer / 2; ++j) {
                const float a = v[2 * j], b = v[2 * j + 1], sn = kSign * s[j];
                v[2 * j] = a * c[j] - b * sn;
                v[2 * j + 1] = a * sn + b * c[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const float other = __shfl_sync(kFull, v[j], src);
                v[j] = v[j] * c[j] + other * (kSign * s[j]);
            }
        }
    }
};

template <class T>
__device__ __forceinline__ void load_weight(const void* w, int lane, float (&v)[kPer]) {
    if (w) {
        Io<T>::widen(Io<T>::load(static_cast<const T*>(w) + (lane & (kRowLanes - 1)) * kPer), v);
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = 1.f;
    }
}

// A warp's share: 4 tokens and a run of heads.  Heads 0 .. Hq-1 are the queries',
// Hq .. Hq+Hk-1 the keys'.
struct Share {
    int64_t token;                 // this lane's (clamped to the last: loads stay in bounds)
    bool live;                     // the lane's token exists
    int64_t b, i;
    int h0, h1;
};
__device__ __forceinline__ Share share_of(const QkArgs& a, int64_t unit, int64_t groups, int per_warp, int lane) {
    Share s;
    const int64_t group = unit % groups;
    s.h0 = (int)(unit / groups) * per_warp;
    s.h1 = min(s.h0 + per_warp, a.Hq + a.Hk);
    s.token = group * kTok + lane / kRowLanes;
    s.live = s.token < a.tokens;
    if (!s.live) s.token = a.tokens - 1;
    s.b = s.token / a.n;
    s.i = s.token - s.b * a.n;
    return s;
}
// offset of this lane's features of head h in its own tensor
__device__ __forceinline__ int64_t offset_of(const QkArgs& a, const Share& s, int h, int lane) {
    const bool key = h >= a.Hq;
    const int64_t heads = key ? a.Hk : a.Hq;
    return ((s.b * heads + (key ? h - a.Hq : h)) * a.n + s.i) * kHeadDim + (lane & (kRowLanes - 1)) * kPer;
}

constexpr int kAhead = 4;          // heads whose loads are in flight together

template <class T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) qk_forward_kernel(const __grid_constant__ QkArgs a, int64_t groups,
                                                              int per_warp, int64_t units) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= units) return;
    const Share s = share_of(a, unit, groups, per_warp, lane);
    Turn<kInterleaved> turn;
    turn.set(a.freq, a.rot, a.pos0 + (a.pos ? a.pos[s.token] : s.i), lane);
    float wq[kPer], wk[kPer];
    load_weight<T>(a.wq, lane, wq);
    load_weight<T>(a.wk, lane, wk);
    for (int h = s.h0; h < s.h1; h += kAhead) {
        typename Io<T>::Raw raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (h + u < s.h1)
                raw[u] = Io<T>::load(static_cast<const T*>(h + u >= a.Hq ? a.k : a.q) + offset_of(a, s, h + u, lane));
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (h + u >= s.h1) break;
            const bool key = h + u >= a.Hq;
            float v[kPer];
            Io<T>::widen(raw[u], v);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) ss = fmaf(v[j], v[j], ss);
            const float r = rsqrtf(row_sum(ss) * (1.f / kHeadDim) + a.eps);
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] = v[j] * r * (key ? wk[j] : wq[j]);
            turn.template apply<1>(v);
            if (s.live) Io<T>::store(static_cast<T*>(key ? a.ko : a.qo) + offset_of(a, s, h + u, lane), v);
        }
    }
}

template <class T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) qk_backward_kernel(const __grid_constant__ QkArgs a, int64_t groups,
                                                               int per_warp, int64_t units) {
    __shared__ float sums[kWarps][2 * kHeadDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float wq[kPer], wk[kPer], gq[kPer], gk[kPer];
    load_weight<T>(a.wq, lane, wq);
    load_weight<T>(a.wk, lane, wk);
#pragma unroll
    for (int j = 0; j < kPer; ++j) gq[j] = gk[j] = 0.f;
    for (int64_t unit = (int64_t)blockIdx.x * kWarps + warp; unit < units; unit += (int64_t)gridDim.x * kWarps) {
        const Share s = share_of(a, unit, groups, per_warp, lane);
        Turn<kInterleaved> turn;
        turn.set(a.freq, a.rot, a.pos0 + (a.pos ? a.pos[s.token] : s.i), lane);
        for (int h = s.h0; h < s.h1; ++h) {
            const bool key = h >= a.Hq;
            const int64_t at = offset_of(a, s, h, lane);
            float x[kPer], g[kPer];
            const auto rx = Io<T>::load(static_cast<const T*>(key ? a.k : a.q) + at);
            const auto rg = Io<T>::load(static_cast<const T*>(key ? a.dko : a.dqo) + at);
            Io<T>::widen(rx, x);
            Io<T>::widen(rg, g);
            turn.template apply<-1>(g);
            float ss = 0.f, sd = 0.f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                ss = fmaf(x[j], x[j], ss);
                sd = fmaf(g[j] * (key ? wk[j] : wq[j]), x[j], sd);
            }
            const float r = rsqrtf(row_sum(ss) * (1.f / kHeadDim) + a.eps);
            const float m = row_sum(sd) * (r * (1.f / kHeadDim));      // mean(dn xh)
            float d[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const float xh = x[j] * r;
                d[j] = r * (g[j] * (key ? wk[j] : wq[j]) - xh * m);
                const float add = s.live ? g[j] * xh : 0.f;
                if (key) gk[j] += add; else gq[j] += add;
            }
            if (s.live) Io<T>::store(static_cast<T*>(key ? a.ko : a.qo) + at, d);
        }
    }
    if (!a.partial) return;
    // lanes of the four tokens, then the warps, in a fixed order
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        gq[j] += __shfl_xor_sync(kFull, gq[j], 8);
        gk[j] += __shfl_xor_sync(kFull, gk[j], 8);
        gq[j] += __shfl_xor_sync(kFull, gq[j], 16);
        gk[j] += __shfl_xor_sync(kFull, gk[j], 16);
        if (lane < kRowLanes) {
            sums[warp][lane * kPer + j] = gq[j];
            sums[warp][kHeadDim + lane * kPer + j] = gk[j];
        }
    }
    __syncthreads();
    if (threadIdx.x < 2 * kHeadDim) {
        float t = 0.f;
        for (int w = 0; w < kWarps; ++w) t += sums[w][threadIdx.x];
        a.partial[(int64_t)blockIdx.x * 2 * kHeadDim + threadIdx.x] = t;
    }
}

// dw = the sum of the blocks' partial sums: 8 groups of threads take every eighth
// block, then their sums are added in order.
constexpr int kFinishGroups = 8;
template <class T>
__global__ void __launch_bounds__(2 * kHeadDim * kFinishGroups)
qk_weight_kernel(const float* partial, int64_t blocks, T* dwq, T* dwk) {
    __shared__ float sums[kFinishGroups][2 * kHeadDim];
    const int c = threadIdx.x % (2 * kHeadDim), grp = threadIdx.x / (2 * kHeadDim);
    float t = 0.f;
    for (int64_t b = grp; b < blocks; b += kFinishGroups) t += partial[b * 2 * kHeadDim + c];
    sums[grp][c] = t;
    __syncthreads();
    if (grp) return;
    t = 0.f;
    for (int k = 0; k < kFinishGroups; ++k) t += sums[k][c];
    T* dst = c < kHeadDim ? dwq : dwk;
    if (dst) dst[c % kHeadDim] = Io<T>::round(t);
}

constexpr int64_t kManyWarps = 152 * 48;     // warps that fill the GPU

// heads a warp takes in a row: all of them where the tokens alone make enough warps,
// fewer (down to one) where they do not
int heads_per_warp(int64_t groups, int64_t heads) {
    const int64_t runs = (kManyWarps + groups - 1) / groups;
    const int64_t per = (heads + runs - 1) / runs;
    return (int)(per < 1 ? 1 : per);
}

template <class T>
int forward_as(const QkArgs& a, bool interleaved, cudaStream_t stream) {
    const int64_t groups = (a.tokens + kTok - 1) / kTok, heads = (int64_t)a.Hq + a.Hk;
    const int per = heads_per_warp(groups, heads);
    const int64_t units = groups * ((heads + per - 1) / per);
    const int64_t blocks = (units + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many rows");
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        if (interleaved)
            qk_forward_kernel<T, true><<<(unsigned)blocks, kThreads, 0, stream>>>(a, groups, per, units);
        else
            qk_forward_kernel<T, false><<<(unsigned)blocks, kThreads, 0, stream>>>(a, groups, per, units);
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "qk_forward_kernel");
}

template <class T>
int backward_as(const QkArgs& a, bool interleaved, void* dwq, void* dwk, cudaStream_t stream) {
    const int64_t groups = (a.tokens + kTok - 1) / kTok, heads = (int64_t)a.Hq + a.Hk;
    const int per = heads_per_warp(groups, heads);
    const int64_t units = groups * ((heads + per - 1) / per);
    const int64_t blocks = qk_backward_blocks(a.tokens, heads);
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        if (interleaved)
            qk_backward_kernel<T, true><<<(unsigned)blocks, kThreads, 0, stream>>>(a, groups, per, units);
        else
            qk_backward_kernel<T, false><<<(unsigned)blocks, kThreads, 0, stream>>>(a, groups, per, units);
    }
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return cuda_fail(err, "qk_backward_kernel");
    if (!dwq && !dwk) return DIFFUSER_OK;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        qk_weight_kernel<T><<<1, 2 * kHeadDim * kFinishGroups, 0, stream>>>(a.partial, blocks, static_cast<T*>(dwq),
                                                                           static_cast<T*>(dwk));
    }
    err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "qk_weight_kernel");
}

}  // namespace

// at most four blocks on each of 152 SMs: each block leaves one row of partial sums
int64_t qk_backward_blocks(int64_t tokens, int64_t heads) {
    const int64_t groups = (tokens + kTok - 1) / kTok;
    const int per = heads_per_warp(groups, heads);
    const int64_t units = groups * ((heads + per - 1) / per);
    const int64_t blocks = (units + kWarps - 1) / kWarps;
    return blocks < 152 * 4 ? blocks : 152 * 4;
}

int launch_qk_norm_rope(const QkArgs& a, int32_t dtype, bool interleaved, cudaStream_t stream) {
    return dtype == DIFFUSER_DTYPE_BF16 ? forward_as<__nv_bfloat16>(a, interleaved, stream)
                                        : forward_as<float>(a, interleaved, stream);
}

int launch_qk_norm_rope_backward(const QkArgs& a, int32_t dtype, bool interleaved, void* dwq, void* dwk,
                                 cudaStream_t stream) {
    return dtype == DIFFUSER_DTYPE_BF16 ? backward_as<__nv_bfloat16>(a, interleaved, dwq, dwk, stream)
                                        : backward_as<float>(a, interleaved, dwq, dwk, stream);
}

}  // namespace dfs
