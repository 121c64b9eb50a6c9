// Per-head root-mean-square norms of queries and keys with the position rotation
// in the same pass, forward and backward.
//
// A row x of 64 features (one token of one head) gives
//   y = R(p) (r x w),  r = (mean x^2 + eps)^-1/2,
// R(p) turning feature pair i by the angle p theta^(-2i/rot).  Backward, for
// dy: g = R(-p) dy, dn = g w, xh = r x:
//   dx = r (dn - xh mean(dn xh)),  dw = sum over rows of g xh.
//
// Eight lanes hold a row, a warp four consecutive tokens of a head, and goes on over a run of
// the queries' or the keys' heads with the tokens' cosines and sines kept in registers: they
// depend on the token alone.  A lane holds two pieces of four features, chosen so that it has
// both features of each of its pairs (split halves: pieces t and t + rot / 8): the rotation
// needs no exchange between lanes.  Arithmetic on packed pairs of fp32 (f32x2).
// The angle is integer arithmetic modulo a turn: |p| times theta^(-2i/rot) / (2 pi), a 128-bit
// fraction (turns.h), of which positions below 2^32 need the upper half alone.  Its upper 32 bits
// are used: within 2^-31 turns for any 64-bit position (with a 64-bit fraction throughout the
// worst pair was off by 1e-4 radians at 2^48, a float product would be by p 2^-24).  Both halves
// for all positions cost 1 us of 10 at 2 x 24 heads x 4096 tokens; taking whole quarter turns off
// before the rounding to fp32 costs 0.2 and keeps the plain fp32 form's accuracy (6.2e-8 in the
// 2-norm; 6.8e-8 with the whole fraction rounded).
// Bound by HBM: every row is read and written once (backward: two reads).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "layer_ops.h"
#include "packed.cuh"
#include "sm100_ptx.cuh"

namespace dfs {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRowLanes = 8;                 // lanes of a row
constexpr int kTok = 32 / kRowLanes;         // tokens of a warp
constexpr unsigned kFull = 0xffffffffu;
using namespace packed;

// A lane's eight features of a row: piece A in v[0], v[1], piece B in v[2], v[3].
template <class T> struct Io;
template <> struct Io<float> {
    struct Raw { float4 a, b; };
    static __device__ __forceinline__ Raw load(const float* row, int oa, int ob) {
        return {*reinterpret_cast<const float4*>(row + oa), *reinterpret_cast<const float4*>(row + ob)};
    }
    static __device__ __forceinline__ void widen(const Raw& r, F2 (&v)[4]) {
        v[0] = f2(r.a.x, r.a.y); v[1] = f2(r.a.z, r.a.w);
        v[2] = f2(r.b.x, r.b.y); v[3] = f2(r.b.z, r.b.w);
    }
    static __device__ __forceinline__ Raw narrow(const F2 (&v)[4]) {
        const float2 p = un(v[0]), q = un(v[1]), s = un(v[2]), t = un(v[3]);
        return {make_float4(p.x, p.y, q.x, q.y), make_float4(s.x, s.y, t.x, t.y)};
    }
    // the values of v, or those of `kept`
    static __device__ __forceinline__ Raw either(bool first, const F2 (&v)[4], const F2 (&kept)[4]) {
        F2 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = first ? v[j] : kept[j];
        return narrow(w);
    }
    static __device__ __forceinline__ void store(float* row, int oa, int ob, const Raw& r) {
        *reinterpret_cast<float4*>(row + oa) = r.a;
        *reinterpret_cast<float4*>(row + ob) = r.b;
    }
    static __device__ __forceinline__ float round(float x) { return x; }
};
template <> struct Io<__nv_bfloat16> {
    struct Raw { uint2 a, b; };
    static __device__ __forceinline__ Raw load(const __nv_bfloat16* row, int oa, int ob) {
        return {*reinterpret_cast<const uint2*>(row + oa), *reinterpret_cast<const uint2*>(row + ob)};
    }
    static __device__ __forceinline__ F2 two(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
    static __device__ __forceinline__ void widen(const Raw& r, F2 (&v)[4]) {
        v[0] = two(r.a.x); v[1] = two(r.a.y); v[2] = two(r.b.x); v[3] = two(r.b.y);
    }
    static __device__ __forceinline__ uint32_t pack(F2 v) {
        const float2 f = un(v);
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ Raw narrow(const F2 (&v)[4]) {
        return {make_uint2(pack(v[0]), pack(v[1])), make_uint2(pack(v[2]), pack(v[3]))};
    }
    // the values of v rounded, or those of `kept`, which are as they were loaded (the loaded words themselves, kept
    // beside the next ones: 25 us for 20 on the long case)
    static __device__ __forceinline__ Raw either(bool first, const F2 (&v)[4], const F2 (&kept)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = un(kept[j]);
            w[j] = first ? pack(v[j]) : __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
        }
        return {make_uint2(w[0], w[1]), make_uint2(w[2], w[3])};
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* row, int oa, int ob, const Raw& r) {
        *reinterpret_cast<uint2*>(row + oa) = r.a;
        *reinterpret_cast<uint2*>(row + ob) = r.b;
    }
    static __device__ __forceinline__ __nv_bfloat16 round(float x) { return __float2bfloat16_rn(x); }
};

// Sum of a row's 64 products x y (8 lanes).
__device__ __forceinline__ float row_dot(const F2 (&x)[4], const F2 (&y)[4]) {
    F2 s = mul(x[0], y[0]);
#pragma unroll
    for (int j = 1; j < 4; ++j) s = fma(x[j], y[j], s);
    const float2 p = un(s);
    float t = p.x + p.y;
    t += __shfl_xor_sync(kFull, t, 1);
    t += __shfl_xor_sync(kFull, t, 2);
    t += __shfl_xor_sync(kFull, t, 4);
    return t;
}

// Offsets of a lane's two pieces in a row.  Split halves: pieces t and t + P of the P = rot / 8
// pairs of pieces, then the pieces that are not turned, two a lane.  Neighbouring pairs: 2t, 2t + 1.
template <bool kInterleaved>
__device__ __forceinline__ void pieces(int rot, int lane, int* oa, int* ob) {
    const int t = lane & (kRowLanes - 1), P = rot / 8;
    if (kInterleaved || t >= P) {
        *oa = (kInterleaved ? 2 * t : 2 * P + 2 * (t - P)) * 4;
        *ob = *oa + 4;
    } else {
        *oa = 4 * t;
        *ob = 4 * (t + P);
    }
}

// Cosines and sines of a lane's four pairs (1 and 0 past rot), sin negated for the inverse.
// Split halves: pair j is (A[j], B[j]); neighbouring: (v[j].x, v[j].y).
template <bool kInterleaved>
struct Turn {
    F2 c[kInterleaved ? 4 : 2], s[kInterleaved ? 4 : 2];

    template <int kSign>
    __device__ __forceinline__ void set(const QkArgs& a, int64_t pos, int lane) {
        const int t = lane & (kRowLanes - 1);
        const bool turned = t < a.rot / 8;
        const uint64_t far = pos < 0 ? 0 - (uint64_t)pos : (uint64_t)pos;
        uint32_t phase[4] = {0, 0, 0, 0};        // |pos| turns modulo one, in units of 2^-32
        if (turned) {
            if (far >> 32) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    phase[j] = (uint32_t)((far * a.freq[4 * t + j] + __umul64hi(far, a.freq_low[4 * t + j])) >> 32);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) phase[j] = (uint32_t)(far * a.freq[4 * t + j] >> 32);
            }
        }
        const uint32_t back = (pos < 0) == (kSign < 0) ? 0u : 0x80000000u;       // the sine's sign
        float cs[4], sn[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            cs[j] = 1.f;
            sn[j] = 0.f;
            if (!turned) continue;
            // whole quarter turns come off as integers: what is left, at most an eighth, loses 2^-28
            // turns as fp32, and nothing near a quarter turn, where a sine or cosine is small
            const uint32_t quarter = (phase[j] + (1u << 29)) >> 30;
            float sr, cr;
            sincospif((float)(int32_t)(phase[j] - (quarter << 30)) * 4.656612873077393e-10f, &sr, &cr);   // 2^-31
            const bool odd = quarter & 1;
            cs[j] = __uint_as_float(__float_as_uint(odd ? sr : cr) ^ ((quarter + 1) & 2) << 30);
            sn[j] = __uint_as_float(__float_as_uint(odd ? cr : sr) ^ (quarter & 2) << 30 ^ back);
        }
        if constexpr (kInterleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c[j] = both(cs[j]);
                s[j] = f2(-sn[j], sn[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                c[j] = f2(cs[2 * j], cs[2 * j + 1]);
                s[j] = f2(sn[2 * j], sn[2 * j + 1]);
            }
        }
    }
    __device__ __forceinline__ void scale(float x) {
#pragma unroll
        for (int j = 0; j < (kInterleaved ? 4 : 2); ++j) {
            c[j] = mul(c[j], both(x));
            s[j] = mul(s[j], both(x));
        }
    }
    // (a, b) -> (a cos - b sin, a sin + b cos)
    __device__ __forceinline__ void apply(F2 (&v)[4]) const {
        if constexpr (kInterleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 p = un(v[j]);
                v[j] = fma(v[j], c[j], mul(f2(p.y, p.x), s[j]));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const F2 a = v[j], b = v[2 + j];
                const float2 n = un(s[j]);
                v[j] = fma(a, c[j], mul(b, f2(-n.x, -n.y)));
                v[2 + j] = fma(a, s[j], mul(b, c[j]));
            }
        }
    }
};

template <class T>
__device__ __forceinline__ void load_weight(const T* w, int oa, int ob, F2 (&v)[4]) {
    if (w) {
        Io<T>::widen(Io<T>::load(w, oa, ob), v);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = both(1.f);
    }
}

// A warp's share (a unit): four tokens and a run of the queries' or of the keys' heads.  All of
// the queries' units come first.
struct Work {
    int64_t groups;                // of four tokens
    int64_t q_units, k_units;      // groups x runs
    int32_t per;                   // heads of a run
    int32_t q_blocks, k_blocks;    // backward: blocks that take the queries' units, and the keys'
};
struct Share {
    bool live;                     // this lane's token exists
    int h0, h1;
    int64_t first;                 // offset of (h0, token) in its tensor
    int64_t pos;
};
// unit `unit` of the queries or (key) of the keys
__device__ __forceinline__ Share share_of(const QkArgs& a, const Work& w, bool key, int64_t unit, int lane) {
    Share s;
    const int64_t group = unit % w.groups;
    const int heads = key ? a.Hk : a.Hq;
    s.h0 = (int)(unit / w.groups) * w.per;
    s.h1 = min(s.h0 + w.per, heads);
    int64_t token = group * kTok + lane / kRowLanes;
    s.live = token < a.tokens;
    if (!s.live) token = a.tokens - 1;        // (loads stay in bounds)
    const int64_t b = token / a.n, i = token - b * a.n;
    s.first = ((b * heads + s.h0) * a.n + i) * kHeadDim;
    s.pos = (int64_t)((uint64_t)a.pos0 + (uint64_t)(a.pos ? a.pos[token] : i));
    return s;
}

constexpr int kAhead = 4;          // heads whose loads are in flight together

template <class T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) qk_forward_kernel(const __grid_constant__ QkArgs a, const Work w) {
    const int lane = threadIdx.x & 31;
    int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= w.q_units + w.k_units) return;
    const bool key = unit >= w.q_units;
    if (key) unit -= w.q_units;
    const Share s = share_of(a, w, key, unit, lane);
    int oa, ob;
    pieces<kInterleaved>(a.rot, lane, &oa, &ob);
    const int64_t step = a.n * kHeadDim;      // from head to head
    const T* src = static_cast<const T*>(key ? a.k : a.q) + s.first;
    T* dst = static_cast<T*>(key ? a.ko : a.qo) + s.first;
    typename Io<T>::Raw raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (s.h0 + u < s.h1) raw[u] = Io<T>::load(src + u * step, oa, ob);
    Turn<kInterleaved> turn;
    turn.template set<1>(a, s.pos, lane);
    F2 wt[4];
    load_weight(static_cast<const T*>(key ? a.wk : a.wq), oa, ob, wt);
    for (int h = s.h0; h < s.h1; h += kAhead, src += kAhead * step, dst += kAhead * step) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (h + u >= s.h1) break;
            F2 v[4];
            Io<T>::widen(raw[u], v);
            if (h + u + kAhead < s.h1) raw[u] = Io<T>::load(src + (u + kAhead) * step, oa, ob);
            const F2 r = both(rsqrtf(row_dot(v, v) * (1.f / kHeadDim) + a.eps));
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = mul(mul(v[j], r), wt[j]);
            turn.apply(v);
            if (s.live) Io<T>::store(dst + u * step, oa, ob, Io<T>::narrow(v));
        }
    }
}

// heads whose loads are in flight together in the backward: what 128 registers hold
constexpr int back_ahead(size_t element) { return element == 2 ? 4 : 2; }

// A block takes units of the queries or of the keys alone, so that one weight and one sum of its
// gradient are held.
template <class T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) qk_backward_kernel(const __grid_constant__ QkArgs a, const Work w) {
    constexpr int kAheadBack = back_ahead(sizeof(T));
    __shared__ float sums[kWarps][kHeadDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool key = (int)blockIdx.x >= w.q_blocks;
    const int block = key ? (int)blockIdx.x - w.q_blocks : (int)blockIdx.x, blocks = key ? w.k_blocks : w.q_blocks;
    const int64_t units = key ? w.k_units : w.q_units, step = a.n * kHeadDim;
    int oa, ob;
    pieces<kInterleaved>(a.rot, lane, &oa, &ob);
    F2 wt[4], acc[4];
    load_weight(static_cast<const T*>(key ? a.wk : a.wq), oa, ob, wt);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = both(0.f);
    for (int64_t unit = (int64_t)block * kWarps + warp; unit < units; unit += (int64_t)blocks * kWarps) {
        const Share s = share_of(a, w, key, unit, lane);
        const T* x_row = static_cast<const T*>(key ? a.k : a.q) + s.first;
        const T* g_row = static_cast<const T*>(key ? a.dko : a.dqo) + s.first;
        T* d_row = static_cast<T*>(key ? a.ko : a.qo) + s.first;
        typename Io<T>::Raw rx[kAheadBack], rg[kAheadBack];
#pragma unroll
        for (int u = 0; u < kAheadBack; ++u)
            if (s.h0 + u < s.h1) {
                rx[u] = Io<T>::load(x_row + u * step, oa, ob);
                rg[u] = Io<T>::load(g_row + u * step, oa, ob);
            }
        Turn<kInterleaved> turn;
        turn.template set<-1>(a, s.pos, lane);
        for (int h = s.h0; h < s.h1; h += kAheadBack) {
#pragma unroll
            for (int u = 0; u < kAheadBack; ++u) {
                if (h + u >= s.h1) break;
                F2 x[4], g[4], dn[4];
                Io<T>::widen(rx[u], x);
                Io<T>::widen(rg[u], g);
                if (h + u + kAheadBack < s.h1) {
                    rx[u] = Io<T>::load(x_row + kAheadBack * step, oa, ob);
                    rg[u] = Io<T>::load(g_row + kAheadBack * step, oa, ob);
                }
                turn.apply(g);
#pragma unroll
                for (int j = 0; j < 4; ++j) dn[j] = mul(g[j], wt[j]);
                const float r = rsqrtf(row_dot(x, x) * (1.f / kHeadDim) + a.eps);
                // xh mean(dn xh) = x r^2 (dn . x) / 64
                const F2 m = both(row_dot(dn, x) * (-1.f / kHeadDim) * r * r), r2 = both(r);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    dn[j] = mul(fma(x[j], m, dn[j]), r2);
                    if (s.live) acc[j] = fma(g[j], mul(x[j], r2), acc[j]);
                }
                if (s.live) Io<T>::store(d_row, oa, ob, Io<T>::narrow(dn));
                x_row += step;
                g_row += step;
                d_row += step;
            }
        }
    }
    if (!a.partial) return;
    // lanes of the four tokens, then the warps, in a fixed order
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float2 v = un(acc[j]);
        v.x += __shfl_xor_sync(kFull, v.x, 8);
        v.y += __shfl_xor_sync(kFull, v.y, 8);
        v.x += __shfl_xor_sync(kFull, v.x, 16);
        v.y += __shfl_xor_sync(kFull, v.y, 16);
        if (lane < kRowLanes) {
            const int c = (j < 2 ? oa : ob) + 2 * (j & 1);
            sums[warp][c] = v.x;
            sums[warp][c + 1] = v.y;
        }
    }
    __syncthreads();
    if (threadIdx.x < kHeadDim) {
        float t = 0.f;
        for (int v = 0; v < kWarps; ++v) t += sums[v][threadIdx.x];
        a.partial[(int64_t)blockIdx.x * kHeadDim + threadIdx.x] = t;
    }
}

// dw = the sum of the blocks' partial sums (the queries' blocks, then the keys'): 8 groups of
// threads take every eighth block, then their sums are added in order.
constexpr int kFinishGroups = 8;
template <class T>
__global__ void __launch_bounds__(2 * kHeadDim * kFinishGroups)
qk_weight_kernel(const float* partial, int q_blocks, int k_blocks, T* dwq, T* dwk) {
    __shared__ float sums[kFinishGroups][2 * kHeadDim];
    ptx::griddep_wait();
    const int c = threadIdx.x % (2 * kHeadDim), grp = threadIdx.x / (2 * kHeadDim);
    const bool key = c >= kHeadDim;
    const float* src = partial + (key ? (int64_t)q_blocks * kHeadDim : 0) + c % kHeadDim;
    const int blocks = key ? k_blocks : q_blocks;
    float t = 0.f;
#pragma unroll 8
    for (int b = grp; b < blocks; b += kFinishGroups) t += src[(int64_t)b * kHeadDim];
    sums[grp][c] = t;
    __syncthreads();
    if (grp) return;
    t = 0.f;
    for (int k = 0; k < kFinishGroups; ++k) t += sums[k][c];
    T* dst = key ? dwk : dwq;
    if (dst) dst[c % kHeadDim] = Io<T>::round(t);
}

// The rotation alone: y = magnitude R(p) x on the turned features, the others as they are; kSign -1
// turns back (the gradient).  The same rows, lanes and runs as above without the norm's sum: HBM alone
// bounds it (16 + 16 heads x 16384 tokens in bf16: 20.8 us, 6.5 TB/s; neighbouring pairs 21.0, and 22.9 where two
// registers too many leave three blocks an SM; fp32 needs none held to it: 42 us so, 53 with four blocks).
template <class T, bool kInterleaved, int kSign>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 1) rope_kernel(const __grid_constant__ QkArgs a, const Work w) {
    const int lane = threadIdx.x & 31;
    int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= w.q_units + w.k_units) return;
    const bool key = unit >= w.q_units;
    if (key) unit -= w.q_units;
    const Share s = share_of(a, w, key, unit, lane);
    int oa, ob;
    pieces<kInterleaved>(a.rot, lane, &oa, &ob);
    const int64_t step = a.n * kHeadDim;      // from head to head
    const T* src = static_cast<const T*>(key ? a.k : a.q) + s.first;
    T* dst = static_cast<T*>(key ? a.ko : a.qo) + s.first;
    typename Io<T>::Raw raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (s.h0 + u < s.h1) raw[u] = Io<T>::load(src + u * step, oa, ob);
    Turn<kInterleaved> turn;
    turn.template set<kSign>(a, s.pos, lane);
    turn.scale(a.magnitude);
    // the other lanes' features are copied as bits: 0 times an infinity would be NaN
    const bool turned = (lane & (kRowLanes - 1)) < a.rot / 8;
    for (int h = s.h0; h < s.h1; h += kAhead, src += kAhead * step, dst += kAhead * step) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (h + u >= s.h1) break;
            F2 v[4], kept[4];
            Io<T>::widen(raw[u], v);
            if (h + u + kAhead < s.h1) raw[u] = Io<T>::load(src + (u + kAhead) * step, oa, ob);
#pragma unroll
            for (int j = 0; j < 4; ++j) kept[j] = v[j];
            turn.apply(v);
            if (s.live) Io<T>::store(dst + u * step, oa, ob, Io<T>::either(turned, v, kept));
        }
    }
}

constexpr int64_t kManyWarps = 152 * 48;     // warps that fill the GPU
constexpr int64_t kBackBlocks = 152 * 2;     // the backward's blocks that run at once

// A run is all the heads of a tensor where the tokens alone make enough warps, fewer (down to
// one) where they do not.  (Backward, 3 x (5 + 5) heads x 1021 tokens: 9.2 us with the warps that
// run at once as the measure, 11.5 with three times as many, whose runs are of one head.)
Work plan(int64_t tokens, int64_t Hq, int64_t Hk, bool backward) {
    Work w;
    w.groups = (tokens + kTok - 1) / kTok;
    const int64_t fill = backward ? kBackBlocks * kWarps : kManyWarps;
    const int64_t runs = (fill + w.groups - 1) / w.groups;
    const int64_t per = (Hq + Hk + runs - 1) / runs, most = Hq > Hk ? Hq : Hk;
    w.per = (int32_t)(per < 1 ? 1 : per < most ? per : most);
    w.q_units = w.groups * ((Hq + w.per - 1) / w.per);
    w.k_units = w.groups * ((Hk + w.per - 1) / w.per);
    // backward: as many blocks as run at once (each leaves a row of partial sums), their warps
    // with the same number of units
    const int64_t q = (w.q_units + kWarps - 1) / kWarps, k = (w.k_units + kWarps - 1) / kWarps;
    const int64_t rounds = (q + k + kBackBlocks - 1) / kBackBlocks;
    w.q_blocks = (int32_t)((q + rounds - 1) / rounds);
    w.k_blocks = (int32_t)((k + rounds - 1) / rounds);
    return w;
}

template <class T>
int forward_as(const QkArgs& a, bool interleaved, cudaStream_t stream) {
    const Work w = plan(a.tokens, a.Hq, a.Hk, false);
    const int64_t blocks = (w.q_units + w.k_units + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many rows");
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        if (interleaved) qk_forward_kernel<T, true><<<(unsigned)blocks, kThreads, 0, stream>>>(a, w);
        else qk_forward_kernel<T, false><<<(unsigned)blocks, kThreads, 0, stream>>>(a, w);
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "qk_forward_kernel");
}

template <class T, int kSign>
int rope_as(const QkArgs& a, bool interleaved, cudaStream_t stream) {
    const Work w = plan(a.tokens, a.Hq, a.Hk, false);
    const int64_t blocks = (w.q_units + w.k_units + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return fail(DIFFUSER_ERR_OVERFLOW, "too many rows");
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        if (interleaved) rope_kernel<T, true, kSign><<<(unsigned)blocks, kThreads, 0, stream>>>(a, w);
        else rope_kernel<T, false, kSign><<<(unsigned)blocks, kThreads, 0, stream>>>(a, w);
    }
    const cudaError_t err = cudaGetLastError();
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "rope_kernel");
}

template <class T>
int backward_as(const QkArgs& a, bool interleaved, void* dwq, void* dwk, cudaStream_t stream) {
    const Work w = plan(a.tokens, a.Hq, a.Hk, true);
    const int blocks = w.q_blocks + w.k_blocks;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        if (interleaved) qk_backward_kernel<T, true><<<(unsigned)blocks, kThreads, 0, stream>>>(a, w);
        else qk_backward_kernel<T, false><<<(unsigned)blocks, kThreads, 0, stream>>>(a, w);
    }
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return cuda_fail(err, "qk_backward_kernel");
    if (!dwq && !dwk) return DIFFUSER_OK;
    {
        LaunchScope scope(DIFFUSER_KERNEL_AUX, stream);
        err = launch_pdl(qk_weight_kernel<T>, dim3(1), dim3(2 * kHeadDim * kFinishGroups), 0, stream, a.partial, w.q_blocks,
                         w.k_blocks, static_cast<T*>(dwq), static_cast<T*>(dwk));
    }
    return err == cudaSuccess ? DIFFUSER_OK : cuda_fail(err, "qk_weight_kernel");
}

}  // namespace

int64_t qk_backward_blocks(int64_t tokens, int64_t Hq, int64_t Hk) {
    const Work w = plan(tokens, Hq, Hk, true);
    return w.q_blocks + w.k_blocks;
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

int launch_rope(const QkArgs& a, int32_t dtype, bool interleaved, bool back, cudaStream_t stream) {
    if (dtype == DIFFUSER_DTYPE_BF16)
        return back ? rope_as<__nv_bfloat16, -1>(a, interleaved, stream) : rope_as<__nv_bfloat16, 1>(a, interleaved, stream);
    return back ? rope_as<float, -1>(a, interleaved, stream) : rope_as<float, 1>(a, interleaved, stream);
}

}  // namespace dfs
