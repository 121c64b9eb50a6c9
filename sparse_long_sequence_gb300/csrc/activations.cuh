// The activations of the dense and gated products and their slopes, in fp32.
//   relu       max(p, 0), slope 0 at p <= 0
//   gelu       p Phi(p), Phi the normal distribution function
//   gelu_tanh  p (1 + tanh u) / 2 = p / (1 + exp(-2u)), u = sqrt(2/pi) (p + 0.044715 p^3):
//              the second form has no cancellation for p far below 0
//   silu       p / (1 + exp(-p))
// The logistic function uses the hardware exponential and reciprocal: a relative error of about
// 2^-20 + 2^-24 |x|, the second part from the rounding of the exponent's argument (4e-6 where the
// value nears 2^-126), against the results' bf16 half step 2^-8.  Below 2^-126 it is 0, and it
// saturates to exactly 0 and 1, so that infinite p give their limits.
#pragma once

#include <cuda_runtime.h>

#include "../../include/diffuser.h"
#include "packed.cuh"
#include "sm100_ptx.cuh"

namespace dfs {
namespace act {

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + exp(-x))
__device__ __forceinline__ float logistic(float x) {
    return rcp_approx(1.f + ptx::ex2_approx(-1.4426950408889634f * x));
}
constexpr float kTanhC = 0.7978845608028654f;      // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;
constexpr float kPhiC = 0.3989422804014327f;       // 1 / sqrt(2 pi)

// x, or the lowest finite value for -inf (NaN stays NaN)
__device__ __forceinline__ float finite_below(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(-3.4028234663852886e38f));
    return y;
}
// x * s with s in [0, 1] a saturating factor, 0 at x = -inf
__device__ __forceinline__ float gate(float x, float s) { return finite_below(x) * s; }

// The normal distribution function at p and exp(-p^2 / 2).  With x = |p|, Phi(-x) =
// exp(-x^2 / 2) m(x), m the Mills ratio: t q(t) with t = 1 / (1 + 0.3 x) and q of degree 7, a
// relative minimax fit over 0 <= x <= 20 (the exponential flushes to 0 from 13.2 on), within
// 7e-7 in fp32; the exponential's argument is rounded to 2^-24 of itself, so that the lower tail
// is within 8e-6 of itself near |p| = 13.  (erfcf takes about twice the instructions:
// the gelu backward of 16384 x 4096 went from 140 to 76 us; 72 by now, with the bias gradient.)
__device__ __forceinline__ float2 normal(float p) {
    const float x = fabsf(p);
    const float t = rcp_approx(fmaf(0.3f, x, 1.f));
    float q = 0.0330325861f;
    q = fmaf(q, t, -0.146387965f);
    q = fmaf(q, t, 0.188117857f);
    q = fmaf(q, t, -0.0373392124f);
    q = fmaf(q, t, 0.120191655f);
    q = fmaf(q, t, 0.10235086f);
    q = fmaf(q, t, 0.12038182f);
    q = fmaf(q, t, 0.119652211f);
    const float e = ptx::ex2_approx(-0.7213475204444817f * p * p);
    const float tail = e * t * q;
    return make_float2(p < 0.f ? tail : 1.f - tail, e);
}

template <int kAct>
__device__ __forceinline__ float value(float p) {
    if constexpr (kAct == DIFFUSER_ACT_RELU) {
        return p > 0.f ? p : (p != p ? p : 0.f);
    } else if constexpr (kAct == DIFFUSER_ACT_GELU) {
        return gate(p, normal(p).x);
    } else if constexpr (kAct == DIFFUSER_ACT_GELU_TANH) {
        return gate(p, logistic(2.f * kTanhC * p * fmaf(kTanhA * p, p, 1.f)));
    } else if constexpr (kAct == DIFFUSER_ACT_SILU) {
        return gate(p, logistic(p));
    }
    return p;
}

// value and slope at p
template <int kAct>
__device__ __forceinline__ float2 value_slope(float p) {
    if constexpr (kAct == DIFFUSER_ACT_RELU) {
        return make_float2(value<kAct>(p), p > 0.f ? 1.f : (p != p ? p : 0.f));
    } else if constexpr (kAct == DIFFUSER_ACT_GELU) {
        const float2 n = normal(p);
        return make_float2(gate(p, n.x), n.x + (n.y == 0.f ? 0.f : p * n.y * kPhiC));
    } else if constexpr (kAct == DIFFUSER_ACT_GELU_TANH) {
        const float p2 = p * p;
        const float s = logistic(2.f * kTanhC * p * fmaf(kTanhA, p2, 1.f));
        const float q = s * (1.f - s);
        return make_float2(gate(p, s),
                           s + (q == 0.f ? 0.f : 2.f * kTanhC * p * q * fmaf(3.f * kTanhA, p2, 1.f)));
    } else if constexpr (kAct == DIFFUSER_ACT_SILU) {
        const float s = logistic(p);
        const float q = s * (1.f - s);
        return make_float2(gate(p, s), s + (q == 0.f ? 0.f : p * q));
    }
    return make_float2(p, 1.f);
}

// min(|x|, the largest finite value); NaN stays NaN
__device__ __forceinline__ float finite_abs(float x) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(fabsf(x)), "f"(3.4028234663852886e38f));
    return y;
}
// q(t) of normal(), two at a time
__device__ __forceinline__ packed::F2 mills2(packed::F2 t) {
    using namespace packed;
    F2 q = both(0.0330325861f);
    q = fma(q, t, both(-0.146387965f));
    q = fma(q, t, both(0.188117857f));
    q = fma(q, t, both(-0.0373392124f));
    q = fma(q, t, both(0.120191655f));
    q = fma(q, t, both(0.10235086f));
    q = fma(q, t, both(0.12038182f));
    return fma(q, t, both(0.119652211f));
}

// The same values two at a time: the products and sums of both in one instruction, which the
// dense products' epilogues are bound by.
template <int kAct>
__device__ __forceinline__ packed::F2 value2(packed::F2 p) {
    using namespace packed;
    if constexpr (kAct == DIFFUSER_ACT_SILU || kAct == DIFFUSER_ACT_GELU_TANH) {
        F2 x;                                    // exponent of 2 in 1 / (1 + 2^x)
        if constexpr (kAct == DIFFUSER_ACT_SILU) {
            x = mul(p, both(-1.4426950408889634f));
        } else {
            constexpr float c = -2.f * kTanhC * 1.4426950408889634f;
            x = mul(p, fma(mul(p, p), both(c * kTanhA), both(c)));
        }
        const float2 e = un(x);
        const float2 d = un(add(f2(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y)), both(1.f)));
        const float2 q = un(p);
        return mul(f2(finite_below(q.x), finite_below(q.y)), f2(rcp_approx(d.x), rcp_approx(d.y)));
    } else if constexpr (kAct == DIFFUSER_ACT_GELU) {
        // max(p, 0) - x Phi(-x), x = |p| (the largest finite value for infinity: 0 times it is 0)
        const float2 v = un(p);
        const F2 x = f2(finite_abs(v.x), finite_abs(v.y));
        const float2 d = un(fma(x, both(0.3f), both(1.f)));
        const F2 t = f2(rcp_approx(d.x), rcp_approx(d.y));
        const float2 h = un(mul(mul(x, x), both(-0.7213475204444817f)));
        const F2 tail = mul(mul(f2(ptx::ex2_approx(h.x), ptx::ex2_approx(h.y)), t), mills2(t));
        return fma(mul(x, both(-1.f)), tail, f2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
    } else {
        const float2 q = un(p);
        return f2(value<kAct>(q.x), value<kAct>(q.y));
    }
}

// value<act> for an activation known at run time (uniform over the launch)
__device__ __forceinline__ float value_of(int a, float p) {
    switch (a) {
        case DIFFUSER_ACT_RELU: return value<DIFFUSER_ACT_RELU>(p);
        case DIFFUSER_ACT_GELU: return value<DIFFUSER_ACT_GELU>(p);
        case DIFFUSER_ACT_GELU_TANH: return value<DIFFUSER_ACT_GELU_TANH>(p);
        case DIFFUSER_ACT_SILU: return value<DIFFUSER_ACT_SILU>(p);
        default: return p;
    }
}

}  // namespace act
}  // namespace dfs
