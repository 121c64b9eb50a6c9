// Pairs of fp32 values in one 64-bit register and the instructions that work on both.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace dfs {
namespace packed {

struct F2 { uint64_t w; };
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.w) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 un(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v.w));
    return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.w) : "l"(a.w), "l"(b.w));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.w) : "l"(a.w), "l"(b.w), "l"(c.w));
    return r;
}
__device__ __forceinline__ F2 both(float x) { return f2(x, x); }

__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.w) : "l"(a.w), "l"(b.w));
    return r;
}

}  // namespace packed
}  // namespace dfs
