// Arithmetic on pairs of fp32 values, shared by the recurrence and the heads' kernels.
#pragma once
#include "common.cuh"

namespace osdn {

// Two fp32 values at a time: one instruction for both (fma, mul, add on f32x2).

__device__ __forceinline__ uint64_t bits2(float2 a) { return *reinterpret_cast<uint64_t*>(&a); }
__device__ __forceinline__ float2 pair2(uint64_t a) { return *reinterpret_cast<float2*>(&a); }
__device__ __forceinline__ float2 all2(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return pair2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(r);
}
__device__ __forceinline__ float2 less1(float2 a) { return fma2(a, all2(-1.f), all2(1.f)); }   // 1 - a

__device__ __forceinline__ float rroot(float x) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace osdn
