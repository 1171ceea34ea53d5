// Shared by the recurrence's and the heads' kernels: arithmetic on pairs of fp32 values, and the order of a
// kernel after the one before it.
#pragma once
#include "common.cuh"

namespace osdn {

// These kernels are launched so that they may start while the kernel before them in the stream still runs, once
// all its blocks have called let_next_start(): what they do before wait_for_previous() touches no device memory, and
// that returns when the earlier kernel is done and its writes are seen. A chain of them (a training step, a
// decode loop) then pays for a launch once.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
