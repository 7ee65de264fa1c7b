// Packed fp32 arithmetic: two operations an instruction (sm_100), for the
// kernels whose elementwise work shows.
#pragma once

#include <cuda_runtime.h>

namespace moe {

__device__ __forceinline__ unsigned long long bits2(float2 v) { return *reinterpret_cast<unsigned long long *>(&v); }
__device__ __forceinline__ float2 from2(unsigned long long b) { return *reinterpret_cast<float2 *>(&b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return from2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return from2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return from2(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float2 each(float2 v, float (*f)(float)) { return make_float2(f(v.x), f(v.y)); }

// 2^x and 1 / x by the special function unit, subnormals flushed (2^-22 and one
// step of relative error).
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 1 / (1 + 2^z): z past the range gives 0 (2^z = inf) or 1.
__device__ __forceinline__ float2 logistic2(float2 z) {
    return each(add2(each(z, exp2_approx), both(1.f)), rcp_approx);
}

}  // namespace moe
