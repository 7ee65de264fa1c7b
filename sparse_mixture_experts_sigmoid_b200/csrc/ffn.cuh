// Declarations shared by the kernels of the dense gated feed-forward block:
// the products as they are handed to a kernel, the activations, and the 16-bit
// element helpers.
#pragma once

#include <cuda_fp16.h>

#include "moe_internal.cuh"
#include "packed.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace ffn {

// A row-major matrix of 16-bit elements (the kept u and v: fp32), row stride ld elements.
struct Matrix {
    const void *base;
    int64_t rows, cols, ld;
};

// What an epilogue does (see ffn_pair.cu).
enum Kind : int { GATED = 0, STORE = 1, DGATED = 2 };

// One product C[M, N] = sum over K of A and B (see ffn_pair.cu).
struct Gemm {
    bool a_mn;           // the reduction runs over A's rows (launch_grads)
    Matrix a0, a1, b0, b1;
    Matrix c0, c1;       // GATED: act; STORE: C (C1: second half); DGATED: du, dv
    Matrix u, v;         // the kept pre-activations, fp32: GATED stores them (base null: not), DGATED reads them
    int64_t M, K;        // K per range
    int N;
    int ranges, halves;
    int act;             // moe_ffn_act
    bool bf16;           // else fp16
    uint32_t *err;
};
// act = act(A B0^T) * (A B1^T);  C = A B^T;  du, dv from r = A B.
cudaError_t launch_gated(const Gemm &g, cudaStream_t s);
cudaError_t launch_down(const Gemm &g, cudaStream_t s);
cudaError_t launch_dgated(const Gemm &g, cudaStream_t s);
// C = A B, or A^T B (a_mn), of up to three products in one launch; the second and
// third have the same K.
cudaError_t launch_grads(const Gemm *g, int n, cudaStream_t s);

// Shared-memory descriptor of an MN-major operand of 64 k-rows (128-byte swizzle):
// atoms of 64 columns, kAtom bytes apart; 8-row groups 1 KB apart; a K slice of 16
// rows is 2 KB on.
constexpr int kAtom = 8192;   // 64 k-rows x 128 bytes
__device__ __forceinline__ uint64_t desc_mn(const void *p) {
    const uint32_t a = tc::smem_u32(p);
    return (uint64_t)((a & 0x3FFFF) >> 4) | ((uint64_t)(kAtom >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// ------------------------------------------------------------------ elements

// fmt: 1 bf16, 0 fp16 (the formats of the MMA's instruction descriptor).
__device__ __forceinline__ uint32_t pack2(float a, float b, uint32_t fmt) {
    uint32_t r;
    if (fmt) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        r = *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        r = *reinterpret_cast<const uint32_t *>(&v);
    }
    return r;
}

// ------------------------------------------------------------------ activations
// silu(u) = u s, s = 1 / (1 + exp(-u));  gelu_tanh(u) = u (1 + tanh z) / 2 = u s,
// z = sqrt(2 / pi) (u + 0.044715 u^3), s = 1 / (1 + exp(-2 z)).  Two elements at a
// time: s takes two operations of the special function unit, the rest is packed.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu = 1.5957691216057308f;   // 2 sqrt(2 / pi)

// s of a pair; for gelu_tanh u2 = u^2 as well.
template <int ACT>
__device__ __forceinline__ float2 act_gate(float2 u, float2 &u2) {
    if constexpr (ACT == MOE_ACT_SILU) return logistic2(mul2(u, both(-kLog2e)));
    u2 = mul2(u, u);
    return logistic2(mul2(u, fma2(u2, both(-kLog2e * kGelu * 0.044715f), both(-kLog2e * kGelu))));
}
// act(u) v
template <int ACT>
__device__ __forceinline__ float2 gated2(float2 u, float2 v) {
    float2 u2;
    return mul2(mul2(u, act_gate<ACT>(u, u2)), v);
}
// a = act(u), da = act'(u) = s + u s' with s' = s (1 - s) d(2 z)/du.
template <int ACT>
__device__ __forceinline__ void act_grad2(float2 u, float2 &a, float2 &da) {
    float2 u2;
    const float2 s = act_gate<ACT>(u, u2);
    a = mul2(u, s);
    float2 t = mul2(a, fma2(s, both(-1.f), both(1.f)));
    if constexpr (ACT == MOE_ACT_GELU_TANH) {
        // d(2 z) / du = 2 sqrt(2 / pi) (1 + 3 * 0.044715 u^2); past |u| = 100, where s is 0 or 1
        // and the term vanishes, u^2 is held so that it cannot become 0 * inf
        u2 = make_float2(fminf(u2.x, 1e4f), fminf(u2.y, 1e4f));
        t = mul2(t, fma2(u2, both(3.f * 0.044715f * kGelu), both(kGelu)));
    }
    da = add2(t, s);
}

}  // namespace ffn
}  // namespace moe
