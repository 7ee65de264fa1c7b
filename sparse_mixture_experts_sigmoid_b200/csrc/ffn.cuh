// Declarations shared by the kernels of the dense gated feed-forward block:
// the products as they are handed to a kernel, the activations, and the 16-bit
// element helpers.
#pragma once

#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {
namespace ffn {

// A row-major matrix of 16-bit elements, row stride ld elements.
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
    Matrix c0, c1, c2;   // GATED: act, and u, v (base null: not kept); STORE: C (C1: second half); DGATED: du, dv
    Matrix u, v;         // DGATED: the kept pre-activations
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
__device__ __forceinline__ float2 unpack2(uint32_t w, uint32_t fmt) {
    if (fmt) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// ------------------------------------------------------------------ activations
// silu: silu_f of moe_internal.cuh.  gelu_tanh(u) = u (1 + tanh z) / 2 with
// z = sqrt(2 / pi) (u + 0.044715 u^3); (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)).
__device__ __forceinline__ float gelu_gate(float u) {
    const float z2 = 1.5957691216057308f * u * fmaf(0.044715f * u, u, 1.f);   // 2 z
    return __fdividef(1.f, 1.f + __expf(-z2));
}
__device__ __forceinline__ float gelu_tanh_f(float u) { return u * gelu_gate(u); }

// a = act(u), da = act'(u).
template <int ACT>
__device__ __forceinline__ void act_grad(float u, float &a, float &da) {
    if constexpr (ACT == MOE_ACT_SILU) {
        const float s = __fdividef(1.f, 1.f + __expf(-u));
        a = u * s;
        da = s * (1.f + u * (1.f - s));
    } else {
        const float s = gelu_gate(u);
        a = u * s;
        // d(2 z) / du = 2 sqrt(2 / pi) (1 + 3 * 0.044715 u^2); past |u| = 100, where s is 0 or 1
        // and the term vanishes, u^2 is held so that it cannot become 0 * inf
        da = s + a * (1.f - s) * 1.5957691216057308f * fmaf(0.134145f, fminf(u * u, 1e4f), 1.f);
    }
}

}  // namespace ffn
}  // namespace moe
