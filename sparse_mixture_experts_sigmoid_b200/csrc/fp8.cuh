// Declarations shared by the kernels of the 8-bit floating point product.
#pragma once

#include "moe_internal.cuh"

namespace moe {
namespace fp8 {

constexpr int kBlock = 128;   // columns (and, for weights, rows) that share a scale

// C[M, N] = sum over K blocks kb of sa[m, kb] sb[n / 128, kb] (A_kb B_kb^T).
struct Gemm {
    int64_t M;
    int N, K;
    const uint8_t *a, *b;      // e4m3 [M, K], [N, K]
    const float *sa, *sb;      // [M, KB], [NB, KB]: KB = ceil(K / 128), NB = ceil(N / 128)
    void *c;
    int c_dtype;
    uint32_t *err;
};
cudaError_t launch_pair(const Gemm &g, cudaStream_t s);

}  // namespace fp8
}  // namespace moe
