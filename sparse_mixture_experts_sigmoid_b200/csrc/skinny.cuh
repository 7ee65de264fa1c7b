// The product of a few token rows with a large weight (skinny.cu).
#pragma once

#include "moe_internal.cuh"

namespace moe {
namespace skinny {

// out[t, n] = sum_k x[t, k] w[n, k] (STORE), or act(u) v with u from w0 and v
// from w1 (GATED).  16-bit operands (fp8 = false), or e4m3 with scales (fp8;
// STORE only): sx [T, KB], sw [ceil(N / 128), KB], KB = ceil(K / 128).
struct Product {
    bool gated, fp8, bf16;     // bf16: 16-bit operands are bf16, else fp16
    int64_t T;
    int N, K;
    const void *x, *w0, *w1;   // x [T, K]; w0, w1 [N, K]
    const float *sx, *sw;
    void *out;                 // [T, N]
    int out_dtype;
    float *pre;                // GATED, optional: [T, 2N] u | v
    int act;                   // moe_ffn_act
    bool early;                // the kernel before this one in the stream does not write the weights:
                               // they are requested before it has completed
    uint32_t *err;
};
// Whether the product is one for this kernel (else the 256-row tiles).
enum class Form { kStore, kGated, kFp8 };
bool wants(Form form, int64_t T, int N, int K);
cudaError_t launch(const Product &p, cudaStream_t s);

}  // namespace skinny
}  // namespace moe
