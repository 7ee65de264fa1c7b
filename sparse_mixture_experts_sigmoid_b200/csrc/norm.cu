// Layer norm and RMS norm of token rows, forward and backward, with the
// residual addition in front of the norm.
//
//   h    = round(x + residual)                      (or x itself)
//   mean = layer ? sum_i h_i / d : 0
//   rstd = 1 / sqrt(sum_i (h_i - mean)^2 / d + eps)
//   y_i  = (h_i - mean) * rstd * w_i (+ b_i)
//
// Backward, with xhat = (h - mean) * rstd and g = dy * w:
//
//   dx_i = rstd * (g_i - [layer] avg(g) - xhat_i * avg(g * xhat)) (+ dh_i)
//   dw_i = sum_t dy_ti xhat_ti,   db_i = sum_t dy_ti
//
// Both passes are bound by memory: a few operations per element, every input
// element read once and every output element written once.  A row is held in
// the registers of the W warps that own it (W = 1 for short rows), so the
// variance is summed over (h - mean)^2 after the mean is known, without a
// second read, and all statistics, sums and gradients are fp32.  The next
// row's loads are issued before the current row's reductions, so that bytes
// stay in flight while the warps synchronise.
//
// The gradients of w and b are sums over the tokens: each thread adds its
// columns over the rows of its block in fp32 registers, the blocks write one
// partial row each, and a second kernel adds the partial rows.  Every order is
// fixed, so repeated calls give the same bits.
#include <algorithm>

#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kMaxWarps = 16;      // warps per row at most

// E elements of one 16-byte word.
template <typename T>
constexpr int kElems = 16 / (int)sizeof(T);

__device__ __forceinline__ float el_f32(float v) { return v; }
__device__ __forceinline__ float el_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float el_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T el_from(float v);
template <> __device__ __forceinline__ float el_from<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 el_from<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half el_from<__half>(float v) { return __float2half_rn(v); }

// The elements of a row that one thread holds: VPT words of E elements.  With
// VEC word j is the 16-byte word j * G + i of the row (i the thread in its
// group of G); without it (widths or addresses that are not whole words)
// element e of word j is the row's element (j * E + e) * G + i, so that a
// warp's loads are still of consecutive elements.
template <typename T, int VPT, bool VEC>
struct Row {
    static constexpr int E = kElems<T>;
    union Word {
        uint4 w;
        T e[E];
    };
    Word v[VPT];

    __device__ __forceinline__ static int column(int i, int G, int j, int e) {
        return VEC ? (j * G + i) * E + e : (j * E + e) * G + i;
    }
    __device__ __forceinline__ void load_word(const T *p, int i, int G, int d, int j) {
        if constexpr (VEC) {
            const int c = column(i, G, j, 0);
            v[j].w = c < d ? *reinterpret_cast<const uint4 *>(p + c) : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = column(i, G, j, e);
                v[j].e[e] = c < d ? p[c] : el_from<T>(0.f);
            }
        }
    }
    __device__ __forceinline__ void store_word(T *p, int i, int G, int d, int j) const {
        if constexpr (VEC) {
            const int c = column(i, G, j, 0);
            if (c < d) *reinterpret_cast<uint4 *>(p + c) = v[j].w;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = column(i, G, j, e);
                if (c < d) p[c] = v[j].e[e];
            }
        }
    }
    __device__ __forceinline__ void load(const T *p, int i, int G, int d) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) load_word(p, i, G, d, j);
    }
    __device__ __forceinline__ void store(T *p, int i, int G, int d) const {
#pragma unroll
        for (int j = 0; j < VPT; ++j) store_word(p, i, G, d, j);
    }
    __device__ __forceinline__ float get(int j, int e) const { return el_f32(v[j].e[e]); }
    __device__ __forceinline__ void set(int j, int e, float f) { v[j].e[e] = el_from<T>(f); }
};

// Word j of the weight or bias vector (of type T, or fp32 when wf32) for this
// thread's columns, as fp32.
template <typename T, bool VEC>
__device__ __forceinline__ void load_param(const void *p, bool wf32, int i, int G, int j, int d,
                                           float (&o)[kElems<T>]) {
    constexpr int E = kElems<T>;
    if constexpr (VEC) {
        const int c = (j * G + i) * E;
        if (c >= d) {
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = 0.f;
        } else if (wf32) {
#pragma unroll
            for (int q = 0; q < E / 4; ++q) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + c) + q);
                o[4 * q] = f.x;
                o[4 * q + 1] = f.y;
                o[4 * q + 2] = f.z;
                o[4 * q + 3] = f.w;
            }
        } else {
            union {
                uint4 w;
                T e[E];
            } u;
            u.w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p) + c));
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = el_f32(u.e[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = (j * E + e) * G + i;
            o[e] = c >= d ? 0.f : (wf32 ? static_cast<const float *>(p)[c] : el_f32(static_cast<const T *>(p)[c]));
        }
    }
}

template <typename T>
__device__ __forceinline__ float param(const void *p, bool wf32, int c) {
    return wf32 ? __ldg(static_cast<const float *>(p) + c) : el_f32(static_cast<const T *>(p)[c]);
}

// Sums over the W warps of a row's group.  `slot` is the group's buffer of
// 2 x W values of this type, used in turn: a warp writes half `turn` again
// only after a barrier that every warp reaches after it has read that half.
template <typename V>
__device__ __forceinline__ V group_sum(V v, V *slot, int &turn, int W, int bar, V (*add)(V, V)) {
    if (W == 1) return v;
    V *s = slot + turn * W;
    turn ^= 1;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) % W;
    if (lane == 0) s[w] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(W * 32) : "memory");
    V r = s[0];
    for (int k = 1; k < W; ++k) r = add(r, s[k]);
    return r;
}
__device__ __forceinline__ float add1(float a, float b) { return a + b; }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }

struct NormFwd {
    const void *x, *residual, *weight, *bias;
    void *h, *y;
    float *mean, *rstd;
    int64_t T;
    int d, W, groups;       // warps per row, rows in flight per block
    bool layer, wf32;
    float eps;
};

template <typename T, int VPT, bool VEC>
__global__ void __launch_bounds__(VPT == 3 ? 256 : 512) norm_fwd_kernel(NormFwd a) {
    constexpr int E = kElems<T>;
    __shared__ float red[2 * kMaxWarps];
    const int W = a.W, G = W * 32, d = a.d;
    const int group = threadIdx.x / G, i = threadIdx.x % G;
    float *slot = red + 2 * W * group;
    int turn = 0;
    const float df = (float)d;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    const int64_t step = (int64_t)gridDim.x * a.groups;
    int64_t r = (int64_t)blockIdx.x * a.groups + group;
    pdl_wait();
    pdl_launch_dependents();
    Row<T, VPT, VEC> nx, nr;
    if (r < a.T) {
        nx.load(x + r * d, i, G, d);
        if (res) nr.load(res + r * d, i, G, d);
    }
    for (; r < a.T; r += step) {
        Row<T, VPT, VEC> c = nx;
        if (res) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) c.set(j, e, c.get(j, e) + nr.get(j, e));
        }
        if (r + step < a.T) {
            nx.load(x + (r + step) * d, i, G, d);
            if (res) nr.load(res + (r + step) * d, i, G, d);
        }
        if (res) c.store(static_cast<T *>(a.h) + r * d, i, G, d);
        float mean = 0.f;
        if (a.layer) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) s += c.get(j, e);
            mean = group_sum(warp_sum(s), slot, turn, W, 1 + group, add1) / df;
        }
        float q = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float z = Row<T, VPT, VEC>::column(i, G, j, e) < d ? c.get(j, e) - mean : 0.f;
                q = fmaf(z, z, q);
            }
        const float rstd = rsqrtf(group_sum(warp_sum(q), slot, turn, W, 1 + group, add1) / df + a.eps);
        if (i == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float w[E], b[E];
            load_param<T, VEC>(a.weight, a.wf32, i, G, j, d, w);
            if (a.bias) load_param<T, VEC>(a.bias, a.wf32, i, G, j, d, b);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float z = (c.get(j, e) - mean) * rstd;
                c.set(j, e, a.bias ? fmaf(z, w[e], b[e]) : z * w[e]);
            }
        }
        c.store(static_cast<T *>(a.y) + r * d, i, G, d);
    }
}

struct NormBwd {
    const void *h, *weight, *dy, *dh;
    const float *mean, *rstd;
    void *dx;
    float *part;            // [gridDim.x, 2, d]: dw then db of each block (nullptr: not wanted)
    int64_t T;
    int d, W, groups;
    bool wf32, want_db;
};

template <typename T, int VPT, bool VEC>
__global__ void __launch_bounds__(VPT == 3 ? 256 : 512) norm_bwd_kernel(NormBwd a) {
    // up to three words a thread are held between the two passes over a row
    // (and the next row's requested); of wider rows only the gradients' sums
    // stay in registers, and the second pass reads the row again, from L1
    constexpr bool HOLD = VPT <= 3;
    constexpr int E = kElems<T>;
    __shared__ float2 red[2 * kMaxWarps];
    extern __shared__ float cols[];     // groups > 1: [2, d]
    const int W = a.W, G = W * 32, d = a.d;
    const int group = threadIdx.x / G, i = threadIdx.x % G;
    float2 *slot = red + 2 * W * group;
    int turn = 0;
    const float df = (float)d;
    const T *h = static_cast<const T *>(a.h), *dy = static_cast<const T *>(a.dy), *dh = static_cast<const T *>(a.dh);
    const int64_t step = (int64_t)gridDim.x * a.groups;
    int64_t r = (int64_t)blockIdx.x * a.groups + group;
    float dw[VPT][E], db[VPT][E];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[j][e] = db[j][e] = 0.f;
    pdl_wait();
    pdl_launch_dependents();
    Row<T, VPT, VEC> nh, ny;
    if (HOLD && r < a.T) {
        nh.load(h + r * d, i, G, d);
        ny.load(dy + r * d, i, G, d);
    }
    for (; r < a.T; r += step) {
        Row<T, VPT, VEC> ch, cy, cd;
        if constexpr (HOLD) {
            ch = nh;
            cy = ny;
            if (dh) cd.load(dh + r * d, i, G, d);
        }
        if (HOLD && r + step < a.T) {
            nh.load(h + (r + step) * d, i, G, d);
            ny.load(dy + (r + step) * d, i, G, d);
        }
        const float mean = a.mean ? a.mean[r] : 0.f, rstd = a.rstd[r];
        float2 s = make_float2(0.f, 0.f);   // sums of g and g * xhat
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float w[E];
            load_param<T, VEC>(a.weight, a.wf32, i, G, j, d, w);
            if constexpr (!HOLD) {
                ch.load_word(h + r * d, i, G, d, j);
                cy.load_word(dy + r * d, i, G, d, j);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                // columns past d hold dy = 0: they add nothing to any sum
                const float xh = (ch.get(j, e) - mean) * rstd, y = cy.get(j, e);
                const float g = y * w[e];
                s.x += g;
                s.y = fmaf(g, xh, s.y);
                dw[j][e] = fmaf(y, xh, dw[j][e]);
                db[j][e] += y;
            }
        }
        s.x = warp_sum(s.x);
        s.y = warp_sum(s.y);
        s = group_sum(s, slot, turn, W, 1 + group, add2);
        const float c1 = a.mean ? s.x / df : 0.f, c2 = s.y / df;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float w[E];
            load_param<T, VEC>(a.weight, a.wf32, i, G, j, d, w);
            if constexpr (!HOLD) {
                ch.load_word(h + r * d, i, G, d, j);
                cy.load_word(dy + r * d, i, G, d, j);
                if (dh) cd.load_word(dh + r * d, i, G, d, j);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float xh = (ch.get(j, e) - mean) * rstd;
                const float g = rstd * (fmaf(cy.get(j, e), w[e], -c1) - xh * c2);
                ch.set(j, e, dh ? g + cd.get(j, e) : g);
            }
            ch.store_word(static_cast<T *>(a.dx) + r * d, i, G, d, j);
        }
    }
    if (!a.part) return;
    float *out = a.part + (int64_t)blockIdx.x * 2 * d;
    // the block's groups add their columns one after another
    for (int g = 0; g < a.groups; ++g) {
        if (group == g) {
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int c = Row<T, VPT, VEC>::column(i, G, j, e);
                    if (c >= d) continue;
                    float sw = dw[j][e], sb = db[j][e];
                    if (g > 0) {
                        sw += cols[c];
                        sb += cols[d + c];
                    }
                    if (g + 1 < a.groups) {
                        cols[c] = sw;
                        cols[d + c] = sb;
                    } else {
                        out[c] = sw;
                        if (a.want_db) out[d + c] = sb;
                    }
                }
        }
        if (a.groups > 1) __syncthreads();
    }
}

// Any width and alignment: one block per row at a time, its columns strided
// over the threads and read once per pass (from L1 or L2 after the first).
// Serves the rows that do not fit the register kernels: widths or addresses
// that are not whole 16-byte words, beyond kMaxWarps * 32 threads' elements.
constexpr int kGenThreads = 512;

template <typename V>
__device__ __forceinline__ V block_sum(V v, V *s, V (*add)(V, V)) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    __syncthreads();   // the previous sum has been read
    if (lane == 0) s[w] = v;
    __syncthreads();
    V r = s[0];
    for (int k = 1; k < kGenThreads / 32; ++k) r = add(r, s[k]);
    return r;
}

template <typename T>
__global__ void __launch_bounds__(kGenThreads) norm_fwd_general_kernel(NormFwd a) {
    __shared__ float red[kGenThreads / 32];
    const int d = a.d;
    const float df = (float)d;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + r * d;
        if (a.residual) {
            const T *res = static_cast<const T *>(a.residual) + r * d;
            T *h = static_cast<T *>(a.h) + r * d;
            for (int c = threadIdx.x; c < d; c += kGenThreads) h[c] = el_from<T>(el_f32(x[c]) + el_f32(res[c]));
            x = h;   // each thread goes on with the columns that it wrote
        }
        float mean = 0.f;
        if (a.layer) {
            float s = 0.f;
            for (int c = threadIdx.x; c < d; c += kGenThreads) s += el_f32(x[c]);
            mean = block_sum(warp_sum(s), red, add1) / df;
        }
        float q = 0.f;
        for (int c = threadIdx.x; c < d; c += kGenThreads) {
            const float z = el_f32(x[c]) - mean;
            q = fmaf(z, z, q);
        }
        const float rstd = rsqrtf(block_sum(warp_sum(q), red, add1) / df + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
        T *y = static_cast<T *>(a.y) + r * d;
        for (int c = threadIdx.x; c < d; c += kGenThreads) {
            const float z = (el_f32(x[c]) - mean) * rstd, w = param<T>(a.weight, a.wf32, c);
            y[c] = el_from<T>(a.bias ? fmaf(z, w, param<T>(a.bias, a.wf32, c)) : z * w);
        }
    }
}

// The gradients' sums over the block's rows stand in shared memory, each
// column's owned by one thread.
template <typename T>
__global__ void __launch_bounds__(kGenThreads) norm_bwd_general_kernel(NormBwd a) {
    __shared__ float2 red[kGenThreads / 32];
    extern __shared__ float cols[];   // [2, d]: dw, db
    const int d = a.d;
    const float df = (float)d;
    for (int c = threadIdx.x; c < d; c += kGenThreads) cols[c] = cols[d + c] = 0.f;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t r = blockIdx.x; r < a.T; r += gridDim.x) {
        const T *h = static_cast<const T *>(a.h) + r * d, *dy = static_cast<const T *>(a.dy) + r * d;
        const T *dh = a.dh ? static_cast<const T *>(a.dh) + r * d : nullptr;
        T *dx = static_cast<T *>(a.dx) + r * d;
        const float mean = a.mean ? a.mean[r] : 0.f, rstd = a.rstd[r];
        float2 s = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < d; c += kGenThreads) {
            const float xh = (el_f32(h[c]) - mean) * rstd, y = el_f32(dy[c]), g = y * param<T>(a.weight, a.wf32, c);
            s.x += g;
            s.y = fmaf(g, xh, s.y);
            cols[c] = fmaf(y, xh, cols[c]);
            cols[d + c] += y;
        }
        s.x = warp_sum(s.x);
        s.y = warp_sum(s.y);
        s = block_sum(s, red, add2);
        const float c1 = a.mean ? s.x / df : 0.f, c2 = s.y / df;
        for (int c = threadIdx.x; c < d; c += kGenThreads) {
            const float xh = (el_f32(h[c]) - mean) * rstd;
            const float g = rstd * (fmaf(el_f32(dy[c]), param<T>(a.weight, a.wf32, c), -c1) - xh * c2);
            dx[c] = el_from<T>(dh ? g + el_f32(dh[c]) : g);
        }
    }
    if (!a.part) return;
    float *out = a.part + (int64_t)blockIdx.x * 2 * d;
    for (int c = threadIdx.x; c < d; c += kGenThreads) {
        out[c] = cols[c];
        if (a.want_db) out[d + c] = cols[d + c];
    }
}

// dw and db: the sums of the blocks' partial rows [parts, 2, d].  A block
// takes 32 columns (of dw, or of db in the grid's second half); warp k adds
// every 32nd part from part k, and the 32 sums are added in order.
__global__ void __launch_bounds__(1024) norm_param_kernel(const float *part, int parts, int d, float *dw, float *db) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const float *p = part + (blockIdx.y ? d : 0);
    pdl_wait();
    pdl_launch_dependents();
    float v = 0.f;
    if (c < d)
        for (int k = warp; k < parts; k += 32) v += p[(int64_t)k * 2 * d + c];
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < d) {
        float r = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) r += s[k][lane];
        float *o = blockIdx.y ? db : dw;
        if (o) o[c] = r;
    }
}

// How a row is spread: VPT words per thread, W warps per row, `groups` rows
// per block; vpt = 0 is the general kernel.  Whole words: a short row (up to
// three words a lane) stays in one warp, which needs no barrier; a longer one
// takes as many warps as hold it at two words a thread, at four (eight) where
// more than 16 warps would be needed.  Single elements: as many warps as hold
// the row at eight elements a thread, else the general kernel.
struct Spread {
    int vpt, W, groups;
};
Spread spread(int d, int elems, bool vec) {
    Spread s;
    if (vec) {
        const int words = (d + elems - 1) / elems;
        if (words <= 96) {
            s.vpt = (words + 31) / 32;
            s.W = 1;
        } else {
            s.vpt = words <= 64 * kMaxWarps ? 2 : (words <= 128 * kMaxWarps ? 4 : 8);
            s.W = (words + 32 * s.vpt - 1) / (32 * s.vpt);
        }
    } else {
        s.vpt = 8 / elems;
        s.W = (d + 255) / 256;
        if (s.W > kMaxWarps) return Spread{0, kGenThreads / 32, 1};
    }
    s.groups = std::max(1, 8 / s.W);
    return s;
}

int elem_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// Blocks of the backward pass, and so partial rows of the weight's gradient:
// two per SM, fewer when there are fewer rows.
constexpr int kBwdBlocks = 296;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The kernel for a type and spread (see spread()).
template <typename T>
auto fwd_kernel(int vpt, bool vec) -> void (*)(NormFwd) {
    if (vpt == 0) return norm_fwd_general_kernel<T>;
    if (!vec) return norm_fwd_kernel<T, 8 / kElems<T>, false>;
    switch (vpt) {
        case 1: return norm_fwd_kernel<T, 1, true>;
        case 2: return norm_fwd_kernel<T, 2, true>;
        case 3: return norm_fwd_kernel<T, 3, true>;
        case 4: return norm_fwd_kernel<T, 4, true>;
        default:   // fp32 only: a 16-bit row needs four words at most
            if constexpr (sizeof(T) == 4) return norm_fwd_kernel<T, 8, true>;
            else return nullptr;
    }
}
template <typename T>
auto bwd_kernel(int vpt, bool vec) -> void (*)(NormBwd) {
    if (vpt == 0) return norm_bwd_general_kernel<T>;
    if (!vec) return norm_bwd_kernel<T, 8 / kElems<T>, false>;
    switch (vpt) {
        case 1: return norm_bwd_kernel<T, 1, true>;
        case 2: return norm_bwd_kernel<T, 2, true>;
        case 3: return norm_bwd_kernel<T, 3, true>;
        case 4: return norm_bwd_kernel<T, 4, true>;
        default:
            if constexpr (sizeof(T) == 4) return norm_bwd_kernel<T, 8, true>;
            else return nullptr;
    }
}

moe_status check(const moe_norm_config *c) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->T < 0 || c->d < 1) return MOE_ERR_INVALID_ARG;
    if (c->kind != MOE_NORM_LAYER && c->kind != MOE_NORM_RMS) return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_BF16 && c->dtype != MOE_F32 && c->dtype != MOE_F16) return MOE_ERR_INVALID_ARG;
    if (c->w_dtype != c->dtype && c->w_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
    if (!(c->eps >= 0.f) || c->eps > 3.0e38f) return MOE_ERR_INVALID_ARG;
    if (c->d > MOE_NORM_MAX_WIDTH || c->T >= (int64_t)1 << 40) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_norm_workspace_size(const moe_norm_config *c, size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status st = check(c);
    if (st != MOE_OK) return st;
    *bytes = (size_t)std::min<int64_t>(kBwdBlocks, c->T) * 2 * (size_t)c->d * sizeof(float);
    return MOE_OK;
}

moe_status moe_norm_forward(const moe_norm_config *c, const void *x, const void *residual, const void *weight,
                            const void *bias, void *h, void *y, float *mean, float *rstd, void *stream) {
    const moe_status st = check(c);
    if (st != MOE_OK) return st;
    if ((residual == nullptr) != (h == nullptr)) return MOE_ERR_INVALID_ARG;
    if (c->T == 0) return MOE_OK;
    if (!x || !weight || !y) return MOE_ERR_INVALID_ARG;
    if (!device_error_word()) return MOE_ERR_CUDA;
    const int E = 16 / elem_size(c->dtype);
    const bool vec = c->d % E == 0 && aligned16(x) && aligned16(residual) && aligned16(weight) && aligned16(bias) &&
                     aligned16(h) && aligned16(y);
    const Spread sp = spread(c->d, E, vec);
    const NormFwd a{x, residual, weight, bias, h, y, mean, rstd, c->T, c->d, sp.W, sp.groups,
                    c->kind == MOE_NORM_LAYER, c->w_dtype == MOE_F32, c->eps};
    const int threads = sp.groups * sp.W * 32;
    const int64_t rows = (c->T + sp.groups - 1) / sp.groups;
    const int grid = (int)std::min<int64_t>(rows, (int64_t)num_sms() * std::max(1, 2048 / threads));
    auto kern = c->dtype == MOE_BF16  ? fwd_kernel<__nv_bfloat16>(sp.vpt, vec)
                : c->dtype == MOE_F16 ? fwd_kernel<__half>(sp.vpt, vec)
                                      : fwd_kernel<float>(sp.vpt, vec);
    const cudaError_t e = launch_kernel(kern, grid, threads, 0, static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_norm_backward(const moe_norm_config *c, const void *h, const void *weight, const float *mean,
                             const float *rstd, const void *dy, const void *dh, void *dx, float *dweight,
                             float *dbias, void *ws, size_t ws_bytes, void *stream) {
    const moe_status st = check(c);
    if (st != MOE_OK) return st;
    const bool layer = c->kind == MOE_NORM_LAYER;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c->T == 0) {   // no tokens: the gradients of the parameters are zero
        cudaError_t e = dweight ? cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)c->d, s) : cudaSuccess;
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * (size_t)c->d, s);
        return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    if (!h || !weight || !rstd || !dy || !dx || layer != (mean != nullptr)) return MOE_ERR_INVALID_ARG;
    const bool params = dweight || dbias;
    const int E = 16 / elem_size(c->dtype);
    const bool vec = c->d % E == 0 && aligned16(h) && aligned16(weight) && aligned16(dy) && aligned16(dh) && aligned16(dx);
    const Spread sp = spread(c->d, E, vec);
    const int blocks = (int)std::min<int64_t>(kBwdBlocks, (c->T + sp.groups - 1) / sp.groups);
    if (params && (!ws || ws_bytes < (size_t)std::min<int64_t>(kBwdBlocks, c->T) * 2 * (size_t)c->d * sizeof(float) ||
                   (reinterpret_cast<uintptr_t>(ws) & 255)))
        return MOE_ERR_WORKSPACE;
    if (!device_error_word()) return MOE_ERR_CUDA;
    float *part = params ? static_cast<float *>(ws) : nullptr;
    const NormBwd a{h, weight, dy, dh, mean, rstd, dx, part, c->T, c->d, sp.W, sp.groups, c->w_dtype == MOE_F32,
                    dbias != nullptr};
    const size_t smem = sp.groups > 1 || sp.vpt == 0 ? 2 * sizeof(float) * (size_t)c->d : 0;
    auto kern = c->dtype == MOE_BF16  ? bwd_kernel<__nv_bfloat16>(sp.vpt, vec)
                : c->dtype == MOE_F16 ? bwd_kernel<__half>(sp.vpt, vec)
                                      : bwd_kernel<float>(sp.vpt, vec);
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = launch_kernel(kern, blocks, sp.groups * sp.W * 32, smem, s, a);
    if (e == cudaSuccess && params)
        e = launch_kernel(norm_param_kernel, dim3((c->d + 31) / 32, dbias ? 2 : 1), 1024, 0, s,
                          static_cast<const float *>(part), blocks, (int)c->d, dweight, dbias);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
