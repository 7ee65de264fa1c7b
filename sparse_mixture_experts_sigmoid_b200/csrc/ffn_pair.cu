// The products of the dense gated feed-forward block on two SMs per tile
// (tcgen05.mma.cta_group::2, M = 256), bf16 or fp16 operands, fp32
// accumulation:
//
//   GATED  : u = x Wg^T, v = x Wu^T;  act(u) v is stored (and u, v for training)
//   STORE  : C = A B, rounded once: the down projection, dx (two K ranges, du Wg
//            + dv Wu) and the weight gradients
//   DGATED : r = dy Wd;  du = r v act'(u), dv = r act(u), from the kept u, v
//
// Bound by the tensor cores for all but short inputs, so the kernel is one
// persistent pipeline whose MMAs do not pause between tiles: a ring of K
// blocks of 64 (128 bytes) filled by TMA, two accumulators in TMEM (the
// epilogue of a tile runs under the MMAs of the next), and outputs that leave
// through shared memory by TMA stores, which also cut the edges off.  Each CTA
// of a pair stages its own 128 rows of A and its own half of B's columns, 32 KB
// per K block for 256 x 256 x 64 products.
//
// An operand is K-major (rows of the reduction, as x and the weights lie for
// the forward pass) or MN-major (the reduction runs over its rows: Wd and Wg,
// Wu in the backward pass, and both operands of the weight gradients, whose
// reduction runs over the tokens); the tensor map's boxes differ, the bytes of
// the operand are never moved or transposed in memory.
//
// Every mbarrier wait is bounded as in the grouped kernels.
#include <algorithm>

#include "ffn.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace ffn {
namespace {

using namespace tc;

constexpr int kBM = 256;                   // rows of a pair's tile
constexpr int kBK = 64;                    // 16-bit elements of a 128-byte row
constexpr int kAStage = 128 * 128;         // this CTA's A of one K block
constexpr int kAtom = 8192;                // an MN-major atom: 64 k-rows x 128 bytes
constexpr int kEpiWarps = 8;               // two per TMEM lane quarter
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr int kTmemCols = 512;
constexpr int kBox = 32 * 128;             // a store's box: 32 rows x 64 columns
constexpr int kMaxStages = 8;
constexpr int kSmemMax = 232448;

struct Ctrl {
    uint64_t full[kMaxStages];    // even CTA: operands of a K block landed (both CTAs)
    uint64_t empty[kMaxStages];   // both: the MMAs of a K block are done
    uint64_t tfull[2];            // both: accumulator ready
    uint64_t tempty[2];           // even CTA: accumulator released by both epilogues
    uint64_t done;                // both: all MMAs of the pair completed
    uint64_t kept[kEpiWarps];     // DGATED: an epilogue warp's u and v landed
    uint32_t tmem_base;
    int abort;
};

template <int EPI>
constexpr int epi_bytes() {
    return kEpiWarps * kBox * (EPI == DGATED ? 2 : 1);
}
template <int EPI, int BN>
constexpr int stages() {
    const int s = (kSmemMax - 1024 - (int)sizeof(Ctrl) - epi_bytes<EPI>()) / (kAStage + BN * 64);
    return s > kMaxStages ? kMaxStages : s;
}

struct Params {
    int M, N, K;       // output rows and columns; K per range
    int ranges;        // K ranges (A0 B0, then A1 B1)
    int halves;        // STORE: products that share B and the shape (A0 -> C0, A1 -> C1)
    int mt, nt;        // tiles of one half
    int act;           // moe_ffn_act
    uint32_t fmt;      // operand format of the instruction descriptor: 0 fp16, 1 bf16
    bool keep;         // GATED: store u and v as well
    uint32_t *err;
};

struct Maps {
    CUtensorMap a0, a1, b0, b1;   // operands
    CUtensorMap c0, c1, c2;       // outputs: C0 (act, du), C1 (u, dv), C2 (v)
    CUtensorMap u, v;             // DGATED: the kept pre-activations
};

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, const void *src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The committed stores have read their shared memory / have been written.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ uint64_t desc_mn(const void *p) {
    const uint32_t a = smem_u32(p);
    return (uint64_t)((a & 0x3FFFF) >> 4) | ((uint64_t)(kAtom >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Tile id -> (half, m, n).  Row tiles run in groups of eight with the column
// tiles outside them, so that the pairs at work at one time read about as many
// rows of A as of B and share them through L2.
struct Tile {
    int half, m, n;
};
__device__ __forceinline__ Tile tile_of(int id, const Params &p) {
    const int per = p.mt * p.nt;
    Tile t;
    t.half = id / per;
    id -= t.half * per;
    const int g = id / (8 * p.nt), first = 8 * g, size = min(p.mt - first, 8);
    id -= g * 8 * p.nt;
    t.n = id / size;
    t.m = first + id - t.n * size;
    return t;
}

// A warp's box of 32 rows x 64 columns in shared memory, 128-byte swizzle: the
// 16-byte word j of row i at i * 128 + 16 * (j ^ (i mod 8)).
__device__ __forceinline__ uint4 *box_word(uint8_t *box, int j) {
    const int i = threadIdx.x & 31;
    return reinterpret_cast<uint4 *>(box + i * 128 + ((j ^ (i & 7)) << 4));
}

template <bool A_MN, bool B_MN, int EPI, int BN>
__global__ void __launch_bounds__(kThreads, 1) ffn_pair_kernel(const __grid_constant__ Maps maps, Params p) {
    constexpr int kStages = stages<EPI, BN>();
    constexpr int kBStage = BN * 64;       // this CTA's half of B of one K block
    constexpr int kCols = EPI == GATED ? BN / 2 : BN;   // output columns of a tile
    constexpr int kWarpCols = kCols / 2;   // of one epilogue warp
    static_assert(kWarpCols % 64 == 0, "whole boxes");

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = smem, *sB = sA + kStages * kAStage, *sEpi = sB + kStages * kBStage;
    Ctrl *ctrl = reinterpret_cast<Ctrl *>(sEpi + epi_bytes<EPI>());
    volatile int *abort = &ctrl->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool lead = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ctrl->full[s], 1);
            mbar_init(&ctrl->empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&ctrl->tfull[a], 1);
            mbar_init(&ctrl->tempty[a], 2 * kEpiWarps);
        }
        for (int w = 0; w < kEpiWarps; ++w) mbar_init(&ctrl->kept[w], 1);
        mbar_init(&ctrl->done, 1);
        ctrl->abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc2(&ctrl->tmem_base, kTmemCols);
    if (warp == kTmaWarp && lane == 0) {
        prefetch_tmap(&maps.a0);
        prefetch_tmap(&maps.b0);
        prefetch_tmap(&maps.c0);
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync_all();   // both CTAs' barriers exist before any remote arrive
    pdl_launch_dependents();

    const uint32_t tmem = ctrl->tmem_base;
    const int total = p.halves * p.mt * p.nt;
    const int kr = (p.K + kBK - 1) / kBK, nk = p.ranges * kr;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (warp == kTmaWarp) {
        if (lane == 0) {
            constexpr uint32_t kTx = 2u * (kAStage + kBStage);   // of both CTAs
            const uint32_t full_lead = mapa_shared(&ctrl->full[0], 0);
            uint32_t it = 0;
            bool ok = true;
            for (int id = pair; id < total && ok; id += npairs) {
                const Tile t = tile_of(id, p);
                const int m0 = t.m * kBM + (int)rank * 128;
                // GATED: the even CTA holds the gate's rows, the odd one the up projection's
                const int n0 = EPI == GATED ? t.n * kCols : t.n * BN + (int)rank * (BN / 2);
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!wait_bar(&ctrl->empty[s], ((it / kStages) & 1) ^ 1, abort, p.err)) {
                        ok = false;
                        break;
                    }
                    if (lead) mbar_expect_tx(&ctrl->full[s], kTx);
                    const uint32_t fb = full_lead + s * (uint32_t)sizeof(uint64_t);
                    const bool second = kb >= kr;
                    const int k0 = (second ? kb - kr : kb) * kBK;
                    const CUtensorMap *ma = second || t.half ? &maps.a1 : &maps.a0;
                    const CUtensorMap *mb = (EPI == GATED ? !lead : second) ? &maps.b1 : &maps.b0;
                    uint8_t *a = sA + s * kAStage, *b = sB + s * kBStage;
                    if constexpr (A_MN) {
                        tma_load_2d_pair(ma, a, fb, m0, k0);
                        tma_load_2d_pair(ma, a + kAtom, fb, m0 + 64, k0);
                    } else {
                        tma_load_2d_pair(ma, a, fb, k0, m0);
                    }
                    if constexpr (B_MN) {
#pragma unroll
                        for (int j = 0; j < BN / 128; ++j) tma_load_2d_pair(mb, b + j * kAtom, fb, n0 + 64 * j, k0);
                    } else {
                        tma_load_2d_pair(mb, b, fb, k0, n0);
                    }
                }
            }
            if (!ok) {
                // aborting: let this CTA's copies land before it leaves
                for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0; j < it; ++j) {
                    const uint64_t t0 = globaltimer();
                    while (!mbar_try_wait(&ctrl->empty[j % kStages], (j / kStages) & 1) &&
                           globaltimer() - t0 < 100000000ull) {
                    }
                }
            }
        }
    } else if (warp == kMmaWarp) {
        if (lead) {   // the whole warp: one lane's instructions take effect
            const bool mine = lane == 0;
            const uint32_t idesc = (1u << 4) | (p.fmt << 7) | (p.fmt << 10) | ((uint32_t)A_MN << 15) |
                                   ((uint32_t)B_MN << 16) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
            uint32_t it = 0, tc = 0;
            bool ok = true;
            for (int id = pair; id < total && ok; id += npairs, ++tc) {
                const uint32_t acc = tc & 1;
                if (!wait_bar(&ctrl->tempty[acc], ((tc >> 1) & 1) ^ 1, abort, p.err)) break;
                tc_fence_after();
                const uint32_t d = tmem + acc * BN;
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int s = it % kStages;
                    const uint32_t ph = (it / kStages) & 1;
                    // the operands of both CTAs have landed
                    if (!mbar_try_wait(&ctrl->full[s], ph) && !wait_bar(&ctrl->full[s], ph, abort, p.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t ad = A_MN ? desc_mn(sA + s * kAStage + kk * 2048)
                                                 : smem_desc(sA + s * kAStage) + 2 * kk;
                        const uint64_t bd = B_MN ? desc_mn(sB + s * kBStage + kk * 2048)
                                                 : smem_desc(sB + s * kBStage) + 2 * kk;
                        mma_if<2, kF16>(mine, d, ad, bd, idesc, (kb | kk) != 0);
                    }
                    mma_commit2_if(mine, &ctrl->empty[s], 0x3);
                }
                if (ok) mma_commit2_if(mine, &ctrl->tfull[acc], 0x3);
            }
            mma_commit2_if(mine, &ctrl->done, 0x3);
        }
    } else {
        const uint32_t tempty_lead = mapa_shared(&ctrl->tempty[0], 0);
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const int cw = (warp >> 2) * kWarpCols;   // this warp's first output column of the tile
        uint8_t *box = sEpi + warp * (epi_bytes<EPI>() / kEpiWarps), *box2 = box + kBox;
        uint32_t tc = 0;
        [[maybe_unused]] uint32_t loads = 0;      // DGATED: u, v box loads issued so far
        // stores the packed 64 columns of this warp's 32 rows (8 words a row)
        auto put = [&](const CUtensorMap *m, const uint4 (&w)[8], int c, int r) {
            if (lane == 0) bulk_wait_read();   // the previous store has left the box
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) *box_word(box, j) = w[j];
            fence_proxy_async();
            __syncwarp();
            if (lane == 0 && r < p.M && c < p.N) {
                tma_store_2d(m, box, c, r);
                bulk_commit();
            }
        };
        auto pack = [&](const float (&f)[64], uint4 (&w)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = make_uint4(pack2(f[8 * j], f[8 * j + 1], p.fmt), pack2(f[8 * j + 2], f[8 * j + 3], p.fmt),
                                  pack2(f[8 * j + 4], f[8 * j + 5], p.fmt), pack2(f[8 * j + 6], f[8 * j + 7], p.fmt));
        };
        auto read64 = [&](uint32_t at, float (&f)[64]) {
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld16(at + 16 * q, *reinterpret_cast<float(*)[16]>(&f[16 * q]));
            tmem_wait_ld();
        };
        // DGATED: the kept u and v of 64 columns from c into the warp's two boxes
        auto ask = [&](int c, int r) {
            if (lane == 0) {
                bulk_wait_read();
                mbar_expect_tx(&ctrl->kept[warp], 2 * kBox);
                tma_load_2d(&maps.u, box, &ctrl->kept[warp], c, r);
                tma_load_2d(&maps.v, box2, &ctrl->kept[warp], c, r);
            }
            ++loads;
        };
        for (int id = pair; id < total; id += npairs, ++tc) {
            const Tile t = tile_of(id, p);
            const uint32_t acc = tc & 1;
            const int r = t.m * kBM + (int)rank * 128 + (warp & 3) * 32, c0 = t.n * kCols + cw;
            if constexpr (EPI == DGATED) {
                if (r < p.M && c0 < p.N) ask(c0, r);
            }
            if (!wait_bar(&ctrl->tfull[acc], (tc >> 1) & 1, abort, p.err)) {
                if constexpr (EPI == DGATED) {
                    // the copies into this warp's boxes land before the CTA leaves
                    const uint64_t t0 = globaltimer();
                    while (loads && !mbar_try_wait(&ctrl->kept[warp], (loads - 1) & 1) &&
                           globaltimer() - t0 < 100000000ull) {
                    }
                }
                break;
            }
            tc_fence_after();
            const uint32_t tb = tmem + acc * BN + lane_base;
            if (r < p.M && c0 < p.N) {
                if constexpr (EPI == STORE) {
                    const CUtensorMap *mc = t.half ? &maps.c1 : &maps.c0;
#pragma unroll 1
                    for (int q = 0; q < kWarpCols; q += 64) {
                        if (c0 + q >= p.N) break;
                        float f[64];
                        uint4 w[8];
                        read64(tb + cw + q, f);
                        pack(f, w);
                        put(mc, w, c0 + q, r);
                    }
                } else if constexpr (EPI == GATED) {
                    float g[64], u[64];
                    uint4 w[8];
                    read64(tb + cw, g);
                    read64(tb + BN / 2 + cw, u);
                    if (p.keep) {
                        pack(g, w);
                        put(&maps.c1, w, c0, r);
                        pack(u, w);
                        put(&maps.c2, w, c0, r);
                    }
                    if (p.act == MOE_ACT_SILU) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) g[i] = silu_f(g[i]) * u[i];
                    } else {
#pragma unroll
                        for (int i = 0; i < 64; ++i) g[i] = gelu_tanh_f(g[i]) * u[i];
                    }
                    pack(g, w);
                    put(&maps.c0, w, c0, r);
                } else {
#pragma unroll 1
                    for (int q = 0; q < kWarpCols; q += 64) {
                        if (c0 + q >= p.N) break;
                        if (q) ask(c0 + q, r);
                        if (!wait_bar(&ctrl->kept[warp], (loads - 1) & 1, abort, p.err)) break;
                        float f[64];
                        read64(tb + cw + q, f);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            uint4 wu = *box_word(box, j), wv = *box_word(box2, j);
                            uint32_t *pu = reinterpret_cast<uint32_t *>(&wu), *pv = reinterpret_cast<uint32_t *>(&wv);
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                const float2 uu = unpack2(pu[z], p.fmt), vv = unpack2(pv[z], p.fmt);
                                float a[2], da[2];
                                act_grad(p.act, uu.x, a[0], da[0]);
                                act_grad(p.act, uu.y, a[1], da[1]);
                                const float r0 = f[8 * j + 2 * z], r1 = f[8 * j + 2 * z + 1];
                                pu[z] = pack2(r0 * vv.x * da[0], r1 * vv.y * da[1], p.fmt);
                                pv[z] = pack2(r0 * a[0], r1 * a[1], p.fmt);
                            }
                            *box_word(box, j) = wu;
                            *box_word(box2, j) = wv;
                        }
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&maps.c0, box, c0 + q, r);
                            tma_store_2d(&maps.c1, box2, c0 + q, r);
                            bulk_commit();
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (lead) mbar_arrive(&ctrl->tempty[acc]);
                else mbar_arrive_remote_relaxed(tempty_lead + acc * (uint32_t)sizeof(uint64_t));
            }
        }
        if (lane == 0) bulk_wait_all();
    }

    // every MMA of the pair has completed (its arrivals on this CTA's barriers
    // included) before the pair meets for the last time and frees TMEM
    if (threadIdx.x == 0) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(&ctrl->done, 0) && globaltimer() - t0 < kWaitLimitNs) {
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc2(tmem, kTmemCols);
}

// ------------------------------------------------------------------ host side

// A row-major matrix of 16-bit elements, boxes of 64 columns (128 bytes, 128-byte
// swizzle) by box_rows; what lies outside reads as zero and is not written.
bool make_map16(CUtensorMap *m, const Matrix &x, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn || !x.base) return false;
    cuuint64_t dims[2] = {(cuuint64_t)x.cols, (cuuint64_t)x.rows};
    cuuint64_t strides[1] = {(cuuint64_t)x.ld * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(x.base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool A_MN, bool B_MN, int EPI, int BN>
cudaError_t launch(const Gemm &g, cudaStream_t s) {
    constexpr int kCols = EPI == GATED ? BN / 2 : BN;
    Maps maps{};
    // operand boxes: K-major 128 (A) or BN / 2 (B) rows of 64 k; MN-major 64 k-rows of 64 columns
    bool ok = make_map16(&maps.a0, g.a0, A_MN ? 64 : 128) && make_map16(&maps.b0, g.b0, B_MN ? 64 : BN / 2) &&
              make_map16(&maps.c0, g.c0, 32);
    if (ok && g.a1.base) ok = make_map16(&maps.a1, g.a1, A_MN ? 64 : 128);
    if (ok && g.b1.base) ok = make_map16(&maps.b1, g.b1, B_MN ? 64 : BN / 2);
    if (ok && g.c1.base) ok = make_map16(&maps.c1, g.c1, 32);
    if (ok && g.c2.base) ok = make_map16(&maps.c2, g.c2, 32);
    if (ok && EPI == DGATED) ok = make_map16(&maps.u, g.u, 32) && make_map16(&maps.v, g.v, 32);
    if (!ok) return cudaErrorInvalidValue;
    Params p{};
    p.M = (int)g.M;
    p.N = g.N;
    p.K = (int)g.K;
    p.ranges = g.ranges;
    p.halves = g.halves;
    p.mt = (int)((g.M + kBM - 1) / kBM);
    p.nt = (g.N + kCols - 1) / kCols;
    p.act = g.act;
    p.fmt = g.bf16 ? 1u : 0u;
    p.keep = g.c1.base != nullptr;
    p.err = g.err;
    const size_t smem = 1024 + (size_t)stages<EPI, BN>() * (kAStage + BN * 64) + epi_bytes<EPI>() + sizeof(Ctrl);
    auto kern = ffn_pair_kernel<A_MN, B_MN, EPI, BN>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)p.halves * p.mt * p.nt;
    const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(num_sms() / 2, tiles));
    return launch_kernel_pair(kern, 2 * pairs, kThreads, smem, s, maps, p);
}

// Whether tiles of 128 columns end sooner than tiles of 256: their rounds over
// the pairs, at (per K block) 512 and 256 cycles of MMA and a tile's fixed cost.
// The narrow tiles read half as much again per product, which does not show
// while few pairs are at work; for full rounds the wide ones win.
bool narrow_tiles(const Gemm &g) {
    const int64_t pairs = num_sms() / 2, mt = (g.M + kBM - 1) / kBM * g.halves;
    const int64_t nk = (int64_t)g.ranges * ((g.K + kBK - 1) / kBK);
    auto rounds = [&](int bn) { return (mt * ((g.N + bn - 1) / bn) + pairs - 1) / pairs; };
    return rounds(128) * (nk * 290 + 2000) < rounds(256) * (nk * 512 + 3000);
}

}  // namespace

cudaError_t launch_pair_gemm(const Gemm &g, cudaStream_t s) {
    switch (g.kind) {
        case GATED: return launch<false, false, GATED, 256>(g, s);
        case DGATED:
            return narrow_tiles(g) ? launch<false, true, DGATED, 128>(g, s) : launch<false, true, DGATED, 256>(g, s);
        default:
            if (narrow_tiles(g)) {
                if (g.a_mn) return launch<true, true, STORE, 128>(g, s);
                if (g.b_mn) return launch<false, true, STORE, 128>(g, s);
                return launch<false, false, STORE, 128>(g, s);
            }
            if (g.a_mn) return launch<true, true, STORE, 256>(g, s);
            if (g.b_mn) return launch<false, true, STORE, 256>(g, s);
            return launch<false, false, STORE, 256>(g, s);
    }
}

}  // namespace ffn
}  // namespace moe
