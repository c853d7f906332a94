// k3moe_linear.cu -- y = act(x W^T + bias) + residual, x [T][K] and W [N][K] bf16 (the
// projections of a decoder layer around its token mixer).
//
// Two kernels:
//   linear_rows_kernel   a few tokens: the weight stream, one warp a row, plain FMAs;
//   linear_tc_kernel     all else on tcgen05, weights as the M side (128 rows a block, 256
//                        a pair of blocks), tokens as the N side.  With the weights on M
//                        a thread of the epilogue owns one output column and a warp's
//                        lanes 32 neighbouring ones, so bias is a register and every
//                        load of the residual and store of y is contiguous over the
//                        lanes, whatever y's row stride: no staging through shared memory.
#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>

#include "k3moe_internal.cuh"
#include "k3moe_tc_warp.cuh"

namespace k3moe {
namespace {

// The activations in float, branch-free (256 of them a thread in a tile's epilogue), each within a few
// units of its own last place, and in a tail within as many as a rounding of z would make of it:
//   sigmoid  1 / (1 + e), e = exp(-z); past z = -87 the division gives 0;
//   gelu     z Phi(z), with Phi(-|z|) = exp(-z^2 / 2) R(t), t = 1 / (1 + 0.3 |z|): R = t times a
//            polynomial, fitted here to least relative error over |z| <= 14 (1.5e-7; all of the float
//            arithmetic within (4 + 0.63 z^2) 2^-23), so that the far negative side is a product of relative
//            accuracy, not a difference;
//   logsigmoid  min(z, 0) - log(1 + e), e = exp(-|z|), with log(1 + e) = 2 atanh(s),
//            s = e / (2 + e) <= 1/3, by atanh's series to s^15: relative error 2e-9 and the rounding.
template <int ACT>
__device__ __forceinline__ float lin_act(float z)
{
    if (ACT == K3MOE_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if (ACT == K3MOE_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));
    if (ACT == K3MOE_ACT_SIGMOID) return __fdividef(1.0f, 1.0f + __expf(-z));
    if (ACT == K3MOE_ACT_GELU) {
        const float t = __fdividef(1.0f, fmaf(0.3f, fabsf(z), 1.0f));
        float p = fmaf(0.03567477f, t, -0.15720306f);
        p = fmaf(p, t, 0.20635349f);
        p = fmaf(p, t, -0.053683624f);
        p = fmaf(p, t, 0.12856162f);
        p = fmaf(p, t, 0.09991349f);
        p = fmaf(p, t, 0.12075396f);
        p = fmaf(p, t, 0.1196293f);
        float e;                                             // exp(-z^2 / 2), as a power of 2
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * z * -0.72134752f));
        const float tail = p * t * e;
        return z * (z > 0.0f ? 1.0f - tail : tail);
    }
    if (ACT == K3MOE_ACT_LOGSIGMOID) {
        const float e = __expf(-fabsf(z));
        const float s = __fdividef(e, 2.0f + e), w = s * s;
        float p = fmaf(w, 1.0f / 15.0f, 1.0f / 13.0f);
        p = fmaf(p, w, 1.0f / 11.0f);
        p = fmaf(p, w, 1.0f / 9.0f);
        p = fmaf(p, w, 1.0f / 7.0f);
        p = fmaf(p, w, 1.0f / 5.0f);
        p = fmaf(p, w, 1.0f / 3.0f);
        p = fmaf(p, w, 1.0f);
        return (z < 0.0f ? z : (z != z ? z : 0.0f)) - 2.0f * s * p;
    }
    return z;
}

// f(integral constant act) for a runtime act.
template <int N> struct ActC { static constexpr int value = N; };
template <typename F>
__device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case K3MOE_ACT_RELU: f(ActC<K3MOE_ACT_RELU>{}); break;
    case K3MOE_ACT_SILU: f(ActC<K3MOE_ACT_SILU>{}); break;
    case K3MOE_ACT_GELU: f(ActC<K3MOE_ACT_GELU>{}); break;
    case K3MOE_ACT_SIGMOID: f(ActC<K3MOE_ACT_SIGMOID>{}); break;
    case K3MOE_ACT_LOGSIGMOID: f(ActC<K3MOE_ACT_LOGSIGMOID>{}); break;
    default: f(ActC<K3MOE_ACT_NONE>{}); break;
    }
}

__device__ __forceinline__ float lin_residual(const LinearArgs &a, int t, int n)
{
    if (!a.residual) return 0.0f;
    const size_t r = (size_t)t * a.residual_stride + n;
    return a.f32 ? reinterpret_cast<const float *>(a.residual)[r]
                 : bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(a.residual)[r]);
}

// One output, rounded once.
__device__ __forceinline__ void lin_put(const LinearArgs &a, int t, int n, float z)
{
    const size_t o = (size_t)t * a.y_stride + n;
    if (a.f32)
        reinterpret_cast<float *>(a.y)[o] = z;
    else
        reinterpret_cast<__nv_bfloat16 *>(a.y)[o] = __float2bfloat16_rn(z);
}

// ---------------------------------------------------------------- a few tokens
// One warp an output column at a time, its weight row read with 16-byte loads, eight in
// flight a lane, against the tokens held in shared memory; sums in float, per lane in
// chunk order and then over the warp by a fixed butterfly.  Bound by the weights' bytes: one
// token, 7168 x 3584 with SiLU, takes 8.5 us a call with the weights in the L2 and 10.5 with them
// in DRAM, 4.9 TB/s (11.5 without asking for the first row under the kernel before).
constexpr int kLrThreads = 256, kLrWarps = kLrThreads / 32, kLrDeep = 8;
constexpr size_t kLrSmem = 200 * 1024;
// Weights up to which three and four tokens go this way; one and two always do.  This kernel
// against the tensor cores, us: four tokens, K 2048, N 2048 6.1, 11.7, N 4096 9.1, 9.2; K = N =
// 4096 14.2, 10.9; two tokens there 8.8, 10.9 and K 7168, N 3584 13.4, 13.5; one 11.4, 13.6.
constexpr long long kLrFour = 8 << 20;

template <int NT>
__global__ void __launch_bounds__(kLrThreads) linear_rows_kernel(const LinearArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    {   // the warp's first row to the L2 under the kernel before (asked for, not read: it may still be written)
        const int n = blockIdx.x * kLrWarps + warp;
        if (lane == 0 && n < a.N) prefetch_bulk(a.w + (size_t)n * a.K, (uint32_t)a.K * 2);
    }
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) uint4 xsm[];         // NT x K bf16
    const int nchunk = a.K / 8;
    for (int q = threadIdx.x; q < NT * nchunk; q += kLrThreads) {
        const int t = q / nchunk, c = q % nchunk;
        xsm[q] = t < a.T ? *(reinterpret_cast<const uint4 *>(a.x + (size_t)t * a.x_stride) + c)
                         : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    for (int n = blockIdx.x * kLrWarps + warp; n < a.N; n += gridDim.x * kLrWarps) {
        const uint4 *wr = reinterpret_cast<const uint4 *>(a.w + (size_t)n * a.K);
        float acc[NT];
#pragma unroll
        for (int t = 0; t < NT; t++) acc[t] = 0.0f;
        for (int c0 = lane; c0 < nchunk; c0 += 32 * kLrDeep) {
            uint4 wv[kLrDeep];
#pragma unroll
            for (int j = 0; j < kLrDeep; j++)
                wv[j] = c0 + 32 * j < nchunk ? __ldcs(wr + c0 + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < kLrDeep; j++) {
                const int c = c0 + 32 * j;
                if (c >= nchunk) break;
                const uint32_t wu[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w};
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    const uint4 xv = xsm[t * nchunk + c];
                    const uint32_t xu[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        acc[t] = fmaf(__uint_as_float(xu[r] << 16), __uint_as_float(wu[r] << 16), acc[t]);
                        acc[t] = fmaf(__uint_as_float(xu[r] & 0xFFFF0000u), __uint_as_float(wu[r] & 0xFFFF0000u),
                                      acc[t]);
                    }
                }
            }
        }
        const float b = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
        for (int t = 0; t < NT; t++) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
        }
        float z = acc[0];
#pragma unroll
        for (int t = 1; t < NT; t++) z = lane == t ? acc[t] : z;
        if (lane < NT && lane < a.T)
            with_act(a.act, [&](auto act) {
                lin_put(a, lane, n, lin_act<decltype(act)::value>(z + b) + lin_residual(a, lane, n));
            });
    }
}

// ---------------------------------------------------------------- tensor cores
constexpr int kLtBK = 64;                                    // K columns a stage: one 128-byte swizzled row
constexpr int kLtABytes = 128 * kLtBK * 2;                   // a block's weight tile
constexpr int kLtRing = 192 * 1024, kLtRing2 = 96 * 1024;    // the stage ring: one block an SM, or two
constexpr int kLtMaxStg = 10;
constexpr int kLtWarpProd = 0, kLtWarpMma = 1, kLtWarpEpi0 = 2, kLtNumEpi = 8;
constexpr int kLtThreads = (kLtWarpEpi0 + kLtNumEpi) * 32;   // 320

struct LinTile {
    int bn;          // tokens a tile (of both blocks of a pair)
    int n_rb, n_tt;  // weight row blocks (128 x CG rows) and token tiles
    int P;           // K parts: blocks of a cluster that share one tile
    int per_sm;      // blocks an SM: 1, or 2 with half the ring and half the tensor memory
    int acc;         // columns from one accumulator to the next (two, or one when P > 1)
    int cols;        // columns of tensor memory
    int nks;         // K stages in all
    int nstg, stage_bytes;
    int group;       // weight row blocks visited together, for the L2
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The cluster address of a shared-memory address in block `rank`.
__device__ __forceinline__ uint32_t mapa(uint32_t a, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
// Tile copy (by one lane of a converged warp, as tma2d_warp) whose bytes are counted on a
// barrier of either block of the pair.
__device__ __forceinline__ void tma2d_pair_warp(void *dst, const CUtensorMap *m, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
        "{%2, %3}], [%4];\n\t}" ::"r"(saddr(dst)),
        "l"(m), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
// The pair's forms of umma_warp and umma_commit_warp; the commit arrives on the barrier at
// this address in both blocks once the issued MMAs are done.
__device__ __forceinline__ void umma_pair_warp(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kDescSw128)
        : "memory");
}
__device__ __forceinline__ void umma_commit_pair_warp(uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            saddr(bar)),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void mb_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Sixteen tokens' accumulators, the first `left` of them wanted, of a lane's output column.
template <typename Y>
__device__ __forceinline__ void lin_column(const LinearArgs &a, uint32_t taddr, int t0, int left, int col, float b)
{
    constexpr bool kF32 = sizeof(Y) == 4;
    float r[16];
    if (a.residual) {                                        // all loaded before any is stored (y may be the residual)
        const Y *p = reinterpret_cast<const Y *>(a.residual) + (size_t)t0 * a.residual_stride + col;
#pragma unroll
        for (int j = 0; j < 16; j++, p += a.residual_stride) {
            r[j] = 0.0f;
            if (j < left) r[j] = kF32 ? (float)*reinterpret_cast<const float *>(p) : bf16_bits_to_f32((uint32_t)*p);
        }
    }
    uint32_t v[16];
    tmem_ld16_nowait(taddr, v);
    tmem_wait_ld();
    with_act(a.act, [&](auto act) {
#pragma unroll
        for (int j = 0; j < 16; j++) v[j] = __float_as_uint(lin_act<decltype(act)::value>(__uint_as_float(v[j]) + b));
    });
    if (a.residual)
#pragma unroll
        for (int j = 0; j < 16; j++) v[j] = __float_as_uint(__uint_as_float(v[j]) + r[j]);
    Y *p = reinterpret_cast<Y *>(a.y) + (size_t)t0 * a.y_stride + col;
#pragma unroll
    for (int j = 0; j < 16; j++, p += a.y_stride) {
        if (j >= left) break;
        if (kF32) {
            *reinterpret_cast<uint32_t *>(p) = v[j];
        } else {
            const __nv_bfloat16 w = __float2bfloat16_rn(__uint_as_float(v[j]));
            *reinterpret_cast<__nv_bfloat16 *>(p) = w;
        }
    }
}

// Sixteen tokens' accumulators of a warp's 32 output columns (lane = column) through the
// epilogue.  In bf16, with rows that start on a word, neighbouring lanes trade a token
// each, so that a store takes two columns of one token from a lane (half the stores, 64
// contiguous bytes of two tokens each); the residual is read the same way.
__device__ __forceinline__ void lin_chunk(const LinearArgs &a, uint32_t taddr, int t0, int left, int col, bool pairs,
                                          float b)
{
    const bool odd = threadIdx.x & 1;
    uint32_t v[16];
    if (pairs) {
        const int c2 = col & ~1, mine = odd ? 1 : 0;             // columns c2, c2 + 1 of tokens j + mine
        const bool in0 = c2 < a.N, in1 = c2 + 1 < a.N;
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            r[j] = 0;
            if (a.residual && in0 && 2 * j + mine < left) {
                const uint16_t *p = reinterpret_cast<const uint16_t *>(a.residual) +
                                    (size_t)(t0 + 2 * j + mine) * a.residual_stride + c2;
                r[j] = in1 ? *reinterpret_cast<const uint32_t *>(p) : (uint32_t)*p;
            }
        }
        tmem_ld16_nowait(taddr, v);
        tmem_wait_ld();
        with_act(a.act, [&](auto act) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float z0 = lin_act<decltype(act)::value>(__uint_as_float(v[2 * j]) + b);
                const float z1 = lin_act<decltype(act)::value>(__uint_as_float(v[2 * j + 1]) + b);
                const float got = __shfl_xor_sync(0xffffffffu, odd ? z0 : z1, 1);
                const float lo = (odd ? got : z0) + __uint_as_float(r[j] << 16);
                const float hi = (odd ? z1 : got) + __uint_as_float(r[j] & 0xFFFF0000u);
                const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
                if (in0 && 2 * j + mine < left) {
                    uint16_t *p = reinterpret_cast<uint16_t *>(a.y) + (size_t)(t0 + 2 * j + mine) * a.y_stride + c2;
                    const uint32_t u = *reinterpret_cast<const uint32_t *>(&w);
                    if (in1)
                        *reinterpret_cast<uint32_t *>(p) = u;
                    else
                        *p = (uint16_t)u;
                }
            }
        });
        return;
    }
    const bool in = col < a.N;
    if (a.f32)
        lin_column<float>(a, taddr, t0, in ? left : 0, col, b);
    else
        lin_column<uint16_t>(a, taddr, t0, in ? left : 0, col, b);
}

// CG = 2: a pair of blocks computes 256 weight rows x bn tokens, each block holding 128
// rows of the accumulator, its own weight rows and half of the token rows.  CG = 1 with
// P > 1: the blocks of a cluster take a part of K each and add their sums through
// distributed shared memory, in part order.  Persistent over tiles unless P > 1.
// What bounds it: large calls the tensor cores (89% busy, 4096 x 7168 x 7168 in 221 us, 1.90
// PFLOP/s; 16384 x 3584 x 14336 with GELU in 1.05 ms, 1.60 PFLOP/s, the power limit); small ones the weights' bytes
// with a start and, in clusters, a joining of 4 us (48 x 3584 x 7168: 11.3 us, 4.6 TB/s).
template <int CG>
__global__ void __launch_bounds__(kLtThreads, CG == 1 ? 2 : 1) linear_tc_kernel(const LinearArgs a, const LinTile tl,
                                                                  const __grid_constant__ CUtensorMap mw,
                                                                  const __grid_constant__ CUtensorMap mx)
{
    extern __shared__ __align__(1024) uint8_t lsm_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(lsm_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[kLtMaxStg], empty[kLtMaxStg], acc_full[2], acc_empty[2], drain;
    __shared__ uint32_t tmem_base;
    __shared__ volatile int bail;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = CG == 1 ? tl.P : 1, nstg = tl.nstg;
    const uint32_t rank = (CG == 2 || P > 1) ? cluster_rank() : 0;
    const bool leader = CG == 1 || rank == 0;
    const int cid = CG == 2 ? blockIdx.x / 2 : blockIdx.x / P;       // this cluster, and how many there are
    const int ncl = CG == 2 ? gridDim.x / 2 : gridDim.x / P;
    const int n_items = tl.n_rb * tl.n_tt;
    const int part = P > 1 ? (int)rank : 0;
    const int ks0 = (int)((long long)tl.nks * part / P), ks1 = (int)((long long)tl.nks * (part + 1) / P);
    if (threadIdx.x == 0) {
        for (int s = 0; s < nstg; s++) { mb_init(&full[s], 1); mb_init(&empty[s], 1); }
        for (int b = 0; b < 2; b++) { mb_init(&acc_full[b], 1); mb_init(&acc_empty[b], kLtNumEpi * CG); }
        mb_init(&drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        bail = 0;
        prefetch_map(&mw);
        prefetch_map(&mx);
    }
    pdl_wait();                       // nothing above touches memory or takes what the kernel before may still need
    pdl_trigger();
    if (warp == kLtWarpMma) {
        if (CG == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&tmem_base)),
                         "r"(512));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&tmem_base)),
                         "r"(tl.cols));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2 || P > 1) cluster_sync_all();                        // the peers' barriers are set up
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    auto timeout = [&]() {
        set_status(a.status, K3MOE_DEV_TIMEOUT);
        bail = 1;
    };
    // tile i: `group` row blocks side by side, token tile by token tile, so that the blocks
    // at work share both few weight rows and few token rows in the L2
    auto tile_of = [&](int i, int *rb, int *tt) {
        const int g = i / (tl.group * tl.n_tt), r = i % (tl.group * tl.n_tt);
        const int w = min(tl.group, tl.n_rb - g * tl.group);
        *rb = g * tl.group + r % w;
        *tt = r / w;
    };

    if (warp == kLtWarpProd) {
        const int bn_own = tl.bn / CG;                               // token rows this block loads
        uint32_t st = 0, s = 0, phase = 1;                           // stages so far, its slot, the phase its slot was freed in
        const uint32_t full0 = CG == 2 ? mapa(saddr(&full[0]), 0) : 0;
        uint8_t *stage = sm;
        for (int i = cid; i < n_items && !bail; i += ncl) {
            int rb, tt;
            tile_of(i, &rb, &tt);
            const int n0 = rb * 128 * CG + (int)rank * 128 * (CG - 1);
            const int t0 = tt * tl.bn + (int)rank * bn_own * (CG - 1);
            for (int k = ks0 * kLtBK; k < ks1 * kLtBK; k += kLtBK, st++) {
                if (st >= (uint32_t)nstg && !mb_wait_warp(&empty[s], phase)) {
                    timeout();
                    break;
                }
                if (leader) mb_expect_tx_warp(&full[s], (uint32_t)(tl.stage_bytes * CG));
                if (CG == 2) {
                    const uint32_t fb = full0 + 8 * s;
                    tma2d_pair_warp(stage, &mw, k, n0, fb);
                    tma2d_pair_warp(stage + kLtABytes, &mx, k, t0, fb);
                } else {
                    tma2d_warp(stage, &mw, k, n0, &full[s]);
                    tma2d_warp(stage + kLtABytes, &mx, k, t0, &full[s]);
                }
                stage += tl.stage_bytes;
                if (++s == (uint32_t)nstg) {
                    s = 0;
                    stage = sm;
                    phase ^= 1;
                }
            }
        }
        if (leader)                    // the last copies land (or a bounded wait gives up) before the block ends, whoever gave up
            for (uint32_t f = st > (uint32_t)nstg ? st - nstg : 0; f < st; f++)
                mb_wait_warp(&full[f % nstg], (f / nstg) & 1u);
    } else if (warp == kLtWarpMma) {
        if (leader) {
            uint32_t s = 0, phase = 0, n = 0;                        // slot, the phase it is filled in, tiles so far
            const uint32_t first = desc_lo(saddr(sm));
            uint32_t A = first;
            const uint32_t id = (idesc(1, tl.bn) & ~(31u << 24)) | ((uint32_t)(128 * CG >> 4) << 24);
            const uint32_t base = __reduce_max_sync(0xffffffffu, tmem);      // the same on every lane: a uniform register
            auto commit = [&](uint64_t *b) {
                if (CG == 2)
                    umma_commit_pair_warp(b);
                else
                    umma_commit_warp(b);
            };
            for (int i = cid; i < n_items && !bail; i += ncl, n++) {
                const int buf = n & 1;
                if (n >= 2 && !mb_wait_warp(&acc_empty[buf], ((n >> 1) - 1) & 1u)) { timeout(); break; }
                tc_fence_after();
                const uint32_t d0 = base + (uint32_t)(buf * tl.acc);
                for (int ks = ks0; ks < ks1; ks++) {
                    if (!mb_wait_warp(&full[s], phase)) { timeout(); break; }
                    tc_fence_after();
                    const uint32_t B = A + (kLtABytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < kLtBK / 16; kk++) {
                        const uint32_t acc = (ks != ks0 || kk) ? 1u : 0u;
                        if (CG == 2)
                            umma_pair_warp(d0, A + kk * 2, B + kk * 2, id, acc);
                        else
                            umma_warp(d0, A + kk * 2, B + kk * 2, id, acc);
                    }
                    commit(&empty[s]);
                    A += (uint32_t)(tl.stage_bytes >> 4);
                    if (++s == (uint32_t)nstg) {
                        s = 0;
                        A = first;
                        phase ^= 1;
                    }
                }
                if (bail) break;
                commit(&acc_full[buf]);
            }
            __syncwarp();
            commit(&drain);                                          // every issued MMA done before the dealloc
            mb_wait_warp(&drain, 0);
        }
    } else {
        // ---------------- epilogue: output column 32 q + lane of the row block per thread
        const int q = warp & 3;                                      // tensor-memory lane quadrant of this warp
        const int half = (warp - kLtWarpEpi0) >> 2;                  // which of every two 16-token chunks it takes
        const bool pairs = !a.f32 && a.y_stride % 2 == 0 && reinterpret_cast<uintptr_t>(a.y) % 4 == 0 &&
                           (!a.residual || (a.residual_stride % 2 == 0 &&
                                            reinterpret_cast<uintptr_t>(a.residual) % 4 == 0));
        uint32_t n = 0;
        for (int i = cid; i < n_items && !bail; i += ncl, n++) {
            int rb, tt;
            tile_of(i, &rb, &tt);
            const int col = rb * 128 * CG + (int)rank * 128 * (CG - 1) + 32 * q + lane;
            const float b = a.bias && col < a.N ? a.bias[col] : 0.0f;
            const int t0 = tt * tl.bn, ncols = min(tl.bn, a.T - t0);
            const int buf = n & 1;
            if (!mb_wait_warp(&acc_full[buf], (n >> 1) & 1u)) { timeout(); break; }
            tc_fence_after();
            const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(buf * tl.acc);
            for (int c0 = 16 * half; c0 < ncols; c0 += 32) {
                if (P > 1) {
                    // this part's sums, [token][weight row], over the ring (its copies are consumed)
                    float v[16];
                    tmem_ld16(lane_addr + c0, v);
                    float *dst = reinterpret_cast<float *>(sm) + (size_t)c0 * 128 + 32 * q + lane;
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (c0 + j < ncols) dst[(size_t)j * 128] = v[j];
                } else {
                    lin_chunk(a, lane_addr + c0, t0 + c0, ncols - c0, col, pairs, b);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2)
                    mb_arrive_cluster(mapa(saddr(&acc_empty[buf]), 0));
                else
                    mb_arrive(&acc_empty[buf]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (CG == 2 || P > 1) cluster_sync_all();       // peers' sums are written, and no block leaves with one still to come
    tc_fence_after();
    if (CG == 1 && P > 1) {
        int rb, tt;
        tile_of(cid, &rb, &tt);
        const int t0 = tt * tl.bn, ncols = min(tl.bn, a.T - t0);
        // a token in each P is this block's to finish: a thread four columns of it, every part's
        // sums asked for before any is added (a load from another block takes a few hundred clocks)
        const int mine = (ncols - (int)rank + P - 1) / P;
        if (!bail)
            for (int i = threadIdx.x; i < mine * 32; i += kLtThreads) {
                const int c = (int)rank + (i >> 5) * P, row = (i & 31) * 4, col = rb * 128 + row;
                if (col >= a.N) continue;
                const uint32_t at = saddr(sm) + (uint32_t)(c * 128 + row) * 4u;
                float4 v[8];
#pragma unroll
                for (int p = 0; p < 8; p++)
                    if (p < P) v[p] = ld_cluster4(mapa(at, (uint32_t)p));
                float z[4] = {}, r[4] = {};
                const int w = min(4, a.N - col);
                for (int j = 0; j < w; j++) r[j] = lin_residual(a, t0 + c, col + j);
#pragma unroll
                for (int p = 0; p < 8; p++)
                    if (p < P) {
                        z[0] += v[p].x;
                        z[1] += v[p].y;
                        z[2] += v[p].z;
                        z[3] += v[p].w;
                    }
#pragma unroll
                for (int j = 0; j < 4; j++)
                    if (j < w) {
                        const float b = a.bias ? a.bias[col + j] : 0.0f;
                        with_act(a.act, [&](auto act) { lin_put(a, t0 + c, col + j, lin_act<decltype(act)::value>(z[j] + b) + r[j]); });
                    }
            }
        cluster_sync_all();                                          // nobody leaves while its sums are read
    }
    if (warp == kLtWarpMma) {
        __syncwarp();
        if (CG == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tl.cols));
    }
}

template <int NT>
cudaError_t launch_rows(const LinearArgs &a, cudaStream_t s)
{
    const size_t smem = (size_t)NT * a.K * 2;
    if (smem > 48 * 1024) {
        const cudaError_t e = once_a_device([] {
            return cudaFuncSetAttribute(linear_rows_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLrSmem);
        });
        if (e != cudaSuccess) return e;
    }
    static thread_local size_t asked = 0;                     // the occupancy of the last shared-memory size
    static thread_local int per_sm = 0;
    if (per_sm == 0 || asked != smem) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, linear_rows_kernel<NT>, kLrThreads, smem) !=
                cudaSuccess ||
            per_sm < 1)
            per_sm = 1;
        asked = smem;
    }
    const int grid = std::max(1, std::min(num_sms() * per_sm, (a.N + kLrWarps - 1) / kLrWarps));
    return launch_pdl(linear_rows_kernel<NT>, dim3(grid), dim3(kLrThreads), smem, s, a);
}

// The tile of a call: the token tile, the K parts and the blocks an SM whose estimated time is
// least, or a pair of blocks (256 x 256) where that is estimated faster still.  The
// estimate, in SM clocks: a block's K stage takes its products' time on the tensor cores (2 a token
// of 128 rows) or its bytes' at kLtRate from the L2, shared by the blocks of an SM; a tile's
// start and epilogue about 2500 + 16 bn; a cluster's launch and joining 8000.  Single blocks in
// full waves load a third faster than that, so pairs have to be 1.3 times ahead.  Single
// against pairs, us: T 512, K = N = 7168 52, 41; T 600 52, 71; T 1024 81, 72; T 4096 256, 215; T
// 1024, K 3584, N 3584 24.8, 25.6, N 4096 27.0, 25.5, N 5120 33, 40; T 300, K 1024, N 4096 8.6, 13.8.
constexpr double kLtRate = 48.0;      // bytes a clock an SM

template <int CG> cudaError_t allow_tc()
{
    return once_a_device([] {
        return cudaFuncSetAttribute(linear_tc_kernel<CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + kLtRing);
    });
}

// Blocks at work at once in clusters of P: a cluster stays within a group of SMs, so that
// fewer fit than the SMs would hold (P = 8: 15 clusters where 152 SMs have room for 19; 8 x 2048 x
// 2048 in 16 of them took 10.9 us, in two goes, and in 16 of P = 6 6.2).
int lin_slots(int P)
{
    static std::atomic<int> known[9];
    int n = known[P].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms() / P * P));
        cfg.blockDim = dim3(kLtThreads);
        cfg.dynamicSmemBytes = 1024 + kLtRing;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)P;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int fit = 0;
        if (P > 1 && (allow_tc<1>() != cudaSuccess || cudaOccupancyMaxActiveClusters(&fit, linear_tc_kernel<1>, &cfg) != cudaSuccess)) fit = 0;
        n = (fit > 0 ? fit : num_sms() / P) * P;
        known[P].store(n, std::memory_order_relaxed);
    }
    return n;
}

int lin_plan(const LinearArgs &a, LinTile *tl)
{
    const int sms = num_sms();
    tl->nks = (a.K + kLtBK - 1) / kLtBK;
    tl->P = 1;
    tl->per_sm = 1;
    tl->acc = 256;
    tl->cols = 512;
    tl->group = 8;
    tl->n_rb = (a.N + 127) / 128;
    double best = 1e30;
    for (int n_tt = (a.T + 255) / 256; n_tt <= 64; n_tt++) {
        const int bn = ((a.T + n_tt - 1) / n_tt + 15) & ~15;
        if (n_tt > 1 && bn < 64) break;
        for (int P = 1; P <= 8; P++) {
            if (P > 1 && tl->nks / P < 4) break;
            for (int per_sm = 1; per_sm <= (bn <= 128 ? 2 : 1); per_sm++) {
                const long long items = (long long)tl->n_rb * n_tt * P, slots = lin_slots(P);
                const long long waves = (items + slots * per_sm - 1) / (slots * per_sm);
                const double load = (128.0 + bn) * 128.0 / kLtRate * (items > slots ? per_sm : 1);
                const double t = waves * ((double)((tl->nks + P - 1) / P) * std::max(2.0 * bn, load) + 2500.0 + 16.0 * bn / P +
                                          (P > 1 ? 8000.0 + 16.0 * bn : 0.0));
                if (t < best) {
                    best = t;
                    tl->bn = bn;
                    tl->n_tt = n_tt;
                    tl->P = P;
                    tl->per_sm = per_sm;
                }
            }
        }
    }
    const long long pairs = (long long)((a.N + 255) / 256) * ((a.T + 255) / 256), waves = (pairs + sms / 2 - 1) / (sms / 2);
    const double paired = waves * tl->nks * std::max(512.0, 2.0 * kLtABytes / kLtRate) + 2500.0 + 16.0 * 256;
    if (best > 1.3 * paired) {
        tl->P = tl->per_sm = 1;
        tl->bn = 256;
        tl->acc = 256;
        tl->cols = 512;
        tl->n_rb = (a.N + 255) / 256;
        tl->n_tt = (a.T + 255) / 256;
        tl->stage_bytes = 2 * kLtABytes;
        tl->nstg = kLtRing / tl->stage_bytes;
        return 2;
    }
    tl->acc = tl->bn <= 32 ? 32 : tl->bn <= 64 ? 64 : tl->bn <= 128 ? 128 : 256;
    tl->cols = tl->P > 1 ? tl->acc : 2 * tl->acc;
    tl->stage_bytes = kLtABytes + tl->bn * kLtBK * 2;
    tl->nstg = std::min(kLtMaxStg, (tl->per_sm == 2 ? kLtRing2 : kLtRing) / tl->stage_bytes);
    return 1;
}

template <int CG>
cudaError_t launch_tc(const LinearArgs &a, const LinTile &tl, cudaStream_t s)
{
    CUtensorMap mw{}, mx{};
    if (!map16s(&mw, a.w, (uint64_t)a.N, (uint64_t)a.K, (uint64_t)a.K, 128) ||
        !map16s(&mx, a.x, (uint64_t)a.T, (uint64_t)a.K, (uint64_t)a.x_stride, (uint32_t)(tl.bn / CG)))
        return cudaErrorInvalidValue;
    const size_t smem = 1024 + (tl.per_sm == 2 ? kLtRing2 : kLtRing);
    if (allow_tc<CG>() != cudaSuccess) return cudaErrorInvalidConfiguration;
    const int csize = CG == 2 ? 2 : tl.P;
    const int items = tl.n_rb * tl.n_tt;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(CG == 1 && tl.P > 1 ? items * tl.P : std::min(items, num_sms() * tl.per_sm / csize) * csize));
    cfg.blockDim = dim3(kLtThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)csize;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_tc_kernel<CG>, a, tl, mw, mx);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, cudaStream_t s)
{
    timing_begin("linear", s);
    cudaError_t err;
    if (a.T == 1 && (size_t)a.K * 2 <= kLrSmem) {
        err = launch_rows<1>(a, s);
    } else if (a.T <= 2 && (size_t)a.K * 4 <= kLrSmem) {
        err = launch_rows<2>(a, s);
    } else if (a.T <= 4 && (size_t)a.K * 8 <= kLrSmem && (long long)a.N * a.K <= kLrFour) {
        err = launch_rows<4>(a, s);
    } else {
        LinTile tl{};
        err = lin_plan(a, &tl) == 2 ? launch_tc<2>(a, tl, s) : launch_tc<1>(a, tl, s);
    }
    count_launch();
    timing_end("linear", s);
    return err;
}

}  // namespace k3moe
