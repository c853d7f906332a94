// k3moe_head.cu -- y[t][h] = W[h] x[t][h]: each head's own projection (a latent attention's
// queries into the latent, and what they attended back to values).
//
// A block has 128 of a head's output columns and up to 64 tokens: the weights [128][K] are
// the A operand and the tokens [64][K] B, both loaded whole by TMA (K <= 512 fits the shared
// memory), a barrier for every 64 columns of K, so that the products follow the loads.  A thread of the
// epilogue owns an output column and its warp's lanes 32 neighbouring ones.
#include <cuda.h>
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"
#include "k3moe_tc_warp.cuh"

namespace k3moe {
namespace {

constexpr int kHdBN = 64, kHdABytes = 128 * 128;              // tokens a block; a 64-column chunk of weights
constexpr int kHdThreads = 192, kHdMaxChunks = kMaxHeadK / 64;    // four epilogue warps, loads, MMAs

__global__ void __launch_bounds__(kHdThreads) head_linear_kernel(const HeadLinearArgs a, const int bn,
                                                                const __grid_constant__ CUtensorMap mw,
                                                                const __grid_constant__ CUtensorMap mx)
{
    extern __shared__ __align__(1024) uint8_t hsm_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(hsm_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[kHdMaxChunks], done;
    __shared__ uint32_t tmem_base;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = (a.K + 63) / 64, chunk_bytes = kHdABytes + bn * 128;
    const int n0 = blockIdx.x * 128, h = blockIdx.y, t0 = blockIdx.z * bn;
    const uint32_t cols = bn <= 32 ? 32 : 64;
    if (threadIdx.x == 0) {
        for (int c = 0; c < chunks; c++) mb_init(&full[c], 1);
        mb_init(&done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&mw);
        prefetch_map(&mx);
    }
    pdl_wait();
    pdl_trigger();
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&tmem_base)), "r"(cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    if (warp == 4) {
        for (int c = 0; c < chunks; c++) {
            mb_expect_tx_warp(&full[c], (uint32_t)chunk_bytes);
            tma3d_warp(sm + c * chunk_bytes, &mw, 64 * c, n0, h, &full[c]);
            tma3d_warp(sm + c * chunk_bytes + kHdABytes, &mx, 64 * c, h, t0, &full[c]);
        }
        bool ok = true;                                       // the copies land before the block ends
        for (int c = 0; c < chunks; c++) ok = mb_wait_warp(&full[c], 0) && ok;
        if (!ok && lane == 0) set_status(a.status, K3MOE_DEV_TIMEOUT);
    } else if (warp == 5) {
        const uint32_t A = desc_lo(saddr(sm)), base = __reduce_max_sync(0xffffffffu, tmem), id = idesc(1, bn);
        for (int c = 0; c < chunks; c++) {
            if (!mb_wait_warp(&full[c], 0)) break;
            tc_fence_after();
            const uint32_t at = A + (uint32_t)(c * chunk_bytes >> 4);
#pragma unroll
            for (int k = 0; k < 4; k++) umma_warp(base, at + 2 * k, at + (kHdABytes >> 4) + 2 * k, id, c > 0 || k > 0);
        }
        umma_commit_warp(&done);
        mb_wait_warp(&done, 0);
    } else if (mb_wait_warp(&done, 0)) {
        tc_fence_after();
        const int n = n0 + 32 * warp + lane, left = min(bn, a.T - t0);
        const uint32_t la = tmem + ((uint32_t)(32 * warp) << 16);
        uint16_t *y = a.y + (size_t)h * a.y_head + n;
        for (int c0 = 0; c0 < left; c0 += 16) {
            uint32_t v[16];
            tmem_ld16_nowait(la + c0, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j++)
                if (n < a.N && c0 + j < left)
                    *reinterpret_cast<__nv_bfloat16 *>(y + (size_t)(t0 + c0 + j) * a.y_stride) = __float2bfloat16_rn(__uint_as_float(v[j]));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}

}  // namespace

cudaError_t launch_head_linear(const HeadLinearArgs &a, cudaStream_t s)
{
    const int bn = std::min(kHdBN, (a.T + 15) & ~15), chunks = (a.K + 63) / 64;
    CUtensorMap mw{}, mx{};
    if (!map16x3(&mw, a.w, (uint64_t)a.H, (uint64_t)a.N * a.K, (uint64_t)a.N, (uint64_t)a.K, (uint64_t)a.K, 128, 1) ||
        !map16x3(&mx, a.x, (uint64_t)a.T, (uint64_t)a.x_stride, (uint64_t)a.H, (uint64_t)a.x_head, (uint64_t)a.K, 1, (uint32_t)bn))
        return cudaErrorInvalidValue;
    const cudaError_t allowed = once_a_device([] {
        return cudaFuncSetAttribute(head_linear_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    1024 + kHdMaxChunks * (kHdABytes + kHdBN * 128));
    });
    if (allowed != cudaSuccess) return allowed;
    timing_begin("head_linear", s);
    const cudaError_t err = launch_pdl(head_linear_kernel, dim3((unsigned)((a.N + 127) / 128), (unsigned)a.H, (unsigned)((a.T + bn - 1) / bn)),
                                       dim3(kHdThreads), (size_t)(1024 + chunks * (kHdABytes + bn * 128)), s, a, bn, mw, mx);
    count_launch();
    timing_end("head_linear", s);
    return err;
}

}  // namespace k3moe
