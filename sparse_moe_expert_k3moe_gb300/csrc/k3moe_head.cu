// k3moe_head.cu -- y[t][h] = W[h] x[t][h]: each head's own projection (a latent attention's
// queries into the latent, and what they attended back to values).
//
// A block has 128 of a head's output columns and up to 256 tokens: the weights are the A operand and the tokens B, 64
// columns of K a stage of the ring, which leaves room for a second block on the SM whose loads run under this one's
// epilogue; where there are no more blocks than SMs the ring has the room of both.  A thread of the epilogue owns an
// output column and its warp's lanes 32 neighbouring ones.
// What bounds it: one token (56 heads, 128 to 512) start and the first loads, 3.1 us in a graph; a batch the bytes that an SM takes
// from the L2, and an epilogue, once each.  With inputs from the DRAM, 56 heads, 512 to 128: 100 tokens 6.2 us, 333 tokens 9.1 (5.9 where
// the L2 has them), 28 heads 6.4; with up to 128 tokens a block, however many blocks that makes, 7.7, 9.4 and 7.8.
#include <cuda.h>
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"
#include "k3moe_tc_warp.cuh"

namespace k3moe {
namespace {

constexpr int kHdMaxBN = 256, kHdABytes = 128 * 128;          // tokens a block; 64 columns of its weights
constexpr int kHdThreads = 192, kHdMaxStages = 8;             // four epilogue warps, loads, MMAs
constexpr int kHdRing = 100 * 1024, kHdRingAlone = 200 * 1024;            // two blocks an SM; no more blocks than SMs

struct HeadTile {
    int bn, stages, cols;                                     // tokens; ring; columns of tensor memory
};

__global__ void __launch_bounds__(kHdThreads, 2) head_linear_kernel(const HeadLinearArgs a, const HeadTile tl,
                                                                const __grid_constant__ CUtensorMap mw,
                                                                const __grid_constant__ CUtensorMap mx)
{
    extern __shared__ __align__(1024) uint8_t hsm_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(hsm_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[kHdMaxStages], empty[kHdMaxStages], done;
    __shared__ uint32_t tmem_base;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = (a.K + 63) / 64, stage_bytes = kHdABytes + tl.bn * 128;
    const int n0 = blockIdx.x * 128, h = blockIdx.y, t0 = blockIdx.z * tl.bn;
    if (threadIdx.x == 0) {
        for (int i = 0; i < tl.stages; i++) {
            mb_init(&full[i], 1);
            mb_init(&empty[i], 1);
        }
        mb_init(&done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&mw);
        prefetch_map(&mx);
    }
    pdl_wait();
    pdl_trigger();
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&tmem_base)), "r"(tl.cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    auto wait = [&](uint64_t *b, uint32_t phase) {
        const bool ok = mb_wait_warp(b, phase & 1u);
        if (!ok) set_status(a.status, K3MOE_DEV_TIMEOUT);
        return ok;
    };
    if (warp == 4) {
        int c = 0;
        for (int s = 0, phase = 1; c < chunks; c++) {
            if (c >= tl.stages && !wait(&empty[s], phase)) break;
            mb_expect_tx_warp(&full[s], (uint32_t)stage_bytes);
            tma3d_warp(sm + s * stage_bytes, &mw, 64 * c, n0, h, &full[s]);
            tma3d_warp(sm + s * stage_bytes + kHdABytes, &mx, 64 * c, h, t0, &full[s]);
            if (++s == tl.stages) {
                s = 0;
                phase ^= 1;
            }
        }
        for (int f = max(0, c - tl.stages); f < c; f++) mb_wait_warp(&full[f % tl.stages], (f / tl.stages) & 1u);   // the copies land before the block ends
    } else if (warp == 5) {
        const uint32_t A = desc_lo(saddr(sm)), base = __reduce_max_sync(0xffffffffu, tmem), id = idesc(1, tl.bn);
        for (int c = 0, s = 0, phase = 0; c < chunks; c++) {
            if (!wait(&full[s], phase)) break;
            tc_fence_after();
            const uint32_t at = A + (uint32_t)(s * stage_bytes >> 4);
#pragma unroll
            for (int k = 0; k < 4; k++) umma_warp(base, at + 2 * k, at + (kHdABytes >> 4) + 2 * k, id, c > 0 || k > 0);
            umma_commit_warp(&empty[s]);
            if (++s == tl.stages) {
                s = 0;
                phase ^= 1;
            }
        }
        umma_commit_warp(&done);
        mb_wait_warp(&done, 0);
    } else if (wait(&done, 0)) {
        tc_fence_after();
        const int n = n0 + 32 * warp + lane, left = min(tl.bn, a.T - t0), odd = lane & 1;
        const uint32_t la = tmem + ((uint32_t)(32 * warp) << 16);
        // where rows start on a word neighbouring lanes trade a token each, two columns of one token a store
        const bool pairs = a.N % 2 == 0 && a.y_stride % 2 == 0 && a.y_head % 2 == 0 && reinterpret_cast<uintptr_t>(a.y) % 4 == 0;
        uint16_t *y = a.y + (size_t)h * a.y_head + (size_t)t0 * a.y_stride;
        for (int c0 = 0; c0 < left; c0 += 32) {               // (32 columns of tensor memory at a time are always there)
            uint32_t v[2][16];
            tmem_ld16_nowait(la + c0, v[0]);
            tmem_ld16_nowait(la + c0 + 16, v[1]);
            tmem_wait_ld();
            if (pairs) {
                uint16_t *p = y + (size_t)(c0 + odd) * a.y_stride + (n & ~1);
#pragma unroll
                for (int j = 0; j < 16; j++, p += 2 * a.y_stride) {
                    const float z0 = __uint_as_float(v[j >> 3][2 * (j & 7)]), z1 = __uint_as_float(v[j >> 3][2 * (j & 7) + 1]);
                    const float got = __shfl_xor_sync(0xffffffffu, odd ? z0 : z1, 1);
                    const __nv_bfloat162 w = odd ? __floats2bfloat162_rn(got, z1) : __floats2bfloat162_rn(z0, got);
                    if (n < a.N && c0 + 2 * j + odd < left) *reinterpret_cast<__nv_bfloat162 *>(p) = w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; j++)
                    if (n < a.N && c0 + j < left)
                        *reinterpret_cast<__nv_bfloat16 *>(y + (size_t)(c0 + j) * a.y_stride + n) = __float2bfloat16_rn(__uint_as_float(v[j >> 4][j & 15]));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tl.cols));
}

}  // namespace

cudaError_t launch_head_linear(const HeadLinearArgs &a, cudaStream_t s)
{
    HeadTile tl{};
    // as many tokens a block as leaves the SM with the most blocks the fewest rows of weights and tokens to load; 128 at most where K
    // is short and an epilogue longer than the loads (333 tokens, 56 heads, 128 to 512: 10.0 us, with 176 a block 10.9)
    const int most = a.K >= 256 ? kHdMaxBN : 128;
    const long long columns = (long long)((a.N + 127) / 128) * a.H;
    long long least = 0;
    for (int tiles = (a.T + most - 1) / most, i = 0; i < 8; tiles++, i++) {
        const int bn = ((a.T + tiles - 1) / tiles + 15) & ~15;
        const long long blocks = columns * ((a.T + bn - 1) / bn), rows = (blocks + num_sms() - 1) / num_sms() * (128 + bn);
        if (i == 0 || rows < least) {
            least = rows;
            tl.bn = bn;
        }
    }
    tl.cols = tl.bn <= 32 ? 32 : tl.bn <= 64 ? 64 : tl.bn <= 128 ? 128 : 256;
    const int stage_bytes = kHdABytes + tl.bn * 128, ring = columns * ((a.T + tl.bn - 1) / tl.bn) <= num_sms() ? kHdRingAlone : kHdRing;
    tl.stages = std::min(std::min(kHdMaxStages, ring / stage_bytes), (a.K + 63) / 64);
    CUtensorMap mw{}, mx{};
    if (!map16x3(&mw, a.w, (uint64_t)a.H, (uint64_t)a.N * a.K, (uint64_t)a.N, (uint64_t)a.K, (uint64_t)a.K, 128, 1) ||
        !map16x3(&mx, a.x, (uint64_t)a.T, (uint64_t)a.x_stride, (uint64_t)a.H, (uint64_t)a.x_head, (uint64_t)a.K, 1, (uint32_t)tl.bn))
        return cudaErrorInvalidValue;
    const cudaError_t allowed =
        once_a_device([] { return cudaFuncSetAttribute(head_linear_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + kHdRingAlone); });
    if (allowed != cudaSuccess) return allowed;
    timing_begin("head_linear", s);
    const cudaError_t err = launch_pdl(head_linear_kernel, dim3((unsigned)((a.N + 127) / 128), (unsigned)a.H, (unsigned)((a.T + tl.bn - 1) / tl.bn)),
                                       dim3(kHdThreads), (size_t)(1024 + tl.stages * stage_bytes), s, a, tl, mw, mx);
    count_launch();
    timing_end("head_linear", s);
    return err;
}

}  // namespace k3moe
