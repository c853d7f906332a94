// k3moe_latent.cuh -- what the forms of the latent attention share: the workspace's layout, the search
// for a block's piece of work over the sequences, and the repair of values that no arithmetic
// survives where a query does not see them; and the absorbed form's waits.
#pragma once
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"
#include "k3moe_tc_warp.cuh"

namespace k3moe {
namespace {

constexpr float kLatLog2e = 1.4426950408889634f, kLatLn2 = 0.6931471805599453f;

// The workspace behind the counters: what joins parts (of each of up to kMaxShares blocks), then two parts' sums a block,
// 64 queries x 512 columns with their maxima and sums in the absorbed form.
constexpr int kMaxShares = 512;
constexpr size_t kLatPart = (size_t)64 * kLatC + 2 * 64, kLatJoinBytes = (size_t)kMaxShares * 64;
inline float *latent_parts(uint8_t *ws) { return reinterpret_cast<float *>(ws + kCtrOffset + kCtrBytes + kLatJoinBytes); }

// A warp's wait on a barrier's phase.  What follows when it is not complete at the first try, which itself waits a while, is a
// call: the roles of a block share the instruction cache, and every wait written out in full was a fifth of their code.
__device__ __noinline__ bool role_wait_long(uint64_t *b, uint32_t parity, int32_t *status, volatile int *bail)
{
    const bool ok = mb_wait_warp(b, parity);
    if (!ok) {
        set_status(status, K3MOE_DEV_TIMEOUT);
        *bail = 1;
    }
    return ok;
}
__device__ __forceinline__ bool role_wait(uint64_t *b, int phase, int32_t *status, volatile int *bail)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(saddr(b)), "r"((uint32_t)phase & 1u)
        : "memory");
    return __all_sync(0xffffffffu, done != 0) || role_wait_long(b, (uint32_t)phase & 1u, status, bail);
}

// A lane's look at a phase, without a wait.
__device__ __forceinline__ bool role_done(uint64_t &b, int phase)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(saddr(&b)), "r"((uint32_t)phase & 1u)
        : "memory");
    return done != 0;
}
// a / b of positive numbers, in 32 bits where they fit: the long division is a hundred instructions.
__device__ __forceinline__ long long quotient(long long a, int b) { return a >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b); }
__device__ __forceinline__ int quotient(int a, int b) { return (int)((uint32_t)a / (uint32_t)b); }

// A block's search over the sequences, count(i) units each: which one unit want(total) is of (-1: there are not as
// many), how many units of it come before, and the units in all.  I: int where the units are known to fit.
template <typename I> struct UnitSearch {
    I sums[32], before;
    int seq;
};
template <typename I> __device__ __forceinline__ I warp_scan(I v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const I x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}
template <int THREADS, typename I, typename Count, typename Want>
__device__ __forceinline__ int find_unit(UnitSearch<I> &sh, int n_seq, I *before, I *total, Count count, Want want)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (n_seq <= 32) {                                        // every warp for itself
        const I mine = lane < n_seq ? count(lane) : 0, upto = warp_scan(mine, lane);
        *total = __shfl_sync(0xffffffffu, upto, 31);
        const I unit = want(*total);
        const int seq = __popc(__ballot_sync(0xffffffffu, upto <= unit));        // as many end before it
        *before = unit - __shfl_sync(0xffffffffu, upto - mine, seq & 31);
        return seq < n_seq ? seq : -1;
    }
    if (threadIdx.x == 0) sh.seq = -1;
    // units of this thread's sequence of the THREADS from i0 on, those before it (from `base` on), and all of them
    auto scan = [&](int i0, I *mine, I *all) {
        *mine = i0 + (int)threadIdx.x < n_seq ? count(i0 + threadIdx.x) : 0;
        const I upto = warp_scan(*mine, lane);
        __syncthreads();
        if (lane == 31) sh.sums[warp] = upto;
        __syncthreads();
        I ahead = 0;
        *all = 0;
        for (int w = 0; w < THREADS / 32; w++) {
            if (w < warp) ahead += sh.sums[w];
            *all += sh.sums[w];
        }
        return (I)(ahead + upto - *mine);
    };
    auto keep = [&](int i0, I from, I mine, I unit) {
        if (unit >= from && unit < from + mine) {
            sh.seq = i0 + threadIdx.x;
            sh.before = unit - from;
        }
    };
    I mine, all, from = scan(0, &mine, &all);
    *total = all;
    if (n_seq <= THREADS) {
        keep(0, from, mine, want(all));
    } else {
        for (int i0 = THREADS; i0 < n_seq; i0 += THREADS) {
            scan(i0, &mine, &all);
            *total += all;
        }
        I base = 0;
        const I unit = want(*total);
        for (int i0 = 0; i0 < n_seq && base <= unit; i0 += THREADS, base += all) {
            from = base + scan(i0, &mine, &all);
            keep(i0, from, mine, unit);
        }
    }
    __syncthreads();
    *before = sh.before;
    return sh.seq;
}

// Not zero when one of eight bf16 is infinite or NaN.
__device__ __forceinline__ uint32_t spoiled_in(const uint4 &w)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) any |= (u[i] & 0x7F807F80u) + 0x00800080u;       // an exponent of all ones carries
    return any & 0x80008000u;
}
// Clears the elements of eight bf16 that are infinite or NaN; true when there was one.
__device__ __forceinline__ bool clear_spoiled(uint4 &w)
{
    uint32_t u[4] = {w.x, w.y, w.z, w.w}, any = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t m = ((u[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;   // an exponent of all ones carries
        any |= m;
        u[i] &= ~((m >> 15) * 0xFFFFu);
    }
    w = make_uint4(u[0], u[1], u[2], u[3]);
    return any != 0;
}

}  // namespace
}  // namespace k3moe
