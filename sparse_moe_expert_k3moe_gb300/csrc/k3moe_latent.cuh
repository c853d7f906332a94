// k3moe_latent.cuh -- what both forms of the latent attention share: which tokens are a
// sequence's, the search for a block's piece of work over the sequences, and the repair of values that
// no arithmetic survives where a query does not see them.
#pragma once
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"
#include "k3moe_tc_warp.cuh"

namespace k3moe {
namespace {

constexpr float kLatLog2e = 1.4426950408889634f, kLatLn2 = 0.6931471805599453f;

// Queries [first, first + n) of sequence i; false when its offsets are not ascending within 0 .. T.
__device__ __forceinline__ bool latent_queries(const int32_t *start, int n_seq, int T, int i, int *first, int *n)
{
    if (!start) {
        const int each = n_seq == 1 ? T : 1;
        *first = i * each;
        *n = each;
        return true;
    }
    const int s0 = start[i], s1 = start[i + 1];
    *first = s0;
    *n = s1 - s0;
    return s0 >= 0 && s1 >= s0 && s1 <= T;
}

// A block's search for unit `want` over the sequences, count(i) units each, all threads at once: the sequence
// it is of (-1: there are not as many) and how many units of it come before.
struct UnitSearch {
    int sums[32], seq, before;
};
template <int THREADS, typename Count>
__device__ __forceinline__ int find_unit(UnitSearch &sh, int n_seq, int want, int *before, Count count)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) sh.seq = -1;
    int base = 0;
    for (int i0 = 0; i0 < n_seq; i0 += THREADS) {
        const int i = i0 + threadIdx.x;
        const int mine = i < n_seq ? count(i) : 0;
        int upto = mine;                                      // of the warp's lanes up to this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        __syncthreads();
        if (lane == 31) sh.sums[warp] = upto;
        __syncthreads();
        int ahead = base, all = base;
        for (int w = 0; w < THREADS / 32; w++) {
            if (w < warp) ahead += sh.sums[w];
            all += sh.sums[w];
        }
        const int from = ahead + upto - mine;
        if (mine > 0 && want >= from && want < from + mine) {
            sh.seq = i;
            sh.before = want - from;
        }
        base = all;
        if (want < base) break;
    }
    __syncthreads();
    *before = sh.before;
    return sh.seq;
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
