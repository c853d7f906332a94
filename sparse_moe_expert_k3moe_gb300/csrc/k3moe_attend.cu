// k3moe_attend.cu -- latent attention, the simple form: a block per query token and head, a lane a key.
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"

namespace k3moe {
namespace {

constexpr int kSimpleThreads = 128, kSimpleWarps = kSimpleThreads / 32;

// The sequence of token t: its first token and their number; -1 when t is of none.
__device__ __forceinline__ int sequence_of(const int32_t *start, int n_seq, int T, int t, int *first, int *n, int32_t *status)
{
    if (!start) {
        const int each = n_seq == 1 ? T : 1;
        *first = t / each * each;
        *n = each;
        return t / each;
    }
    for (int i = 0; i < n_seq; i++) {
        const int s0 = start[i], s1 = start[i + 1];
        if (s0 < 0 || s1 < s0 || s1 > T) {
            set_status(status, K3MOE_DEV_BAD_OFFSETS);
            continue;
        }
        if (t >= s0 && t < s1) {
            *first = s0;
            *n = s1 - s0;
            return i;
        }
    }
    return -1;
}

template <int DV> struct Simple {
    float q[kLatRow];
    float m[kSimpleWarps], l[kSimpleWarps], o[kSimpleWarps][DV];
};

template <int DV, typename Keys>
__device__ __forceinline__ void simple_attention(Simple<DV> &sh, int n_keys, float scale, uint16_t *out, float *lse, Keys keys)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float m = -INFINITY, l = 0.0f, o[DV / 32];
#pragma unroll
    for (int i = 0; i < DV / 32; i++) o[i] = 0.0f;
    for (int k0 = 32 * warp; k0 < n_keys; k0 += 32 * kSimpleWarps) {
        float s = -INFINITY;
        if (k0 + lane < n_keys) s = scale * keys.score(k0 + lane, sh.q);
        float mx = s;
        for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float m1 = fmaxf(m, mx), f = m1 == -INFINITY ? 1.0f : expf(m - m1);
        const float p = k0 + lane < n_keys ? expf(s - m1) : 0.0f;
        float sum = p;
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l = l * f + sum;
        m = m1;
#pragma unroll
        for (int i = 0; i < DV / 32; i++) o[i] *= f;
        for (int j = 0; j < min(32, n_keys - k0); j++) {
            const float pj = __shfl_sync(0xffffffffu, p, j);
#pragma unroll
            for (int i = 0; i < DV / 32; i++) o[i] = fmaf(pj, keys.value(k0 + j, 32 * i + lane), o[i]);
        }
    }
    sh.m[warp] = m;
    sh.l[warp] = l;
#pragma unroll
    for (int i = 0; i < DV / 32; i++) sh.o[warp][32 * i + lane] = o[i];
    __syncthreads();
    float M = -INFINITY, L = 0.0f;
    for (int w = 0; w < kSimpleWarps; w++) M = fmaxf(M, sh.m[w]);
    for (int w = 0; w < kSimpleWarps; w++) L += sh.m[w] == -INFINITY ? 0.0f : sh.l[w] * expf(sh.m[w] - M);
    for (int d = threadIdx.x; d < DV; d += kSimpleThreads) {
        float v = 0.0f;
        for (int w = 0; w < kSimpleWarps; w++) v += sh.m[w] == -INFINITY ? 0.0f : sh.o[w][d] * expf(sh.m[w] - M);
        reinterpret_cast<__nv_bfloat16 *>(out)[d] = __float2bfloat16_rn(n_keys > 0 ? v / L : 0.0f);
    }
    if (lse && threadIdx.x == 0) *lse = n_keys > 0 ? M + logf(L) : -INFINITY;
}

struct CacheKeys {
    const uint16_t *cache;
    const int32_t *pages;
    int page, n_pages;
    int32_t *status;
    __device__ const uint16_t *row(int j) const
    {
        const int p = pages[j / page];
        if (p < 0 || p >= n_pages) {
            set_status(status, K3MOE_DEV_BAD_INDEX);
            return nullptr;
        }
        return cache + ((size_t)p * page + j % page) * kLatRow;
    }
    __device__ float score(int j, const float *q) const
    {
        const uint16_t *r = row(j);
        float s = 0.0f;
        if (r)
            for (int c = 0; c < kLatRow; c++) s = fmaf(q[c], bf16_bits_to_f32(r[c]), s);
        return s;
    }
    __device__ float value(int j, int d) const
    {
        const uint16_t *r = row(j);
        return r ? bf16_bits_to_f32(r[d]) : 0.0f;
    }
};

__global__ void __launch_bounds__(kSimpleThreads) attend_simple_kernel(const AttendArgs a)
{
    __shared__ Simple<kLatC> sh;
    const int t = blockIdx.x / a.H, h = blockIdx.x % a.H;
    int32_t *status = reinterpret_cast<int32_t *>(a.ws);
    int first, n;
    const int i = sequence_of(a.seq_start, a.n_seq, a.T, t, &first, &n, status);
    if (i < 0) return;
    const int len = a.kv_len[i];
    if (len < 0 || len > a.max_pages * a.page) {
        set_status(status, K3MOE_DEV_BAD_OFFSETS);
        return;
    }
    for (int c = threadIdx.x; c < kLatRow; c += kSimpleThreads)
        sh.q[c] = bf16_bits_to_f32(a.q[(size_t)t * a.q_stride + (size_t)h * a.q_head + c]);
    __syncthreads();
    const size_t o = (size_t)t * a.H + h;
    simple_attention<kLatC>(sh, a.causal ? max(0, len - (n - 1 - (t - first))) : len, a.scale, a.out + o * kLatC, a.lse ? a.lse + o : nullptr,
                            CacheKeys{a.cache, a.pages + (size_t)i * a.max_pages, a.page, a.n_pages, status});
}

}  // namespace

size_t latent_workspace(const k3moe_latent_config &lc, int n_seq, int T)
{
    (void)lc;
    (void)n_seq;
    (void)T;
    return kCtrOffset + kCtrBytes;
}

cudaError_t launch_attend(const AttendArgs &a, cudaStream_t s)
{
    timing_begin("latent_attend", s);
    attend_simple_kernel<<<(unsigned)(a.T * a.H), kSimpleThreads, 0, s>>>(a);
    count_launch();
    timing_end("latent_attend", s);
    return cudaGetLastError();
}

}  // namespace k3moe
