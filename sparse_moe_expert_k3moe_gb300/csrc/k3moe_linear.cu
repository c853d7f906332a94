// k3moe_linear.cu -- y = act(x W^T + bias) + residual, x [T][K] and W [N][K] bf16 (the
// projections of a decoder layer around its token mixer).
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"

namespace k3moe {
namespace {

// The activations in float, from their definitions; expf, erff and log1pf are CUDA's.
__device__ __forceinline__ float lin_act(float z, int act)
{
    switch (act) {
    case K3MOE_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case K3MOE_ACT_SILU: return z / (1.0f + expf(-z));
    case K3MOE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case K3MOE_ACT_SIGMOID: return 1.0f / (1.0f + expf(-z));
    case K3MOE_ACT_LOGSIGMOID: return fminf(z, 0.0f) - log1pf(expf(-fabsf(z)));
    }
    return z;
}

// One output: its sum through the epilogue, rounded once.
__device__ __forceinline__ void lin_store(const LinearArgs &a, int t, int n, float z)
{
    if (a.bias) z += __ldg(a.bias + n);
    z = lin_act(z, a.act);
    const size_t o = (size_t)t * a.y_stride + n, r = (size_t)t * a.residual_stride + n;
    if (a.f32) {
        if (a.residual) z += reinterpret_cast<const float *>(a.residual)[r];
        reinterpret_cast<float *>(a.y)[o] = z;
    } else {
        if (a.residual) z += bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(a.residual)[r]);
        reinterpret_cast<__nv_bfloat16 *>(a.y)[o] = __float2bfloat16_rn(z);
    }
}

// 64 x 64 outputs a block, 4 x 4 a thread, K in steps of 32 through shared memory.
__global__ void __launch_bounds__(256) linear_simple_kernel(const LinearArgs a, int n_nt)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float xs[32][65], wsm[32][65];
    const int t0 = (blockIdx.x / n_nt) * 64, n0 = (blockIdx.x % n_nt) * 64;
    const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += 32) {
        for (int i = threadIdx.x; i < 64 * 32; i += 256) {
            const int r = i / 32, c = i % 32;
            const bool kk = k0 + c < a.K;
            xs[c][r] = kk && t0 + r < a.T ? bf16_bits_to_f32(a.x[(size_t)(t0 + r) * a.x_stride + k0 + c]) : 0.0f;
            wsm[c][r] = kk && n0 + r < a.N ? bf16_bits_to_f32(a.w[(size_t)(n0 + r) * a.K + k0 + c]) : 0.0f;
        }
        __syncthreads();
        for (int c = 0; c < 32; c++)
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) acc[i][j] = fmaf(xs[c][tr * 4 + i], wsm[c][tc + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < 4; j++) {
            const int t = t0 + tr * 4 + i, n = n0 + tc + 16 * j;
            if (t < a.T && n < a.N) lin_store(a, t, n, acc[i][j]);
        }
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, cudaStream_t s)
{
    const int n_nt = (a.N + 63) / 64, n_tt = (a.T + 63) / 64;
    timing_begin("linear", s);
    const cudaError_t err = launch_pdl(linear_simple_kernel, dim3((unsigned)n_nt * n_tt), dim3(256), 0, s, a, n_nt);
    count_launch();
    timing_end("linear", s);
    return err;
}

}  // namespace k3moe
