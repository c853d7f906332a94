// k3moe_norm.cu -- the row-wise operators around a latent attention layer: the norms after a
// block and before the next one, with the block's gate and residual scale (k3moe_norm), and the
// write of the latent cache (k3moe_latent_write).  Both are one pass over their rows.
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"

namespace k3moe {
namespace {

// Eight elements as they are stored: bf16 in 16 bytes, f32 in 32.
struct Eight {
    uint4 lo, hi;
};
__device__ __forceinline__ Eight load8(const void *base, bool f32, size_t at)
{
    Eight e;
    if (f32) {
        const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(base) + at);
        e.lo = p[0];
        e.hi = p[1];
    } else {
        e.lo = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + at);
        e.hi = make_uint4(0, 0, 0, 0);
    }
    return e;
}
__device__ __forceinline__ void bf16x8(uint4 w, float (&x)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void floats(const Eight &e, bool f32, float (&x)[8])
{
    if (f32) {
        const uint32_t u[8] = {e.lo.x, e.lo.y, e.lo.z, e.lo.w, e.hi.x, e.hi.y, e.hi.z, e.hi.w};
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = __uint_as_float(u[i]);
    } else {
        bf16x8(e.lo, x);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 w = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&w);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(void *base, bool f32, size_t at, const float (&x)[8])
{
    if (f32) {
        float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(base) + at);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(base) + at) = pack8(x);
    }
}
__device__ __forceinline__ void load_gain8(const float *g, size_t at, float (&x)[8])
{
    const float4 *p = reinterpret_cast<const float4 *>(g + at);
    const float4 a = p[0], b = p[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
// Sum over the lanes that share lane / width, width a power of two up to 32.
__device__ __forceinline__ float lanes_sum(float v, int width)
{
    for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------- norms around a block
// A row is `tpr` threads', each V pieces of 8 columns, held in registers from the one read to
// the writes; blocks of short rows hold several.  A group's sum is of 8, 16 or 32 neighbouring
// lanes, a row's of all its warps.
constexpr int kNormThreads = 256;

template <int V>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a, const int tpr)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float part[2][32];
    const int in_row = threadIdx.x % tpr, row_in_block = threadIdx.x / tpr, rows = blockDim.x / tpr;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row_warps = tpr >> 5;
    const int t = blockIdx.x * rows + row_in_block;
    const int pieces = a.N >> 3;
    const bool live = t < a.T;
    Eight xe[V], re[V];
    uint4 ge[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int p = in_row + i * tpr;
        const bool in = live && p < pieces;
        xe[i].lo = xe[i].hi = re[i].lo = re[i].hi = ge[i] = make_uint4(0, 0, 0, 0);
        if (in) xe[i] = load8(a.x, a.x_f32, (size_t)t * a.x_stride + 8 * p);
        if (in && a.gate) ge[i] = *reinterpret_cast<const uint4 *>(a.gate + (size_t)t * a.gate_stride + 8 * p);
        if (in && a.residual) re[i] = load8(a.residual, a.sum_f32, (size_t)t * a.residual_stride + 8 * p);
    }
    // the sum of every thread's share over its row
    auto row_sum = [&](float v, int turn) {
        v = lanes_sum(v, 32);
        if (row_warps == 1) return v;
        if (lane == 0) part[turn][warp] = v;
        __syncthreads();
        float s = 0.0f;
        for (int w = 0; w < row_warps; w++) s += part[turn][row_in_block * row_warps + w];
        return s;
    };
    float y[V][8], inv[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        floats(xe[i], a.x_f32, y[i]);
        inv[i] = 1.0f;
    }
    if (a.post_norm) {
        float ss[V], all = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            ss[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; j++) ss[i] = fmaf(y[i][j], y[i][j], ss[i]);
            all += ss[i];
        }
        if (a.group == a.N) {
            const float r = 1.0f / sqrtf(row_sum(all, 0) / (float)a.N + a.eps);
#pragma unroll
            for (int i = 0; i < V; i++) inv[i] = r;
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) inv[i] = 1.0f / sqrtf(lanes_sum(ss[i], a.group >> 3) / (float)a.group + a.eps);
        }
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int p = in_row + i * tpr;
        if (!live || p >= pieces) continue;
        float w[8];
        if (a.post_norm) {
            load_gain8(a.post_gain, a.group == a.N ? 8 * p : (8 * p) & (a.group - 1), w);
#pragma unroll
            for (int j = 0; j < 8; j++) y[i][j] = y[i][j] * inv[i] * w[j];
        }
        if (a.gate_act != K3MOE_GATE_NONE) {
            bf16x8(ge[i], w);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float s = 1.0f / (1.0f + expf(-w[j]));
                y[i][j] *= a.gate_act == K3MOE_GATE_SILU ? w[j] * s : s;
            }
        }
        if (a.alpha != 1.0f)
#pragma unroll
            for (int j = 0; j < 8; j++) y[i][j] *= a.alpha;
        if (a.scale) {
            load_gain8(a.scale, 8 * p, w);
#pragma unroll
            for (int j = 0; j < 8; j++) y[i][j] *= w[j];
        }
        if (a.residual) {
            floats(re[i], a.sum_f32, w);
#pragma unroll
            for (int j = 0; j < 8; j++) y[i][j] += w[j];
        }
        if (a.total) store8(a.total, a.sum_f32, (size_t)t * a.total_stride + 8 * p, y[i]);
#pragma unroll
        for (int j = 0; j < 8; j++) sq = fmaf(y[i][j], y[i][j], sq);
    }
    if (!a.pre_norm) return;
    const float r = 1.0f / sqrtf(row_sum(sq, 1) / (float)a.N + a.eps);
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int p = in_row + i * tpr;
        if (!live || p >= pieces) continue;
        float w[8];
        load_gain8(a.pre_gain, 8 * p, w);
#pragma unroll
        for (int j = 0; j < 8; j++) w[j] *= y[i][j] * r;
        store8(a.out, false, (size_t)t * a.out_stride + 8 * p, w);
    }
}

template <int V>
cudaError_t launch_norm_as(const NormArgs &a, int tpr, cudaStream_t s)
{
    const int rows = std::max(1, kNormThreads / tpr);
    return launch_pdl(norm_kernel<V>, dim3((unsigned)((a.T + rows - 1) / rows)), dim3((unsigned)(tpr * rows)), 0, s, a, tpr);
}

// ---------------------------------------------------------------- the cache's write
// A block a token: threads of the row's 72 pieces of 8 columns norm c (64 of them) and turn r,
// then all turn the queries' heads.  An angle is the position times the frequency in turns as a
// 64-bit fraction: the product drops whole turns by itself, and what it loses is the frequency's rounding
// to 2^-64 turns times the position.
constexpr int kWriteThreads = 128;

// Columns a pair of 8-column pieces has, of the four pairs a rotated head is made of.
__device__ __forceinline__ int rope_first(int how, int j) { return how == K3MOE_ROPE_PAIRS ? 16 * j : 8 * j; }
__device__ __forceinline__ int rope_second(int how, int j) { return how == K3MOE_ROPE_PAIRS ? 16 * j + 8 : 8 * j + kLatR / 2; }
// Turns pair j's 16 columns u, v by the angles 8 j .. 8 j + 7.
__device__ __forceinline__ void rope_turn(int how, const float2 *turn, int j, float (&u)[8], float (&v)[8])
{
    if (how == K3MOE_ROPE_HALVES) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 t = turn[8 * j + i];
            const float x = u[i], y = v[i];
            u[i] = x * t.x - y * t.y;
            v[i] = y * t.x + x * t.y;
        }
    } else if (how == K3MOE_ROPE_PAIRS) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 t = turn[8 * j + i / 2], w = turn[8 * j + 4 + i / 2];
            float x = u[i], y = u[i + 1];
            u[i] = x * t.x - y * t.y;
            u[i + 1] = y * t.x + x * t.y;
            x = v[i];
            y = v[i + 1];
            v[i] = x * w.x - y * w.y;
            v[i + 1] = y * w.x + x * w.y;
        }
    }
}

__global__ void __launch_bounds__(kWriteThreads) latent_write_kernel(const LatentWriteArgs a)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float2 turn[kLatR / 2];                        // cosine, sine
    __shared__ float part[2];
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 3 && a.rope != K3MOE_ROPE_NONE) {
        const double turns = a.inv_freq[lane] * 0.15915494309189533577;       // a position's, 1 / (2 pi)
        const unsigned long long f = (unsigned long long)(long long)__double2ll_rn((turns - rint(turns)) * 18446744073709551616.0 * 0.5) << 1;
        const long long angle = (long long)(f * (unsigned long long)(long long)a.positions[t]);
        float sn, cs;
        sincospif((float)angle * 1.0842021724855044e-19f, &sn, &cs);          // 2^-63: half turns
        turn[lane] = make_float2(cs, sn);
    }
    const uint16_t *c = a.c + (size_t)t * a.c_stride;
    float x[8];
    float ss = 0.0f;
    if (threadIdx.x < kLatC / 8) {
        bf16x8(*reinterpret_cast<const uint4 *>(c + 8 * threadIdx.x), x);
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(x[j], x[j], ss);
        ss = lanes_sum(ss, 32);
        if (lane == 0) part[warp] = ss;
    }
    __syncthreads();
    int64_t slot = a.cache ? a.slots[t] : -1;
    if (slot >= a.n_slots) {
        if (threadIdx.x == 0) set_status(a.status, K3MOE_DEV_BAD_INDEX);
        slot = -1;
    }
    uint16_t *row = a.rows ? a.rows + (size_t)t * a.rows_stride : nullptr;
    uint16_t *cached = slot >= 0 ? a.cache + (size_t)slot * kLatRow : nullptr;
    auto put = [&](int at, const float (&v)[8]) {
        const uint4 w = pack8(v);
        if (row) *reinterpret_cast<uint4 *>(row + at) = w;
        if (cached) *reinterpret_cast<uint4 *>(cached + at) = w;
    };
    if (threadIdx.x < kLatC / 8) {
        if (a.norm) {
            const float r = 1.0f / sqrtf((part[0] + part[1]) * (1.0f / kLatC) + a.eps);
            float g[8];
            load_gain8(a.gain, 8 * threadIdx.x, g);
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = x[j] * r * g[j];
        }
        put(8 * threadIdx.x, x);
    } else if (threadIdx.x < kLatC / 8 + 4) {
        const int j = threadIdx.x - kLatC / 8, u0 = kLatC + rope_first(a.rope, j), v0 = kLatC + rope_second(a.rope, j);
        float v[8];
        bf16x8(*reinterpret_cast<const uint4 *>(c + u0), x);
        bf16x8(*reinterpret_cast<const uint4 *>(c + v0), v);
        rope_turn(a.rope, turn, j, x, v);
        put(u0, x);
        put(v0, v);
    }
    if (!a.q) return;
    const uint16_t *q = a.q + (size_t)t * a.q_stride;
    uint16_t *o = a.q_rope + (size_t)t * a.r_stride;
    for (int i = threadIdx.x; i < 4 * a.H; i += kWriteThreads) {
        const int h = i >> 2, j = i & 3, u0 = rope_first(a.rope, j), v0 = rope_second(a.rope, j);
        float u[8], v[8];
        bf16x8(*reinterpret_cast<const uint4 *>(q + h * a.q_head + u0), u);
        bf16x8(*reinterpret_cast<const uint4 *>(q + h * a.q_head + v0), v);
        rope_turn(a.rope, turn, j, u, v);
        *reinterpret_cast<uint4 *>(o + h * a.r_head + u0) = pack8(u);
        *reinterpret_cast<uint4 *>(o + h * a.r_head + v0) = pack8(v);
    }
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, cudaStream_t s)
{
    const int pieces = a.N / 8;
    const auto warps = [](int n) { return (n + 31) / 32 * 32; };
    timing_begin("norm", s);
    // few columns a thread while the row fits a block that way, four pieces of long rows
    const cudaError_t err = pieces <= 256 ? launch_norm_as<1>(a, warps(pieces), s)
                            : pieces <= 512 ? launch_norm_as<2>(a, warps((pieces + 1) / 2), s)
                                            : launch_norm_as<4>(a, warps((pieces + 3) / 4), s);
    count_launch();
    timing_end("norm", s);
    return err;
}

cudaError_t launch_latent_write(const LatentWriteArgs &a, cudaStream_t s)
{
    timing_begin("latent_write", s);
    const cudaError_t err = launch_pdl(latent_write_kernel, dim3((unsigned)a.T), dim3(kWriteThreads), 0, s, a);
    count_launch();
    timing_end("latent_write", s);
    return err;
}

}  // namespace k3moe
