// k3moe_norm.cu -- the row-wise operators around a latent attention layer: the norms after a
// block and before the next one, with the block's gate and residual scale (k3moe_norm), and the
// write of the latent cache (k3moe_latent_write).  Both are one pass over their rows.
#include <cuda_bf16.h>

#include "k3moe_tc_warp.cuh"

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
// As pairs of floats, the form that most of the arithmetic here takes.
__device__ __forceinline__ void bf16x8(uint4 w, uint64_t (&x)[4])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) x[i] = pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
}
__device__ __forceinline__ void pairs(const Eight &e, bool f32, uint64_t (&x)[4])
{
    if (f32) {
        const uint32_t u[8] = {e.lo.x, e.lo.y, e.lo.z, e.lo.w, e.hi.x, e.hi.y, e.hi.z, e.hi.w};
#pragma unroll
        for (int i = 0; i < 4; i++) x[i] = pack2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
    } else {
        bf16x8(e.lo, x);
    }
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&x)[4])
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 v = unpack2(x[i]);
        const __nv_bfloat162 w = __floats2bfloat162_rn(v.x, v.y);
        u[i] = *reinterpret_cast<const uint32_t *>(&w);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(void *base, bool f32, size_t at, const uint64_t (&x)[4])
{
    if (f32) {
        float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(base) + at);
        const float2 a = unpack2(x[0]), b = unpack2(x[1]), c = unpack2(x[2]), d = unpack2(x[3]);
        p[0] = make_float4(a.x, a.y, b.x, b.y);
        p[1] = make_float4(c.x, c.y, d.x, d.y);
    } else {
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(base) + at) = pack8(x);
    }
}
__device__ __forceinline__ void load_gain8(const float *g, size_t at, uint64_t (&x)[4])
{
    const float4 *p = reinterpret_cast<const float4 *>(g + at);
    const float4 a = p[0], b = p[1];
    x[0] = pack2(a.x, a.y);
    x[1] = pack2(a.z, a.w);
    x[2] = pack2(b.x, b.y);
    x[3] = pack2(b.z, b.w);
}
__device__ __forceinline__ float squares(const uint64_t (&x)[4])
{
    uint64_t s = mul2(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 4; i++) s = fma2(x[i], x[i], s);
    const float2 v = unpack2(s);
    return v.x + v.y;
}
// Sum over the lanes that share lane / width, width a power of two up to 32.
__device__ __forceinline__ float lanes_sum(float v, int width)
{
    for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------- norms around a block
// 1 / (1 + exp(-z)) of two within a few units of their last place, or zero below 2^-125: the exponential's argument in
// powers of two is a rounded product t and its remainder r, exp(-z) = 2^t (1 + r ln 2).
__device__ __forceinline__ uint64_t sigmoid2(uint64_t z2)
{
    float2 z = unpack2(z2);
    asm("max.NaN.f32 %0, %0, 0fC2B10000;" : "+f"(z.x));       // -88.5: 2^t stays finite, its reciprocal is zero
    asm("max.NaN.f32 %0, %0, 0fC2B10000;" : "+f"(z.y));
    z2 = pack2(z.x, z.y);
    const uint64_t log2e = pack2(-1.442695022f, -1.442695022f), rest = pack2(-1.925963033e-8f, -1.925963033e-8f);
    const uint64_t t2 = mul2(z2, log2e), minus = pack2(-1.0f, -1.0f);
    const uint64_t r = fma2(z2, rest, fma2(z2, log2e, mul2(t2, minus)));
    const float2 t = unpack2(t2);
    const uint64_t e = pack2(exp2_fast(t.x), exp2_fast(t.y));
    const float2 d = unpack2(add2(fma2(mul2(e, pack2(0.6931471806f, 0.6931471806f)), r, e), pack2(1.0f, 1.0f)));
    float2 s;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(d.y));
    return pack2(s.x, s.y);
}

// A row is `tpr` threads', each V pieces of 8 columns, held in registers from the one read to
// the writes; blocks of short rows hold several.  A group's sum is of 8, 16 or 32 neighbouring
// lanes, a row's of all its warps.  Many rows are bound by their bytes (8192 x 7168, each head's norm with a gate:
// MANY us, RATE TB/s); a row alone by latency, so it takes as many threads as it has pieces, and their gains are asked for
// with the row (1 x 7168 with all there is: ONE us in a graph; four pieces a thread, gains when they are needed 7.0).
template <int V> constexpr int kNormMax = V == 4 ? 512 : 1024;
constexpr int kNormThreads = 256;

template <int V>
__global__ void __launch_bounds__(kNormMax<V>) norm_kernel(const NormArgs a, const int tpr)
{
    constexpr bool kEarly = V == 1;
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
    uint64_t post[4], scale[4], pre[4];
    auto post_at = [&](int p) { return a.group == a.N ? 8 * p : (8 * p) & (a.group - 1); };
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int p = in_row + i * tpr;
        const bool in = live && p < pieces;
        xe[i].lo = xe[i].hi = re[i].lo = re[i].hi = ge[i] = make_uint4(0, 0, 0, 0);
        if (in) xe[i] = load8(a.x, a.x_f32, (size_t)t * a.x_stride + 8 * p);
        if (in && a.gate) ge[i] = *reinterpret_cast<const uint4 *>(a.gate + (size_t)t * a.gate_stride + 8 * p);
        if (in && a.residual) re[i] = load8(a.residual, a.sum_f32, (size_t)t * a.residual_stride + 8 * p);
        if (kEarly && in) {
            if (a.post_norm) load_gain8(a.post_gain, post_at(p), post);
            if (a.scale) load_gain8(a.scale, 8 * p, scale);
            if (a.pre_norm) load_gain8(a.pre_gain, 8 * p, pre);
        }
    }
    // the sum of every thread's share over its row
    auto row_sum = [&](float v, int turn) {
        v = lanes_sum(v, 32);
        if (row_warps == 1) return v;
        if (lane == 0) part[turn][warp] = v;
        __syncthreads();
        v = lane < row_warps ? part[turn][row_in_block * row_warps + lane] : 0.0f;
        return lanes_sum(v, 32);
    };
    uint64_t y[V][4];                                         // pairs of columns
    float inv[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        pairs(xe[i], a.x_f32, y[i]);
        inv[i] = 1.0f;
    }
    if (a.post_norm) {
        float ss[V], all = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            ss[i] = squares(y[i]);
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
        const float f = inv[i] * a.alpha;
#pragma unroll
        for (int j = 0; j < 4; j++) y[i][j] = mul2(y[i][j], pack2(f, f));
        if (a.post_norm) {
            if (!kEarly) load_gain8(a.post_gain, post_at(p), post);
#pragma unroll
            for (int j = 0; j < 4; j++) y[i][j] = mul2(y[i][j], post[j]);
        }
        if (a.gate_act != K3MOE_GATE_NONE) {
            uint64_t w[4];
            bf16x8(ge[i], w);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                y[i][j] = mul2(y[i][j], sigmoid2(w[j]));
                if (a.gate_act == K3MOE_GATE_SILU) y[i][j] = mul2(y[i][j], w[j]);
            }
        }
        if (a.scale) {
            if (!kEarly) load_gain8(a.scale, 8 * p, scale);
#pragma unroll
            for (int j = 0; j < 4; j++) y[i][j] = mul2(y[i][j], scale[j]);
        }
        if (a.residual) {
            uint64_t w[4];
            pairs(re[i], a.sum_f32, w);
#pragma unroll
            for (int j = 0; j < 4; j++) y[i][j] = add2(y[i][j], w[j]);
        }
        if (a.total) store8(a.total, a.sum_f32, (size_t)t * a.total_stride + 8 * p, y[i]);
        if (a.pre_norm) sq += squares(y[i]);
    }
    if (!a.pre_norm) return;
    const float r = 1.0f / sqrtf(row_sum(sq, 1) / (float)a.N + a.eps);
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int p = in_row + i * tpr;
        if (!live || p >= pieces) continue;
        if (!kEarly) load_gain8(a.pre_gain, 8 * p, pre);
        uint64_t w[4];
#pragma unroll
        for (int j = 0; j < 4; j++) w[j] = mul2(pre[j], mul2(y[i][j], pack2(r, r)));
        store8(a.out, false, (size_t)t * a.out_stride + 8 * p, w);
    }
}

template <int V>
cudaError_t launch_norm_as(const NormArgs &a, cudaStream_t s)
{
    const int tpr = (a.N / 8 + 32 * V - 1) / (32 * V) * 32, rows = std::max(1, kNormThreads / tpr);
    return launch_pdl(norm_kernel<V>, dim3((unsigned)((a.T + rows - 1) / rows)), dim3((unsigned)(tpr * rows)), 0, s, a, tpr);
}

// ---------------------------------------------------------------- the cache's write
// A block a token: threads of the row's 72 pieces of 8 columns norm c (64 of them) and turn r,
// then all turn the queries' heads.  An angle is the position times the frequency in turns as a
// 64-bit fraction: the product drops whole turns by itself, and what it loses is the frequency's rounding
// to 2^-64 turns times the position.
constexpr int kWriteThreads = 128, kWriteDeep = 2;

// Columns a pair of 8-column pieces has, of the four pairs a rotated head is made of.
__device__ __forceinline__ int rope_first(int how, int j) { return how == K3MOE_ROPE_PAIRS ? 16 * j : 8 * j; }
__device__ __forceinline__ int rope_second(int how, int j) { return how == K3MOE_ROPE_PAIRS ? 16 * j + 8 : 8 * j + kLatR / 2; }
// Turns pair j's 16 columns u, v by the angles 8 j .. 8 j + 7: of (x, y), (x cos - y sin, y cos + x sin).
__device__ __forceinline__ void rope_turn(int how, const float *cosine, const float *sine, int j, uint64_t (&u)[4], uint64_t (&v)[4])
{
    const float4 *c = reinterpret_cast<const float4 *>(cosine + 8 * j), *s = reinterpret_cast<const float4 *>(sine + 8 * j);
    const float4 c0 = c[0], c1 = c[1], s0 = s[0], s1 = s[1];
    if (how == K3MOE_ROPE_HALVES) {
        const uint64_t cs[4] = {pack2(c0.x, c0.y), pack2(c0.z, c0.w), pack2(c1.x, c1.y), pack2(c1.z, c1.w)};
        const uint64_t sn[4] = {pack2(s0.x, s0.y), pack2(s0.z, s0.w), pack2(s1.x, s1.y), pack2(s1.z, s1.w)};
        const uint64_t minus = pack2(-1.0f, -1.0f);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint64_t x = u[i], y = v[i];
            u[i] = fma2(x, cs[i], mul2(mul2(y, sn[i]), minus));
            v[i] = fma2(y, cs[i], mul2(x, sn[i]));
        }
    } else if (how == K3MOE_ROPE_PAIRS) {
        auto one = [](uint64_t p, float c, float s) {
            const float2 x = unpack2(p);
            return fma2(p, pack2(c, c), mul2(pack2(x.y, x.x), pack2(-s, s)));
        };
        u[0] = one(u[0], c0.x, s0.x);
        u[1] = one(u[1], c0.y, s0.y);
        u[2] = one(u[2], c0.z, s0.z);
        u[3] = one(u[3], c0.w, s0.w);
        v[0] = one(v[0], c1.x, s1.x);
        v[1] = one(v[1], c1.y, s1.y);
        v[2] = one(v[2], c1.z, s1.z);
        v[3] = one(v[3], c1.w, s1.w);
    }
}

__global__ void __launch_bounds__(kWriteThreads) latent_write_kernel(const LatentWriteArgs a)
{
    pdl_wait();
    pdl_trigger();
    __shared__ __align__(16) float cosine[kLatR / 2], sine[kLatR / 2];
    __shared__ float part[2];
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t *c = a.c + (size_t)t * a.c_stride, *q = a.q + (size_t)t * a.q_stride;
    uint16_t *o = a.q_rope + (size_t)t * a.r_stride;
    // the queries' pieces are asked for with the row: up to kWriteDeep a thread at a time
    const int j = threadIdx.x & 3, u0 = rope_first(a.rope, j), v0 = rope_second(a.rope, j), heads = a.q ? a.H : 0;
    uint4 qu[kWriteDeep], qv[kWriteDeep];
    auto ask = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kWriteDeep; i++) {
            const int h = h0 + i * (kWriteThreads / 4);
            if (h >= heads) break;
            qu[i] = *reinterpret_cast<const uint4 *>(q + h * a.q_head + u0);
            qv[i] = *reinterpret_cast<const uint4 *>(q + h * a.q_head + v0);
        }
    };
    ask(threadIdx.x >> 2);
    int64_t slot = a.cache ? a.slots[t] : -1;
    uint64_t x[4], g[4], v[4];
    float ss = 0.0f;
    if (threadIdx.x < kLatC / 8) {
        bf16x8(*reinterpret_cast<const uint4 *>(c + 8 * threadIdx.x), x);
        if (a.norm) load_gain8(a.gain, 8 * threadIdx.x, g);
        ss = lanes_sum(squares(x), 32);
        if (lane == 0) part[warp] = ss;
    } else if (warp == 2) {
        if (lane < 4) {
            bf16x8(*reinterpret_cast<const uint4 *>(c + kLatC + u0), x);
            bf16x8(*reinterpret_cast<const uint4 *>(c + kLatC + v0), v);
        }
    } else if (a.rope != K3MOE_ROPE_NONE) {
        const double turns = a.inv_freq[lane] * 0.15915494309189533577;       // a position's, 1 / (2 pi)
        const unsigned long long f = (unsigned long long)__double2ll_rn((turns - rint(turns)) * 9223372036854775808.0) << 1;
        const long long angle = (long long)(f * (unsigned long long)(long long)a.positions[t]);
        sincospif((float)angle * 1.0842021724855044e-19f, &sine[lane], &cosine[lane]);    // 2^-63: half turns
    }
    __syncthreads();
    if (slot >= a.n_slots) {
        if (threadIdx.x == 0) set_status(a.status, K3MOE_DEV_BAD_INDEX);
        slot = -1;
    }
    uint16_t *row = a.rows ? a.rows + (size_t)t * a.rows_stride : nullptr;
    uint16_t *cached = slot >= 0 ? a.cache + (size_t)slot * kLatRow : nullptr;
    auto put = [&](int at, const uint64_t (&v)[4]) {
        const uint4 w = pack8(v);
        if (row) *reinterpret_cast<uint4 *>(row + at) = w;
        if (cached) *reinterpret_cast<uint4 *>(cached + at) = w;
    };
    if (threadIdx.x < kLatC / 8) {
        if (a.norm) {
            const float r = 1.0f / sqrtf((part[0] + part[1]) * (1.0f / kLatC) + a.eps);
#pragma unroll
            for (int i = 0; i < 4; i++) x[i] = mul2(mul2(x[i], pack2(r, r)), g[i]);
        }
        put(8 * threadIdx.x, x);
    } else if (threadIdx.x < kLatC / 8 + 4) {
        rope_turn(a.rope, cosine, sine, j, x, v);
        put(kLatC + u0, x);
        put(kLatC + v0, v);
    }
    for (int h0 = threadIdx.x >> 2; h0 < heads; h0 += kWriteDeep * (kWriteThreads / 4)) {
        if (h0 >= kWriteDeep * (kWriteThreads / 4)) ask(h0);
#pragma unroll
        for (int i = 0; i < kWriteDeep; i++) {
            const int h = h0 + i * (kWriteThreads / 4);
            if (h >= heads) break;
            bf16x8(qu[i], x);
            bf16x8(qv[i], v);
            rope_turn(a.rope, cosine, sine, j, x, v);
            *reinterpret_cast<uint4 *>(o + h * a.r_head + u0) = pack8(x);
            *reinterpret_cast<uint4 *>(o + h * a.r_head + v0) = pack8(v);
        }
    }
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, cudaStream_t s)
{
    timing_begin("norm", s);
    // a piece a thread for rows of up to 2048 columns and for a few longer ones, else two, and four for the longest
    const bool few = a.T <= num_sms();
    const cudaError_t err = a.N <= 2048 || (few && a.N <= 8192) ? launch_norm_as<1>(a, s)
                            : a.N <= 8192 || few               ? launch_norm_as<2>(a, s)
                                                               : launch_norm_as<4>(a, s);
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
