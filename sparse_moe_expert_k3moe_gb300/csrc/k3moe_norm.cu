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
        if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {      // a sector at once
            asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
                         "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                         : "memory");
        } else {
            p[0] = make_float4(x[0], x[1], x[2], x[3]);
            p[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
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
__device__ __forceinline__ float squares(const float (&x)[8])
{
    float s = x[0] * x[0];
#pragma unroll
    for (int i = 1; i < 8; i++) s = fmaf(x[i], x[i], s);
    return s;
}
// Sum over the lanes that share lane / width, width a power of two up to 32.
__device__ __forceinline__ float lanes_sum(float v, int width)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, v, o);
        v += o < width ? x : 0.0f;
    }
    return v;
}

// ---------------------------------------------------------------- norms around a block
// 1 / (1 + exp(-z)) within a few units of its last place, or zero below 2^-125: with t = -z log2 e rounded and
// r = -z - t ln 2 (ln 2 in two floats), exp(-z) = 2^t (1 + r).
__device__ __forceinline__ float sigmoid(float z)
{
    asm("max.NaN.f32 %0, %0, 0fC2B10000;\n\tmin.NaN.f32 %0, %0, 0f42B10000;" : "+f"(z));    // within 88.5: 2^t stays finite
    const float t = z * -1.442695041f, r = fmaf(t, 1.904654300e-9f, fmaf(t, -0.6931471825f, -z)), e = exp2_fast(t);
    float s;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(fmaf(e, r, e) + 1.0f));
    return s;
}
// The same to (6 + |z|) 2^-24 of it, for sums that are rounded to bf16: t's rounding is left where it is, and 2^t may pass into infinity.
__device__ __forceinline__ float sigmoid_short(float z)
{
    float s;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(exp2_fast(z * -1.442695041f) + 1.0f));
    return s;
}

// A row is `tpr` threads', each V pieces of 8 columns, held in registers from the one read to
// the writes; blocks of short rows hold several.  A group's sum is of 8, 16 or 32 neighbouring
// lanes, a row's of all its warps.  Fewer rows are bound by latency: one alone takes as many threads as it has pieces, and their
// gains are asked for with the row (1 x 7168 with all there is: 3.3 us in a graph; four pieces a thread, gains when they are needed 7.0).
// Many rows are the kernel's below.
template <int V> constexpr int kNormMax = V == 1 ? 1024 : 512;
constexpr int kNormThreads = 256;
constexpr int kStreamN = 512, kStreamRows = 4, kStreamRing = 208 * 1024;         // rows that are long, and as many an SM that are many

template <int V, bool kX32, bool kSum32, int kGate>
__global__ void __launch_bounds__(kNormMax<V>, V == 2 && !kX32 && !kSum32 ? 3 : 1) norm_kernel(const NormArgs a, const float per_row, const float per_group)
{
    constexpr bool kEarly = V == 1;
    pdl_wait();
    pdl_trigger();
    __shared__ float part[2][32];
    const int tpr = blockDim.x, in_row = threadIdx.x, row_in_block = threadIdx.y;
    const int lane = in_row & 31, row_warps = tpr >> 5, warp = row_in_block * row_warps + (in_row >> 5);
    const int t = blockIdx.x * blockDim.y + row_in_block;
    const int pieces = a.N >> 3;
    const bool live = t < a.T;
    Eight xe[V], re[V];
    uint4 ge[V];
    float post[8], scale[8], pre[8];
    auto post_at = [&](int p) { return a.group == a.N ? 8 * p : (8 * p) & (a.group - 1); };
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int p = in_row + i * tpr;
        const bool in = live && p < pieces;
        xe[i].lo = xe[i].hi = re[i].lo = re[i].hi = ge[i] = make_uint4(0, 0, 0, 0);
        if (in) xe[i] = load8(a.x, kX32, (size_t)t * a.x_stride + 8 * p);
        if (in && kGate != K3MOE_GATE_NONE) ge[i] = *reinterpret_cast<const uint4 *>(a.gate + (size_t)t * a.gate_stride + 8 * p);
        if (in && a.residual) re[i] = load8(a.residual, kSum32, (size_t)t * a.residual_stride + 8 * p);
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
    float y[V][8], inv[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        floats(xe[i], kX32, y[i]);
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
            const float r = rsqrtf(fmaf(row_sum(all, 0), per_row, a.eps));
#pragma unroll
            for (int i = 0; i < V; i++) inv[i] = r;
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) inv[i] = rsqrtf(fmaf(lanes_sum(ss[i], a.group >> 3), per_group, a.eps));
        }
    }
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int p = in_row + i * tpr;
        if (!live || p >= pieces) continue;
        const float f = inv[i] * a.alpha;
#pragma unroll
        for (int j = 0; j < 8; j++) y[i][j] *= f;
        if (a.post_norm) {
            if (!kEarly) load_gain8(a.post_gain, post_at(p), post);
#pragma unroll
            for (int j = 0; j < 8; j++) y[i][j] *= post[j];
        }
        if (kGate != K3MOE_GATE_NONE) {
            float w[8];
            bf16x8(ge[i], w);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                y[i][j] *= kSum32 ? sigmoid(w[j]) : sigmoid_short(w[j]);
                if (kGate == K3MOE_GATE_SILU) y[i][j] *= w[j];
            }
        }
        if (a.scale) {
            if (!kEarly) load_gain8(a.scale, 8 * p, scale);
#pragma unroll
            for (int j = 0; j < 8; j++) y[i][j] *= scale[j];
        }
        if (a.residual) {
            float w[8];
            floats(re[i], kSum32, w);
#pragma unroll
            for (int j = 0; j < 8; j++) y[i][j] += w[j];
        }
        if (a.total) store8(a.total, kSum32, (size_t)t * a.total_stride + 8 * p, y[i]);
        if (a.pre_norm) sq += squares(y[i]);
    }
    if (!a.pre_norm) return;
    const float r = rsqrtf(fmaf(row_sum(sq, 1), per_row, a.eps));
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int p = in_row + i * tpr;
        if (!live || p >= pieces) continue;
        if (!kEarly) load_gain8(a.pre_gain, 8 * p, pre);
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; j++) w[j] = pre[j] * (y[i][j] * r);
        store8(a.out, false, (size_t)t * a.out_stride + 8 * p, w);
    }
}

// Many rows of 512 columns and more: the blocks that fill an SM take every so many rows, a thread 8 columns of each.  Its gains stay in registers (all
// three have three times the bytes of a bf16 row), and the next rows' pieces are asked for ahead (kStages - 1 of them) into shared
// memory, so that the two sums over a row cost no load's wait.  Bound by the bytes: 8192 x 7168, each head's norm with a gate, 54 us
// (6.5 TB/s; a row a block, or several short ones, 60.7), 4096 x 7168 with a residual and both norms 41.2 (47.9), with f32 sums 53.9
// (69.8), 8192 x 1024 13.4 (18.1), 4000 x 2048 13.0 (17.8), 8192 x 512 5.7 either way.  Of blocks as many as the registers hold: one less
// leaves loads unasked (8192 x 2200 33.0 against 26.5), one more waits for a place (4000 x 2048 17.0).  Two or four stages are
// within 2% where a row is long, but for 4000 x 3000 (31.7, 26.0 against 25.4).
__device__ __forceinline__ void ahead16(uint8_t *to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(saddr(to)), "l"(from) : "memory");
}
template <int kStages, bool kX32, bool kSum32, int kGate>
__global__ void __launch_bounds__(1024, 1) norm_stream_kernel(const NormArgs a, const float per_row, const float per_group)
{
    extern __shared__ __align__(128) uint8_t ring[];          // [stage]: x, gate and residual, each thread's 8 columns side by side
    __shared__ float part[2][2][32];
    constexpr int kX = kX32 ? 2 : 1, kG = kGate != K3MOE_GATE_NONE ? 1 : 0, kR = kSum32 ? 2 : 1, kPieces = kX + kG + kR;
    const int p = threadIdx.x, lane = p & 31, warp = p >> 5, warps = blockDim.x >> 5;
    const bool in = p < a.N >> 3;
    auto place = [&](int stage, int piece) { return ring + (stage * kPieces + piece) * blockDim.x * 16; };
    // a warp's 32 bytes a thread of an f32 row, in the order of their addresses: whole sectors
    auto ask_f32 = [&](int stage, int piece, const void *x, int64_t at) {
        const float *row = static_cast<const float *>(x) + at;
#pragma unroll
        for (int q = 64 * warp + lane, k = 0; k < 2; k++, q += 32)
            if (q < a.N >> 2) ahead16(place(stage, piece) + 16 * q, row + 4 * q);
    };
    auto ask_bf16 = [&](int stage, int piece, const void *x, int64_t at) { ahead16(place(stage, piece) + 16 * p, static_cast<const uint16_t *>(x) + at + 8 * p); };
    pdl_wait();
    pdl_trigger();
    auto ask = [&](int t, int stage) {
        if (in && t < a.T) {
            if (!kX32) ask_bf16(stage, 0, a.x, t * a.x_stride);
            if (kG) ask_bf16(stage, kX, a.gate, t * a.gate_stride);
            if (!kSum32 && a.residual) ask_bf16(stage, kX + kG, a.residual, t * a.residual_stride);
        }
        if (kX32 && t < a.T) ask_f32(stage, 0, a.x, t * a.x_stride);
        if (kSum32 && a.residual && t < a.T) ask_f32(stage, kX + kG, a.residual, t * a.residual_stride);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; i++) ask(blockIdx.x + i * gridDim.x, i);
    float post[8], scale[8], pre[8];
#pragma unroll
    for (int j = 0; j < 8; j++) post[j] = scale[j] = pre[j] = 1.0f;
    if (in && a.post_norm) load_gain8(a.post_gain, a.group == a.N ? 8 * p : (8 * p) & (a.group - 1), post);
    if (in && a.scale) load_gain8(a.scale, 8 * p, scale);
    if (in && a.pre_norm) load_gain8(a.pre_gain, 8 * p, pre);
#pragma unroll
    for (int j = 0; j < 8; j++) post[j] *= a.alpha;
    auto row_sum = [&](float v, float *mine) {
        v = lanes_sum(v, 32);
        if (lane == 0) mine[warp] = v;
        __syncthreads();
        return lanes_sum(lane < warps ? mine[lane] : 0.0f, 32);
    };
    int stage = 0;
    for (int t = blockIdx.x, turn = 0; t < a.T; t += gridDim.x, turn ^= 1, stage = stage + 1 == kStages ? 0 : stage + 1) {
        if (kX32 || kSum32) __syncwarp();                     // the row before has been read: pieces are other lanes' too
        ask(t + (kStages - 1) * gridDim.x, stage == 0 ? kStages - 1 : stage - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        if (kX32 || kSum32) __syncwarp();
        float y[8] = {}, w[8];
        auto floats_at = [&](int first, bool f32, float(&v)[8]) { floats(load8(place(stage, first), f32, 8 * p), f32, v); };
        if (in) floats_at(0, kX32, y);
        if (a.post_norm) {
            const float ss = squares(y);
            const float r = a.group == a.N ? rsqrtf(fmaf(row_sum(ss, part[turn][0]), per_row, a.eps)) : rsqrtf(fmaf(lanes_sum(ss, a.group >> 3), per_group, a.eps));
#pragma unroll
            for (int j = 0; j < 8; j++) y[j] *= r;
        }
        float sq = 0.0f;
        if (in) {
#pragma unroll
            for (int j = 0; j < 8; j++) y[j] *= post[j];
            if (kG) {
                floats_at(kX, false, w);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    y[j] *= kSum32 ? sigmoid(w[j]) : sigmoid_short(w[j]);
                    if (kGate == K3MOE_GATE_SILU) y[j] *= w[j];
                }
            }
            if (a.scale)
#pragma unroll
                for (int j = 0; j < 8; j++) y[j] *= scale[j];
            if (a.residual) {
                floats_at(kX + kG, kSum32, w);
#pragma unroll
                for (int j = 0; j < 8; j++) y[j] += w[j];
            }
            if (a.total) store8(a.total, kSum32, (size_t)t * a.total_stride + 8 * p, y);
            sq = squares(y);
        }
        if (a.pre_norm) {
            const float r = rsqrtf(fmaf(row_sum(sq, part[turn][1]), per_row, a.eps));
            if (in) {
#pragma unroll
                for (int j = 0; j < 8; j++) w[j] = pre[j] * (y[j] * r);
                store8(a.out, false, (size_t)t * a.out_stride + 8 * p, w);
            }
        }
    }
}

template <int V, bool kX32, bool kSum32, int kGate>
cudaError_t launch_norm_as(const NormArgs &a, cudaStream_t s)
{
    const int threads = (a.N / 8 + 31) / 32 * 32, stage = threads * 16 * ((kX32 ? 2 : 1) + (kGate != K3MOE_GATE_NONE ? 1 : 0) + (kSum32 ? 2 : 1));
    if (V <= 2 && a.N >= kStreamN && a.T >= kStreamRows * num_sms()) {
        const bool three = 3 * stage <= kStreamRing;
        const auto kernel = three ? norm_stream_kernel<3, kX32, kSum32, kGate> : norm_stream_kernel<2, kX32, kSum32, kGate>;
        static const int warps = [] {                         // that fit an SM's registers, eight a thread at a time
            int most = 64;
            for (const void *k : {(const void *)norm_stream_kernel<3, kX32, kSum32, kGate>, (const void *)norm_stream_kernel<2, kX32, kSum32, kGate>}) {
                cudaFuncAttributes fa{};
                if (cudaFuncGetAttributes(&fa, k) != cudaSuccess) return 32;
                most = std::min(most, 65536 / 32 / ((fa.numRegs + 7) / 8 * 8));
            }
            return most;
        }();
        const int blocks = std::max(1, std::min(warps / (threads / 32), kStreamRing / (stage * (three ? 3 : 2))));    // an SM's
        if (a.T >= kStreamRows * blocks * num_sms()) {
            const cudaError_t allowed = once_a_device([] {
                const cudaError_t e = cudaFuncSetAttribute(norm_stream_kernel<3, kX32, kSum32, kGate>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamRing);
                return e != cudaSuccess ? e : cudaFuncSetAttribute(norm_stream_kernel<2, kX32, kSum32, kGate>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamRing);
            });
            if (allowed != cudaSuccess) return allowed;
            return launch_pdl(kernel, dim3((unsigned)(blocks * num_sms())), dim3((unsigned)threads), (size_t)stage * (three ? 3 : 2), s, a, 1.0f / (float)a.N,
                              1.0f / (float)a.group);
        }
    }
    const int tpr = (a.N / 8 + 32 * V - 1) / (32 * V) * 32, rows = std::max(1, kNormThreads / tpr);
    return launch_pdl(norm_kernel<V, kX32, kSum32, kGate>, dim3((unsigned)((a.T + rows - 1) / rows)), dim3((unsigned)tpr, (unsigned)rows), 0, s, a,
                      1.0f / (float)a.N, 1.0f / (float)a.group);
}
template <int V, bool kX32, bool kSum32> cudaError_t launch_norm_gate(const NormArgs &a, cudaStream_t s)
{
    return a.gate_act == K3MOE_GATE_SIGMOID ? launch_norm_as<V, kX32, kSum32, K3MOE_GATE_SIGMOID>(a, s)
           : a.gate_act == K3MOE_GATE_SILU  ? launch_norm_as<V, kX32, kSum32, K3MOE_GATE_SILU>(a, s)
                                            : launch_norm_as<V, kX32, kSum32, K3MOE_GATE_NONE>(a, s);
}
template <int V> cudaError_t launch_norm_types(const NormArgs &a, cudaStream_t s)
{
    return a.x_f32 ? (a.sum_f32 ? launch_norm_gate<V, true, true>(a, s) : launch_norm_gate<V, true, false>(a, s))
                   : (a.sum_f32 ? launch_norm_gate<V, false, true>(a, s) : launch_norm_gate<V, false, false>(a, s));
}

// ---------------------------------------------------------------- the cache's write
// A block a token: threads of the row's 72 pieces of 8 columns norm c (64 of them) and turn r,
// then all turn the queries' heads.  An angle is the position times the frequency in turns as a
// 64-bit fraction: the product drops whole turns by itself, and what it loses is the frequency's rounding
// to 2^-64 turns times the position.  Bound by the bytes: 8192 tokens x 56 heads 24.7 us (5.9 TB/s; one pair of the queries' pieces
// ahead 28.1; ten blocks an SM, whose registers spill, 35), 37 tokens 2.3.
constexpr int kWriteThreads = 128, kWriteDeep = 2;

// Columns a pair of 8-column pieces has, of the four pairs a rotated head is made of.
__device__ __forceinline__ int rope_first(int how, int j) { return how == K3MOE_ROPE_PAIRS ? 16 * j : 8 * j; }
__device__ __forceinline__ int rope_second(int how, int j) { return how == K3MOE_ROPE_PAIRS ? 16 * j + 8 : 8 * j + kLatR / 2; }
// Turns pair j's 16 columns u, v by the angles 8 j .. 8 j + 7: of (x, y), (x cos - y sin, y cos + x sin).
__device__ __forceinline__ void rope_turn(int how, const float *cosine, const float *sine, int j, float (&u)[8], float (&v)[8])
{
    if (how == K3MOE_ROPE_NONE) return;
    float c[8], s[8];
    load_gain8(cosine, 8 * j, c);
    load_gain8(sine, 8 * j, s);
    auto turn = [](float &x, float &y, float c, float s) {
        const float z = x;
        x = fmaf(z, c, -(y * s));
        y = fmaf(y, c, z * s);
    };
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if (how == K3MOE_ROPE_HALVES)
            turn(u[i], v[i], c[i], s[i]);
        else if (i < 4)
            turn(u[2 * i], u[2 * i + 1], c[i], s[i]);
        else
            turn(v[2 * i - 8], v[2 * i - 7], c[i], s[i]);
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
    float x[8], g[8], v[8];
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
    auto put = [&](int at, const float (&v)[8]) {
        const uint4 w = pack8(v);
        if (row) *reinterpret_cast<uint4 *>(row + at) = w;
        if (cached) *reinterpret_cast<uint4 *>(cached + at) = w;
    };
    if (threadIdx.x < kLatC / 8) {
        if (a.norm) {
            const float r = rsqrtf(fmaf(part[0] + part[1], 1.0f / kLatC, a.eps));
#pragma unroll
            for (int i = 0; i < 8; i++) x[i] = x[i] * r * g[i];
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
    const cudaError_t err = a.N <= 2048 || (few && a.N <= 8192) ? launch_norm_types<1>(a, s)
                            : a.N <= 8192                      ? launch_norm_types<2>(a, s)
                                                               : launch_norm_types<4>(a, s);
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
