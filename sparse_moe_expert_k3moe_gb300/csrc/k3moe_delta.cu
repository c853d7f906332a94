// k3moe_delta.cu -- the gated delta rule (the recurrence of the README's k3_kda_step,
// Part II): per sequence and value head, with the state S [D keys][D values] in float,
//   S = diag(exp(g_t)) S;  u = beta_t (v_t - S^T k_t);  S = S + k_t u^T;  o_t = scale S^T q_t.
//
// Recurrent form, for sequences of a few tokens (a decode step, drafted tokens): the
// state's tile stays in registers from its one read to its one write, and a token costs
// one pass over it.  With W = diag(exp(g)) S both products need only W:
//   r = W^T k,  u = beta (v - r),  o = W^T q + (q . k) u,  S = W + k u^T,
// so the block meets once a token (the sums of r and W^T q over the key rows), not twice.
// Bound by the state's bytes: 2 x 64 KB a head and sequence against 3 KB a token.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "k3moe_internal.cuh"
#include "k3moe_tc_warp.cuh"

namespace k3moe {
namespace {

constexpr int kD = kDeltaD;
constexpr int kRecThreads = 256, kRecWarps = kRecThreads / 32, kRecCols = 64;

// Tokens [first, first + len) and the state slot of sequence i; false (with a status bit)
// when the caller's arrays do not describe one.
__device__ __forceinline__ bool delta_seq(const DeltaArgs &a, int i, int *first, int *len, int *slot)
{
    int s0, s1;
    if (a.seq_start) {
        s0 = a.seq_start[i];
        s1 = a.seq_start[i + 1];
    } else {
        const int each = a.n_seq == 1 ? a.T : 1;
        s0 = i * each;
        s1 = s0 + each;
    }
    int32_t *status = reinterpret_cast<int32_t *>(a.ws);
    if (s0 < 0 || s1 < s0 || s1 > a.T) {
        set_status(status, K3MOE_DEV_BAD_OFFSETS);
        return false;
    }
    const int sl = a.slots ? a.slots[i] : i;
    if (sl < 0 || sl >= a.n_slots) {
        set_status(status, K3MOE_DEV_BAD_INDEX);
        return false;
    }
    *first = s0;
    *len = s1 - s0;
    *slot = sl;
    return true;
}

// Four bf16 of an 8-byte word.
__device__ __forceinline__ float4 bf4(uint2 w)
{
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ float dot4(float4 a, float4 b) { return a.x * b.x + a.y * b.y + (a.z * b.z + a.w * b.w); }

// Two floats side by side, for the instructions that work on both.
__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ float2 unpack2(uint64_t p)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// One block per (sequence, head, 64 value columns).  A warp holds 16 key rows of the state, a
// lane two value columns of them, rows in pairs for the instructions that take two floats.
// The tokens' k, q and exp(g) are made ready eight at a time, one by each warp, so that a
// token's own steps are the two products over the state, their sums over the block (one
// barrier) and the update.  What bounds it: with one token a sequence the state's bytes, with more the
// barrier and the sums.  64 columns and four blocks an SM (64 registers): 96 single-token
// sequences of 32 heads take 60.6 us, 6.6 TB/s, 37 x 4 tokens of 56 heads 56.5 us; three blocks
// 62.7 and 60.7.  A lane with four columns and eight rows: 62.2 and 69.4 (twice the sums
// to add), two tokens a barrier there 72.8.
__global__ void __launch_bounds__(kRecThreads, 4) delta_recurrent_kernel(const DeltaArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int CW = kRecCols;
    constexpr int RPT = kD / kRecWarps;                  // rows a warp holds
    constexpr int kSplit = kD / CW;
    static_assert(CW == 64, "two columns a lane");
    __shared__ __align__(16) float red[2][2][kRecWarps][CW];     // partial sums of r and W^T q, two tokens' worth
    __shared__ __align__(16) float vec[kRecWarps][3][kD];        // eight tokens' k, q and exp(g)
    __shared__ float qks[kRecWarps], bts[kRecWarps];             // their q . k and beta
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cs = blockIdx.x % kSplit, h = (blockIdx.x / kSplit) % a.H, seq = blockIdx.x / (kSplit * a.H);
    int first, len, slot;
    if (!delta_seq(a, seq, &first, &len, &slot)) return;
    const int col = cs * CW + 2 * lane, row0 = warp * RPT;
    const size_t sbase = ((size_t)slot * a.H + h) * kD * kD + (size_t)row0 * kD + col;

    uint64_t S[RPT / 2][2];                              // pairs of rows, two columns
#pragma unroll
    for (int j = 0; j < RPT; j += 2) {
        float2 x[2];
#pragma unroll
        for (int i = 0; i < 2; i++)
            x[i] = a.state_in ? __ldcs(reinterpret_cast<const float2 *>(a.state_in + sbase + (size_t)(j + i) * kD))
                              : make_float2(0.f, 0.f);
        S[j / 2][0] = pack2(x[0].x, x[1].x);
        S[j / 2][1] = pack2(x[0].y, x[1].y);
    }
    const int hq = h / (a.H / a.Hq);
    // token i of the sequence, by this warp, into its place
    auto ready = [&](int i) {
        const size_t tok = (size_t)(first + i);
        float4 q = bf4(*reinterpret_cast<const uint2 *>(a.q + tok * a.q_stride + hq * kD + 4 * lane));
        float4 k = bf4(*reinterpret_cast<const uint2 *>(a.k + tok * a.k_stride + hq * kD + 4 * lane));
        float4 g;
        if (a.gate == 1) {
            const float g1 = a.g[tok * a.H + h];
            g = make_float4(g1, g1, g1, g1);
        } else {
            g = *reinterpret_cast<const float4 *>(a.g + (tok * a.H + h) * kD + 4 * lane);
        }
        const float beta = a.beta[tok * a.H + h];
        float qk = dot4(q, k), qq = dot4(q, q), kk = dot4(k, k);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            qk += __shfl_xor_sync(0xffffffffu, qk, o);
            qq += __shfl_xor_sync(0xffffffffu, qq, o);
            kk += __shfl_xor_sync(0xffffffffu, kk, o);
        }
        const float qs = a.qk_norm ? a.scale / sqrtf(qq + a.eps) : a.scale, ks = a.qk_norm ? 1.0f / sqrtf(kk + a.eps) : 1.0f;
        reinterpret_cast<float4 *>(vec[warp][0])[lane] = make_float4(k.x * ks, k.y * ks, k.z * ks, k.w * ks);
        reinterpret_cast<float4 *>(vec[warp][1])[lane] = make_float4(q.x * qs, q.y * qs, q.z * qs, q.w * qs);
        reinterpret_cast<float4 *>(vec[warp][2])[lane] = make_float4(expf(g.x), expf(g.y), expf(g.z), expf(g.w));
        if (lane == 0) {
            qks[warp] = qk * qs * ks;
            bts[warp] = beta;
        }
    };
    auto value = [&](int i) {
        return *reinterpret_cast<const uint32_t *>(a.v + (size_t)(first + i) * a.v_stride + h * kD + col);
    };
    uint32_t vnext = 0;
    if (len > 0) vnext = value(0);
    for (int i = 0; i < len; i++) {
        const int w8 = i & (kRecWarps - 1);
        if (w8 == 0) {
            if (i > 0) __syncthreads();                  // the last eight are used
            if (i + warp < len) ready(i + warp);
            __syncthreads();
        }
        const float v0 = __uint_as_float(vnext << 16), v1 = __uint_as_float(vnext & 0xFFFF0000u);
        if (i + 1 < len) vnext = value(i + 1);           // in flight under this token's work
        const float qk = qks[w8], beta = bts[w8];
        uint64_t r0 = pack2(0.0f, 0.0f), r1 = r0, o0 = r0, o1 = r0;
#pragma unroll
        for (int j4 = 0; j4 < RPT; j4 += 4) {
            const ulonglong2 k4 = *reinterpret_cast<const ulonglong2 *>(&vec[w8][0][row0 + j4]);
            const ulonglong2 q4 = *reinterpret_cast<const ulonglong2 *>(&vec[w8][1][row0 + j4]);
            const ulonglong2 d4 = *reinterpret_cast<const ulonglong2 *>(&vec[w8][2][row0 + j4]);
            const uint64_t kj[2] = {k4.x, k4.y}, qj[2] = {q4.x, q4.y}, dj[2] = {d4.x, d4.y};
#pragma unroll
            for (int j = 0; j < 2; j++) {
                uint64_t &x = S[j4 / 2 + j][0], &y = S[j4 / 2 + j][1];
                x = mul2(x, dj[j]);
                y = mul2(y, dj[j]);
                r0 = fma2(kj[j], x, r0);
                r1 = fma2(kj[j], y, r1);
                o0 = fma2(qj[j], x, o0);
                o1 = fma2(qj[j], y, o1);
            }
        }
        // over the warps, in warp order
        float (*rd)[kRecWarps][CW] = red[i & 1];         // the other buffer is still being read
        {
            const float2 a0 = unpack2(r0), a1 = unpack2(r1), b0 = unpack2(o0), b1 = unpack2(o1);
            *reinterpret_cast<float2 *>(&rd[0][warp][2 * lane]) = make_float2(a0.x + a0.y, a1.x + a1.y);
            *reinterpret_cast<float2 *>(&rd[1][warp][2 * lane]) = make_float2(b0.x + b0.y, b1.x + b1.y);
        }
        __syncthreads();
        auto total = [&](int which) {
            uint64_t x = *reinterpret_cast<const uint64_t *>(&rd[which][0][2 * lane]);
#pragma unroll
            for (int w = 1; w < kRecWarps; w++) x = add2(x, *reinterpret_cast<const uint64_t *>(&rd[which][w][2 * lane]));
            return unpack2(x);
        };
        const float2 r = total(0);
        const float u0 = beta * (v0 - r.x), u1 = beta * (v1 - r.y);
        const uint64_t uu0 = pack2(u0, u0), uu1 = pack2(u1, u1);
#pragma unroll
        for (int j4 = 0; j4 < RPT; j4 += 4) {
            const ulonglong2 k4 = *reinterpret_cast<const ulonglong2 *>(&vec[w8][0][row0 + j4]);
            S[j4 / 2][0] = fma2(k4.x, uu0, S[j4 / 2][0]);
            S[j4 / 2][1] = fma2(k4.x, uu1, S[j4 / 2][1]);
            S[j4 / 2 + 1][0] = fma2(k4.y, uu0, S[j4 / 2 + 1][0]);
            S[j4 / 2 + 1][1] = fma2(k4.y, uu1, S[j4 / 2 + 1][1]);
        }
        if (warp == (i & (kRecWarps - 1))) {             // a warp in turn
            const float2 o = total(1);
            const __nv_bfloat162 x = __floats2bfloat162_rn(fmaf(qk, u0, o.x), fmaf(qk, u1, o.y));
            *reinterpret_cast<__nv_bfloat162 *>(a.out + ((size_t)(first + i) * a.H + h) * kD + col) = x;
        }
    }
#pragma unroll
    for (int j = 0; j < RPT; j += 2) {
        const float2 x = unpack2(S[j / 2][0]), y = unpack2(S[j / 2][1]);
        __stcs(reinterpret_cast<float2 *>(a.state_out + sbase + (size_t)j * kD), make_float2(x.x, y.x));
        __stcs(reinterpret_cast<float2 *>(a.state_out + sbase + (size_t)(j + 1) * kD), make_float2(x.y, y.y));
    }
}

// ---------------------------------------------------------------- chunks of 64 tokens
// For a chunk, with G_t the decay's logarithm summed from its start to token t (a number, or
// one a key channel; products over channels are then weighted channel by channel):
//   A_ti = beta_t exp(G_t - G_i) k_t . k_i  (i < t),   P_ti = scale exp(G_t - G_i) q_t . k_i  (i <= t)
//   T = (I + A)^-1 diag(beta),  U = T (V - (exp(G) K) S),
//   O = scale (exp(G) Q) S + P U,   S <- exp(G_C) S + (exp(G_C - G) K)^T U.
// A unit lower triangular solve replaces 64 dependent steps, and all else is products on
// the tensor cores.  Two kernels: delta_prepare_kernel computes T and P of every chunk and
// head at once (they do not need the state), delta_chunk_kernel walks a sequence and head
// through its chunks.  T and P pass through the workspace, 20 KB a chunk and head: their
// nonzero 16-column blocks only, in the layout the tensor core reads.
//
// Numbers.  bf16 operands hold 8 bits, and one such rounding would show in the float state
// (2^-9), so what is not a given bf16 tensor enters as two bf16 terms hi + mid (16 bits,
// 2^-18 of the element), a product of two such as hi hi + hi mid + mid hi.  All sums are
// float, in tensor memory; the state's carry exp(G_C) S + .. is a float sum.  A decay
// below exp(-90) is zero in float beside 1: logarithms count as at least -90.
constexpr int kC = 64;                                        // tokens a chunk
constexpr int kAllChunks = 0x7fffffff;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinGate = -90.0f;
constexpr int kTermBytes = 5120;                              // T or P, one term: 16-column blocks j of rows 16 j..63
constexpr int kTpBytes = 4 * kTermBytes;                      // T hi, T mid, P hi, P mid
constexpr int kRecFloats = 256 + 8 * kDeltaD;
constexpr int kRecBytes = kTpBytes + kRecFloats * 4;          // a chunk and head's record in the workspace
// The record's floats, a token each: kr and qr weigh the columns of K S and Q S, kd what
// enters the state.  Decay per head: kr = exp(G_t) / |k_t|, qr = scale exp(G_t) / |q_t|, kd =
// exp(G_C - G_t) / |k_t|, and one exp(G_C).  Per channel, where the operands carry the decay:
// kr = 1 / |k_t|, qr = scale / |q_t|, kd = log2 kr, and the log2 decays' sums over each 8
// tokens [8][D].  (Norms are 1 without qk_norm; past the sequence's end all are 0, log2 kr
// minus infinity.)
constexpr int kRecKr = 0, kRecKd = 64, kRecQr = 128, kRecDec = 192, kRecSum = 256;
__host__ __device__ constexpr int term_block(int j) { return 2048 * j - 256 * j * (j - 1); }

// A sequence's chunk c has the workspace record (seq_start / 64 + seq + c, head): a sequence
// of len tokens spans at most (end / 64 - start / 64) + 1 chunks, so records never overlap.
__host__ __device__ inline long long chunk_records(long long n_seq, long long T) { return T / kC + n_seq; }

// The two bf16 of a word.
__device__ __forceinline__ uint64_t pair_bf16(uint32_t w)
{
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// A pair as two packed bf16 terms: hi rounded to nearest, mid the rounded remainder.
__device__ __forceinline__ void split2(uint64_t xy, uint32_t *hi, uint32_t *mid)
{
    const float2 v = unpack2(xy);
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    const uint32_t u = *reinterpret_cast<const uint32_t *>(&h);
    const float2 r = unpack2(fma2(pair_bf16(u), pack2(-1.0f, -1.0f), xy));
    const __nv_bfloat162 m = __floats2bfloat162_rn(r.x, r.y);
    *hi = u;
    *mid = *reinterpret_cast<const uint32_t *>(&m);
}
__device__ __forceinline__ void split2(float x, float y, uint32_t *hi, uint32_t *mid) { split2(pack2(x, y), hi, mid); }
// A whole warp's wait, asleep in the barrier's own wait (up to 20 us a time) rather than
// polling beside the warps at work; bounded as mb_wait.
__device__ __forceinline__ bool mb_wait_asleep(uint64_t *b, uint32_t parity)
{
    const uint32_t a = saddr(b);
    const long long t0 = clock64();
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(a), "r"(parity), "r"(20000u)
            : "memory");
        const bool ok = __all_sync(0xffffffffu, done != 0);
        if (ok) return true;
        if (clock64() - t0 > kTcWaitCyc) return false;
    }
}
__device__ __forceinline__ float max_nan(float x, float y)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float clamp_gate(float g) { return max_nan(g, kMinGate); }   // NaN stays

// Eight values of row r, columns 8 c8.., of a lower triangular tile, as two terms in the
// tensor core's unswizzled order: 16-column block j = c8 / 2 holds rows from 16 j on, in
// pieces of 8 rows x 8 columns (128 bytes), the two column halves of 8 rows side by side.
__device__ __forceinline__ void put_terms(uint8_t *tile, int r, int c8, const float (&x)[8])
{
    const int j = c8 >> 1;
    if (r < 16 * j) return;
    uint32_t h[4], m[4];
#pragma unroll
    for (int i = 0; i < 4; i++) split2(x[2 * i], x[2 * i + 1], &h[i], &m[i]);
    uint8_t *p = tile + term_block(j) + ((r - 16 * j) >> 3) * 256 + (c8 & 1) * 128 + (r & 7) * 16;
    *reinterpret_cast<uint4 *>(p) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(p + kTermBytes) = make_uint4(m[0], m[1], m[2], m[3]);
}

// ---- the inverse
constexpr int kPpThreads = 256;
constexpr int kChLd = 68;                                     // row stride of the float scratch
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// A warp's 16 x 8 tile of sign X Y over columns k0 .. k1 of X, X and Y in shared memory with
// rows kChLd floats apart, into D: tf32 MMAs on two terms each (hi + lo, 22 bits; hi hi +
// hi lo + lo hi), which read an element once a tile where plain FMAs read it once a thread.
template <int K>
__device__ __forceinline__ void block_product(float *D, float sign, const float *X, const float *Y, int k0, int k1,
                                              int lane)
{
    const int g = lane >> 2, t = lane & 3;
    float d[3][4] = {};
#pragma unroll
    for (int k = 0; k < K; k += 8) {
        if (k < k0 || k >= k1) continue;
        const float a[4] = {X[g * kChLd + k + t], X[(g + 8) * kChLd + k + t], X[g * kChLd + k + t + 4],
                            X[(g + 8) * kChLd + k + t + 4]};
        const float b[2] = {Y[(k + t) * kChLd + g], Y[(k + t + 4) * kChLd + g]};
        uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            ah[i] = __float_as_uint(a[i]) & 0xFFFFE000u;
            al[i] = __float_as_uint(a[i] - __uint_as_float(ah[i]));
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            bh[i] = __float_as_uint(b[i]) & 0xFFFFE000u;
            bl[i] = __float_as_uint(b[i] - __uint_as_float(bh[i]));
        }
        mma_tf32(d[0], al, bh);
        mma_tf32(d[1], ah, bl);
        mma_tf32(d[2], ah, bh);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) d[2][i] = sign * ((d[0][i] + d[1][i]) + d[2][i]);
    *reinterpret_cast<float2 *>(&D[g * kChLd + 2 * t]) = make_float2(d[2][0], d[2][1]);
    *reinterpret_cast<float2 *>(&D[(g + 8) * kChLd + 2 * t]) = make_float2(d[2][2], d[2][3]);
}

// A <- (I + A)^-1 of a strictly lower triangular 64 x 64 A (rows kChLd floats apart), in
// place and by blocks: the 16 x 16 diagonal blocks by substitution, then twice
// [X11 0; -X22 A21 X11, X22].  Above the diagonal blocks is scratch.
// Up to 32 x 32: four warps (w of them), which meet at barrier 1.
__device__ __forceinline__ void four_warps() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ void invert32(float *A, int w, int lane)
{
    if (w < 2) {   // a lane a column of one of two diagonal blocks
        float *a = A + 16 * (2 * w + (lane >> 4)) * (kChLd + 1);
        float x[16];
        const int col = lane & 15;
#pragma unroll
        for (int t = 0; t < 16; t++) {
            float p[4] = {t == col ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i4 = 0; i4 < t; i4 += 4) {
                const float4 r4 = *reinterpret_cast<const float4 *>(&a[t * kChLd + i4]);
                const float r[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                for (int i = i4; i < t && i < i4 + 4; i++) p[i & 3] = fmaf(-r[i & 3], x[i], p[i & 3]);
            }
            x[t] = (p[0] + p[1]) + (p[2] + p[3]);
        }
        __syncwarp();
#pragma unroll
        for (int t = 0; t < 16; t++) a[t * kChLd + col] = x[t];       // zero above the diagonal
    }
    four_warps();
    {   // 16 -> 32: two pairs of blocks, two tiles of 16 x 8 each
        float *a = A + 32 * (w >> 1) * (kChLd + 1);
        const int n0 = (w & 1) * 8;
        block_product<16>(&a[16 + n0], 1.0f, &a[16 * kChLd], &a[n0], n0, 16, lane);                     // A21 X11
        four_warps();
        block_product<16>(&a[16 * kChLd + n0], -1.0f, &a[16 * kChLd + 16], &a[16 + n0], 0, 16, lane);   // X22 (..)
        four_warps();
#pragma unroll
        for (int r = w & 1; r < 16; r += 8)
            *reinterpret_cast<float2 *>(&a[(r + 2 * (lane >> 3)) * kChLd + 16 + (lane & 7) * 2]) = make_float2(0.f, 0.f);
    }
}
// 32 -> 64, by eight warps: eight tiles of 16 x 8; X11 and X22 are lower triangular
__device__ __forceinline__ void invert64(float *A, int warp, int lane)
{
    const int m0 = 16 * (warp >> 2), n0 = 8 * (warp & 3);
    block_product<32>(&A[m0 * kChLd + 32 + n0], 1.0f, &A[(32 + m0) * kChLd], &A[n0], n0, 32, lane);
    __syncthreads();
    block_product<32>(&A[(32 + m0) * kChLd + n0], -1.0f, &A[(32 + m0) * kChLd + 32], &A[32 + n0], 0, m0 + 16, lane);
    __syncthreads();
}

// ---------------------------------------------------------------- T and P
// A block one chunk and head at a time.  With the rows of K over those of Q as the 128 rows of a
// tensor-core tile, one product against K's rows gives A's and P's dot products.
//
// Decay per head: K and Q go in as they are and the float dot products are weighted after,
// with G as a pair of floats (a sum, and what it lost), so that differences of G hold
// however strong an earlier decay was.  The product goes against all 128 rows, whose
// diagonal is the squared norms.  Blocks stay, four an SM, and load their next chunk under this
// one's weighing and inversion.
//
// Decay per channel: the weights are inside the products.  In each 32-token half b, with m
// its G in the middle (after 16 tokens), rows are x_t exp(G_t - m), columns k_i exp(m - G_i),
// and the first half's columns go in a second time against the second half's m; a pair's
// two exponentials multiply to exp(G_t - G_i).  G counts from the half's start.  That holds
// while no |G_t - m| passes 60 (a factor of 1e26 either way; a token's mean decay of 1e-2
// over 16 tokens would reach it).  Where one does, the chunk's products are summed one by
// one, the weight's logarithm accumulated backwards from t: exact for any decay, and 30
// times slower (8192 tokens x 56 heads with one channel of each head at -5 a token: 19.9 ms
// instead of 0.66).
//
// What bounds it: its barriers and instructions (half of the issue slots, a tenth of the tensor
// cores, a quarter of the DRAM).  8192 tokens of eight sequences of 56 heads: 108 us (a block a
// chunk 129; norms from the rows instead of the diagonal 121), per channel 261, a block a chunk, three
// an SM (80 registers, operands of two terms; blocks that stay 264: their loads have nowhere to wait).
constexpr int kPpA = 128 * 128;                               // an operand's term, 64 channels: 128 rows
constexpr int kPpB = 96 * 128;                                // and 96 rows
constexpr float kPpRange = 60.0f * kLog2e;
constexpr int kPpScratch = kC * kChLd * 4;                    // per channel over the operands, once they are used
constexpr size_t pp_smem(bool channel) { return 1024 + (channel ? 2 * kPpA + 2 * kPpB : 2 * kPpA + kPpScratch); }
template <bool kChannel> constexpr int kPpBlocks = kChannel ? 3 : 4;           // of them an SM

template <bool kChannel> struct PrepShared {
    uint64_t full, done;
    uint32_t tmem;
    int far, bad;
    struct { int rec, tok0, n, head; } unit[2];               // this turn's chunk and the next; n = 0: none
    alignas(16) float gin[kC], bin[kC];                       // the next one's decays (per head) and steps
    alignas(16) float gh[kC], gl[kC], rk[kC], kb[kC], qn[kC], beta[kC];
    alignas(16) float sum[8][kChannel ? kD : 2];              // log2 decays summed over each 8 tokens
};

// The record, first token and length of chunk `unit`, false when there is none; by a whole
// warp.  All chunks at once (the call's only stretch): units are records.  A stretch: units
// are its chunks of each sequence in turn.  The sequences are searched from the first on, 32 at
// a time, which thousands of them show (65536 tokens x 8 heads as 64 sequences 343 us, as 2048, each a
// half-empty chunk and a chain of its own, 1454; per channel 626, 3025).
__device__ __forceinline__ bool find_chunk(const DeltaArgs &a, int unit, int lane, int *rec, int *tok0, int *n)
{
    auto range = [&](int s, int *s0, int *len) {
        *s0 = a.seq_start ? a.seq_start[s] : 0;
        const int s1 = a.seq_start ? a.seq_start[s + 1] : a.T;
        *len = s1 - *s0;
        return *s0 >= 0 && s1 >= *s0 && s1 <= a.T;
    };
    int s0, len, s = 0, c;
    if (a.chunk1 < kAllChunks) {
        s = unit / (a.chunk1 - a.chunk0);
        c = a.chunk0 + unit % (a.chunk1 - a.chunk0);
        if (!range(s, &s0, &len) || kC * c >= len) return false;
    } else {
        unsigned held = 0;
        for (int b = 0; b < a.n_seq && !held; b += 32) {
            const int i = b + lane;
            const bool holds = i < a.n_seq && range(i, &s0, &len) && unit >= s0 / kC + i && unit < s0 / kC + i + (len + kC - 1) / kC;
            held = __ballot_sync(0xffffffffu, holds);
            s = b + __ffs(held) - 1;
        }
        if (!held) return false;
        range(s, &s0, &len);
        c = unit - (s0 / kC + s);
    }
    *rec = s0 / kC + s + c;
    *tok0 = s0 + kC * c;
    *n = min(kC, len - kC * c);
    return true;
}

template <bool kChannel>
__global__ void __launch_bounds__(kPpThreads, kPpBlocks<kChannel>)
    delta_prepare_kernel(const DeltaArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk)
{
    // A later stretch is prepared beside the chain of the one before, launched when all of that
    // chain's blocks run: its inputs were there before they did.
    if (a.chunk0 == 0) pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(1024) uint8_t psm_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(psm_raw) + 1023) & ~(uintptr_t)1023);
    float *As = reinterpret_cast<float *>(sm + (kChannel ? 0 : 2 * kPpA));
    __shared__ PrepShared<kChannel> sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int32_t *status = reinterpret_cast<int32_t *>(a.ws);
    constexpr int kCols = 128;                                // tensor memory
    int rec0 = 0, first0 = 0, n0 = 0;                         // per channel the block's only chunk
    if (kChannel && !find_chunk(a, blockIdx.x / a.H, lane, &rec0, &first0, &n0)) {
        if (a.chunk0 > 0 && blockIdx.x == gridDim.x - 1) pdl_wait();
        return;
    }
    if (kChannel && tid < kC) sh.beta[tid] = tid < n0 ? a.beta[(size_t)(first0 + tid) * a.H + blockIdx.x % a.H] : 0.0f;
    if (tid == 0) {
        mb_init(&sh.full, 1);
        mb_init(&sh.done, 1);
        sh.far = 0;
        sh.bad = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sh.tmem)), "r"(kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    auto wait = [&](uint64_t &b, uint32_t parity) {
        if (mb_wait_asleep(&b, parity)) return true;
        set_status(status, K3MOE_DEV_TIMEOUT);
        sh.bad = 1;
        return false;
    };
    // Per head, by one warp, under the turn before: the block's turn-th chunk, its decays and steps
    // and, into the operands' place, K and Q.
    int at = blockIdx.x;
    float bnext[2] = {}, gnext[2] = {};
    auto next = [&](int turn) {
        auto &unit = sh.unit[turn & 1];
        int rec = 0, tok0 = 0, n = 0, head = 0;
        for (; at < a.units; at += gridDim.x) {
            head = at % a.H;
            if (find_chunk(a, at / a.H, lane, &rec, &tok0, &n)) break;
        }
        const bool any = at < a.units;
        at += gridDim.x;
        if (lane == 0) {
            unit.rec = rec;
            unit.tok0 = tok0;
            unit.n = any ? n : 0;
            unit.head = head;
        }
        if (!any) return;
        if (lane == 0) {
            const int hq = head / (a.H / a.Hq);
            mb_expect_tx(&sh.full, 2 * kPpA);
            for (int b = 0; b < 2; b++) {
                tma2d(sm + b * kPpA, &mk, hq * kD + 64 * b, tok0, &sh.full);
                tma2d(sm + b * kPpA + kC * 128, &mq, hq * kD + 64 * b, tok0, &sh.full);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int t = lane + 32 * i;
            const size_t tok = (size_t)(tok0 + min(t, n - 1)) * a.H + head;
            bnext[i] = t < n ? a.beta[tok] : 0.0f;
            gnext[i] = t < n ? a.g[tok] : 0.0f;
        }
    };
    auto keep = [&]() {                                       // later: the loads are then there
#pragma unroll
        for (int i = 0; i < 2; i++) {
            sh.bin[lane + 32 * i] = bnext[i];
            sh.gin[lane + 32 * i] = clamp_gate(gnext[i]);
        }
    };
    constexpr int kWarpNext = 6;                              // idle while the others weigh
    if (!kChannel) {
        if (warp == kWarpNext) {
            next(0);
            keep();
        }
        __syncthreads();
    }
    for (int turn = 0; turn < (kChannel ? 1 : 0x7fffffff); turn++) {
        const int n = kChannel ? n0 : sh.unit[turn & 1].n;
        if (n == 0) break;
        const int rec = kChannel ? rec0 : sh.unit[turn & 1].rec, tok0 = kChannel ? first0 : sh.unit[turn & 1].tok0;
        const int h = kChannel ? blockIdx.x % a.H : sh.unit[turn & 1].head, hq = h / (a.H / a.Hq);
        uint8_t *out = a.ws + kCtrOffset + kCtrBytes + ((size_t)rec * a.H + h) * kRecBytes;
        float *outf = reinterpret_cast<float *>(out + kTpBytes);
        bool far = false;                                         // per channel: the weights reach too far

        if (!kChannel) {
            if (warp == 4 && wait(sh.full, turn & 1)) {
                const uint32_t d = desc_lo(saddr(sm));
#pragma unroll
                for (int s = 0; s < 8; s++) {
                    const uint32_t at = d + (((s >> 2) * kPpA + (s & 3) * 32) >> 4);
                    umma_warp(tmem, at, at, idesc(1, 2 * kC), s > 0);
                }
                umma_commit_warp(&sh.done);
            }
            const int row = tid, t = row & (kC - 1);              // threads 0-63: K's rows, 64-127: Q's
            if (warp < 4) {
                // inclusive sums over the 64 tokens, two a lane, as sum + lost
                float s[2], e[2] = {0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 2; i++)
                    s[i] = sh.gin[lane + 32 * i];
                auto add = [](float &x, float &ex, float y, float ey) {      // two-sum, then the lost parts
                    const float z = x + y, v = z - x;
                    ex = ((x - (z - v)) + (y - v)) + (ex + ey);
                    x = z;
                };
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float p = __shfl_up_sync(0xffffffffu, s[i], o), ep = __shfl_up_sync(0xffffffffu, e[i], o);
                        if (lane >= o) add(s[i], e[i], p, ep);
                    }
                add(s[1], e[1], __shfl_sync(0xffffffffu, s[0], 31), __shfl_sync(0xffffffffu, e[0], 31));
                const float gc = __shfl_sync(0xffffffffu, s[1], 31), ec = __shfl_sync(0xffffffffu, e[1], 31);
                const float G = (warp & 1) ? s[1] : s[0], E = (warp & 1) ? e[1] : e[0];
                float norm = 1.0f;
                if (a.qk_norm && wait(sh.done, turn & 1)) {   // the diagonal: lane l has its own in column l of 32
                    tc_fence_after();
                    float x[32];
                    const uint32_t at32 = tmem + ((uint32_t)(32 * warp) << 16) + 32 * warp;
                    tmem_ld16_nowait(at32, *reinterpret_cast<uint32_t(*)[16]>(&x[0]));
                    tmem_ld16_nowait(at32 + 16, *reinterpret_cast<uint32_t(*)[16]>(&x[16]));
                    tmem_wait_ld();
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                        for (int i = 0; i < o; i++) x[i] = lane & o ? x[i + o] : x[i];
                    norm = 1.0f / sqrtf(x[0] + a.eps);
                }
                const bool in = t < n;
                const float eG = expf(G + E);
                if (row < kC) {
                    const float b = sh.bin[t];
                    sh.gh[t] = G;
                    sh.gl[t] = E;
                    sh.rk[t] = in ? norm : 0.0f;
                    sh.beta[t] = b;
                    sh.kb[t] = in ? b * norm : 0.0f;
                    outf[kRecKr + t] = in ? norm * eG : 0.0f;
                    outf[kRecKd + t] = in ? norm * expf((gc - G) + (ec - E)) : 0.0f;
                    if (t == 0) outf[kRecDec] = expf(gc + ec);
                } else {
                    sh.qn[t] = in ? a.scale * norm : 0.0f;
                    outf[kRecQr + t] = in ? a.scale * norm * eG : 0.0f;
                }
            }
            __syncthreads();
            if (!sh.bad) wait(sh.done, turn & 1);
        } else {
            // a warp 8 tokens, a lane two of the 64 channels at hand
            const int t0 = 8 * warp;
            float nk[8] = {}, nq[8] = {}, reach = 0.0f;
            for (int half = 0; half < 2; half++) {
                const int ch = 64 * half + 2 * lane;
                uint32_t k[8], q[8];
                float2 g[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const size_t tok = (size_t)tok0 + min(t0 + i, n - 1);
                    k[i] = *reinterpret_cast<const uint32_t *>(a.k + tok * a.k_stride + hq * kD + ch);
                    q[i] = *reinterpret_cast<const uint32_t *>(a.q + tok * a.q_stride + hq * kD + ch);
                    g[i] = *reinterpret_cast<const float2 *>(a.g + (tok * a.H + h) * kD + ch);
                }
                float2 L = make_float2(0.0f, 0.0f);               // sums over this warp's tokens so far, in log2
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const bool in = t0 + i < n;
                    L.x += in ? clamp_gate(g[i].x) * kLog2e : 0.0f;
                    L.y += in ? clamp_gate(g[i].y) * kLog2e : 0.0f;
                    g[i] = L;
                }
                *reinterpret_cast<float2 *>(&sh.sum[warp][ch]) = L;
                *reinterpret_cast<float2 *>(&outf[kRecSum + warp * kD + ch]) = L;
                if (half == 1) wait(sh.done, 0);                  // the first half's operands are used
                __syncthreads();
                if (sh.bad) break;
                float2 s[8];
#pragma unroll
                for (int w = 0; w < 8; w++) s[w] = *reinterpret_cast<const float2 *>(&sh.sum[w][ch]);
                // G at this warp's start less the middle of its 32 tokens; the second half's middle
                // less the first half's end (both counted from their own half's start)
                const int b = (warp >> 2) * 4;
                float2 base = make_float2(0.f, 0.f);
                float2 m1 = make_float2(s[4].x + s[5].x, s[4].y + s[5].y);
                switch (warp & 3) {
                case 0: base = make_float2(-(s[b].x + s[b + 1].x), -(s[b].y + s[b + 1].y)); break;
                case 1: base = make_float2(-s[b + 1].x, -s[b + 1].y); break;
                case 2: break;
                default: base = make_float2(s[b + 2].x, s[b + 2].y); break;
                }
                // (first half only) the second's middle less G at this warp's start
                float2 tail = m1;
#pragma unroll
                for (int w = 3; w >= 0; w--)
                    if (w >= warp) { tail.x += s[w].x; tail.y += s[w].y; }
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int t = t0 + i;
                    const uint64_t kk = pair_bf16(k[i]), qq = pair_bf16(q[i]);
                    const float2 kf = unpack2(kk), qf = unpack2(qq);
                    nk[i] = fmaf(kf.x, kf.x, fmaf(kf.y, kf.y, nk[i]));
                    nq[i] = fmaf(qf.x, qf.x, fmaf(qf.y, qf.y, nq[i]));
                    const float dx = base.x + g[i].x, dy = base.y + g[i].y;       // G_t - m
                    reach = max_nan(reach, max_nan(fabsf(dx), fabsf(dy)));
                    const uint64_t e = pack2(exp2_fast(dx), exp2_fast(dy));
                    const uint32_t at = t * 128 + (((lane >> 2) ^ (t & 7)) << 4) + (lane & 3) * 4;
                    uint32_t hi, mid;
                    split2(mul2(kk, e), &hi, &mid);
                    *reinterpret_cast<uint32_t *>(sm + at) = hi;
                    *reinterpret_cast<uint32_t *>(sm + kPpA + at) = mid;
                    split2(mul2(qq, e), &hi, &mid);
                    *reinterpret_cast<uint32_t *>(sm + kC * 128 + at) = hi;
                    *reinterpret_cast<uint32_t *>(sm + kPpA + kC * 128 + at) = mid;
                    uint8_t *B = sm + 2 * kPpA;
                    split2(mul2(kk, pack2(exp2_fast(-dx), exp2_fast(-dy))), &hi, &mid);
                    *reinterpret_cast<uint32_t *>(B + at) = hi;
                    *reinterpret_cast<uint32_t *>(B + kPpB + at) = mid;
                    if (warp < 4) {
                        split2(mul2(kk, pack2(exp2_fast(tail.x - g[i].x), exp2_fast(tail.y - g[i].y))), &hi, &mid);
                        *reinterpret_cast<uint32_t *>(B + kC * 128 + at) = hi;
                        *reinterpret_cast<uint32_t *>(B + kPpB + kC * 128 + at) = mid;
                    }
                }
                fence_async_smem();
                __syncthreads();
                if (warp == 0) {
                    const uint32_t A = desc_lo(saddr(sm)), B = desc_lo(saddr(sm + 2 * kPpA));
#pragma unroll
                    for (int term = 0; term < 3; term++)
#pragma unroll
                        for (int s4 = 0; s4 < 4; s4++)
                            umma_warp(tmem, A + (((term == 2 ? kPpA : 0) + s4 * 32) >> 4), B + (((term == 1 ? kPpB : 0) + s4 * 32) >> 4),
                                      idesc(1, 96), half > 0 || term > 0 || s4 > 0);
                    umma_commit_warp(&sh.done);
                }
            }
            if (!(reach <= kPpRange)) sh.far = 1;
            // the norms, a warp's eight rows of each: every exchange halves the rows a lane still sums
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const bool up = lane & 16;
                nk[i] = (up ? nq[i] : nk[i]) + __shfl_xor_sync(0xffffffffu, up ? nk[i] : nq[i], 16);
            }
#pragma unroll
            for (int o = 8; o >= 2; o >>= 1) {
                const bool up = lane & o;
#pragma unroll
                for (int i = 0; i < o / 2; i++)
                    nk[i] = (up ? nk[i + o / 2] : nk[i]) + __shfl_xor_sync(0xffffffffu, up ? nk[i] : nk[i + o / 2], o);
            }
            const float n2 = nk[0] + __shfl_xor_sync(0xffffffffu, nk[0], 1);      // lanes below 16 K's, the others Q's
            if (!(lane & 1)) {
                const int t = t0 + ((lane >> 1) & 7);
                const bool in = t < n;
                const float norm = a.qk_norm ? 1.0f / sqrtf(n2 + a.eps) : 1.0f;
                if (lane < 16) {
                    const float rk = in ? norm : 0.0f;
                    sh.rk[t] = rk;
                    sh.kb[t] = sh.beta[t] * rk;
                    outf[kRecKr + t] = rk;
                    outf[kRecKd + t] = log2f(rk);
                } else {
                    const float qn = in ? a.scale * norm : 0.0f;
                    sh.qn[t] = qn;
                    outf[kRecQr + t] = qn;
                }
            }
            if (!sh.bad) wait(sh.done, 1);
            __syncthreads();
            far = sh.far != 0;
        }
        __syncthreads();

        if (!sh.bad) {
            // the operands are used (per channel the scratch goes over them), and what the block had of
            // this chunk's steps and decays
            if (!kChannel && warp == kWarpNext) next(turn + 1);
            if (tid == 0) sh.far = 0;
            // lanes 0-63 of tensor memory hold A's rows, 64-127 P's; a warp takes 32 rows of one of
            // the two, half of their columns (the upper right quarter of either is zero: not done).
            // A's four warps go on to invert its 32 x 32 blocks while the others write P.
            tc_fence_after();
            const int row = 32 * (warp & 3) + lane, t = row & (kC - 1), i00 = 32 * (warp >> 2);
            const bool is_a = row < kC;
            const float rowf = is_a ? sh.kb[t] : sh.qn[t];
            const int last = t < n ? (is_a ? t - 1 : t) : -1;     // the row's last token
            const bool zero = i00 == 32 && (warp & 1) == 0;
            float v[32];
            if (zero) {
            } else if (kChannel && far) {
                // one product at a time, the weight's logarithm summed backwards from t
                const uint16_t *x = (is_a ? a.k + (size_t)(tok0 + min(t, n - 1)) * a.k_stride
                                          : a.q + (size_t)(tok0 + min(t, n - 1)) * a.q_stride) + hq * kD;
#pragma unroll
                for (int j = 0; j < 32; j++) v[j] = 0.0f;
                for (int c = 0; c < kD; c++) {
                    const float xc = bf16_bits_to_f32(x[c]);
                    float D = 0.0f;
                    for (int i = t; i >= i00 + 32; i--)           // tokens between the columns and t
                        if (i < n) D += clamp_gate(a.g[((size_t)(tok0 + i) * a.H + h) * kD + c]);
#pragma unroll
                    for (int j = 31; j >= 0; j--) {
                        const int i = i00 + j;
                        if (i <= t && t < n) {
                            v[j] = fmaf(xc * bf16_bits_to_f32(a.k[(size_t)(tok0 + i) * a.k_stride + hq * kD + c]),
                                        exp2_fast(D * kLog2e), v[j]);
                            D += clamp_gate(a.g[((size_t)(tok0 + i) * a.H + h) * kD + c]);
                        }
                    }
                }
            } else {
                const uint32_t at = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (kChannel && t >= 32 && i00 == 0 ? 64 : i00);
                tmem_ld16_nowait(at, *reinterpret_cast<uint32_t(*)[16]>(&v[0]));
                tmem_ld16_nowait(at + 16, *reinterpret_cast<uint32_t(*)[16]>(&v[16]));
                tmem_wait_ld();
            }
            if (!zero) {
                const float gh = kChannel ? 0.0f : sh.gh[t], gl = kChannel ? 0.0f : sh.gl[t];
                const uint64_t minus = pack2(-1.0f, -1.0f);
#pragma unroll
                for (int j4 = 0; j4 < 32; j4 += 4) {
                    const float4 r4 = *reinterpret_cast<const float4 *>(&sh.rk[i00 + j4]);
                    const float r[4] = {r4.x, r4.y, r4.z, r4.w};
                    float gi[4] = {}, li[4] = {};
                    if (!kChannel) {
                        const float4 h4 = *reinterpret_cast<const float4 *>(&sh.gh[i00 + j4]);
                        const float4 l4 = *reinterpret_cast<const float4 *>(&sh.gl[i00 + j4]);
                        gi[0] = h4.x; gi[1] = h4.y; gi[2] = h4.z; gi[3] = h4.w;
                        li[0] = l4.x; li[1] = l4.y; li[2] = l4.z; li[3] = l4.w;
                    }
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const int at = j4 + j;
                        uint64_t x = mul2(pack2(v[at], v[at + 1]), mul2(pack2(rowf, rowf), pack2(r[j], r[j + 1])));
                        if (!kChannel) {
                            const uint64_t e = add2(fma2(pack2(gi[j], gi[j + 1]), minus, pack2(gh, gh)),
                                                    fma2(pack2(li[j], li[j + 1]), minus, pack2(gl, gl)));
                            const float2 w = unpack2(mul2(e, pack2(kLog2e, kLog2e)));
                            x = mul2(x, pack2(exp2_fast(w.x), exp2_fast(w.y)));
                        }
                        const float2 y = unpack2(x);
                        v[at] = i00 + at <= last ? y.x : 0.0f;
                        v[at + 1] = i00 + at + 1 <= last ? y.y : 0.0f;
                    }
                }
            }
            if (is_a) {
                if (!zero)
#pragma unroll
                    for (int j = 0; j < 8; j++)                   // over the operands: they are used
                        *reinterpret_cast<float4 *>(&As[t * kChLd + i00 + 4 * j]) =
                        make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                four_warps();
                invert32(As, (warp & 1) + 2 * (warp >> 2), lane);
            } else if (!zero) {
                const float(*v8)[8] = reinterpret_cast<const float(*)[8]>(v);
#pragma unroll
                for (int j = 0; j < 4; j++) put_terms(out + 2 * kTermBytes, t, i00 / 8 + j, v8[j]);
            }
            __syncthreads();
            invert64(As, warp, lane);
            if (!kChannel && warp == kWarpNext) keep();
            // T = (I + A)^-1 diag(beta): a warp 16 columns of half the rows
            const int r = 32 * (warp >> 2) + lane, c0 = 16 * (warp & 3);
            if (c0 < 32 * (warp >> 2) + 32)
#pragma unroll
                for (int j8 = 0; j8 < 2; j8++) {
                    float x[8], b[8];
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        *reinterpret_cast<float4 *>(&x[j]) = *reinterpret_cast<const float4 *>(&As[r * kChLd + c0 + 8 * j8 + j]);
                        *reinterpret_cast<float4 *>(&b[j]) = *reinterpret_cast<const float4 *>(&sh.beta[c0 + 8 * j8 + j]);
                    }
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const float y = x[j] * b[j];
                        x[j] = c0 + 8 * j8 + j <= r ? y : 0.0f;
                    }
                    put_terms(out, r, c0 / 8 + j8, x);
                }
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (sh.bad) {                                             // given up: not before the copies on their way
            if (!kChannel && sh.unit[(turn + 1) & 1].n > 0) wait(sh.full, (turn + 1) & 1);
            break;
        }
    }
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
    // the last block of such a launch ends after that chain: what follows finds both complete
    if (a.chunk0 > 0 && blockIdx.x == gridDim.x - 1) pdl_wait();
}

// ---------------------------------------------------------------- the chain
// One block per sequence and head walks its chunks; everything is transposed so that a
// thread owns one value column v (a lane of tensor memory) of the state S^T [v][k], and the A
// operands (S, R = V - exp(G) K S, U) go from tensor memory to registers and back, never
// through shared memory; the B operands (K and Q, T, P) are shared tiles.
//   decay per head: K and Q as they are (exact in bf16); exp(G) weighs the results' columns,
//     and U's a second time before K^T U;
//   per channel: eight warps more write exp(G) K, exp(G) Q and exp(G_C - G) K / |k| as two
//     terms each, a chunk ahead.
// The chain's eight warps keep 64 floats of the state a thread, in tensor memory: in
// registers they made the other roles spill, and the spills' way through the L2 made a chunk
// three times as long.  Sixteen warps with 32 each took as long a phase: they share four schedulers.
// What bounds it: the steps follow from one another, 3.3 us a chunk and 4.7 per channel with the
// tensor cores busy a quarter of it; the loops over the terms stay rolled, as straight code misses
// the instruction cache every chunk (eight sequences of 1024 tokens x 56 heads: 186 -> 178 us, per
// channel 287 -> 263).
constexpr int kChChain = 8, kChOut = 4, kChMake = 8;
constexpr int kChPartK = kD / (kChChain / 4), kChPartT = kC / (kChChain / 4);     // channels and tokens of a chain warp
constexpr int kChStagesHead = 3, kChStagesChannel = 2;
constexpr int kChBox = kC * 128;                              // 64 tokens x 64 channels: 8 KB
constexpr int kChKq = 4 * kChBox;                             // decay per head: K and Q, [box][K, Q]
constexpr int kChV = 2 * kChBox;
constexpr int kChTp = 21 * 1024;                              // T and P and the scales
constexpr int kChTpCopy = kTpBytes + 1024;                    // with the record's first floats
constexpr int kChStageHead = kChKq + kChV + kChTp, kChStageChannel = kChV + kChTp;
constexpr int kChTerm = 2 * kChBox;                           // per channel: one term of 64 x 128
constexpr int kChMade = 4 * kChTerm + 4 * kChTerm;            // [hi, mid][box][K, Q]; the late K [chunk parity][hi, mid][box]
static_assert(kTpBytes + (kRecDec + 1) * 4 <= kChTp && kTpBytes + 1024 <= kChTp, "a stage holds the record's head");
template <bool kChannel> struct ChunkShape {
    static constexpr int warps = kChChain + kChOut + (kChannel ? kChMake : 0) + 2;    // and MMA issue, loads
    static constexpr int threads = kChannel ? (warps + 3) / 4 * 128 : warps * 32;     // per channel whole warpgroups: registers move
    static constexpr int stages = kChannel ? kChStagesChannel : kChStagesHead;
    static constexpr int stage = kChannel ? kChStageChannel : kChStageHead;
    static constexpr int smem = 1024 + (kChannel ? kChMade : 0) + stages * stage;
};
constexpr int kChWarpOut = kChChain, kChWarpMake = kChWarpOut + kChOut;
// Registers a thread per channel: 80 at launch (768 threads), shares moved between the
// warpgroups so that no role spills in a chunk's way.
constexpr int kChRegs = 80, kChRegsChain = 88, kChRegsOut = 88, kChRegsMake = 80, kChRegsLast = 56;
static_assert(kChRegsChain >= kChRegs && kChRegsOut >= kChRegs && kChRegsMake <= kChRegs && kChRegsLast <= kChRegs,
              "inc only from below, dec only from above");
static_assert(2 * kChRegsChain + kChRegsOut + 2 * kChRegsMake + kChRegsLast <= 6 * kChRegs, "shares within the launch's");
static_assert(kChChain == 8 && kChOut == 4 && kChMake == 8, "the shares are of whole warpgroups");
// tensor memory columns
constexpr uint32_t kTmS = 0;      // S^T as an operand, [quarter of k][hi, mid][16]; the new S's sums over it
constexpr uint32_t kTmR = 128;    // K S, then T R; per head then U as an operand
constexpr uint32_t kTmOq = 192;   // Q S
constexpr uint32_t kTmOp = 256;   // P U
constexpr uint32_t kTmRU = 320;   // R, then U (per head: weighted for the state), as an operand [half of t][hi, mid][16]
constexpr uint32_t kTmF = 384;    // the state, float [128]

// Up to this many sequences are taken by length (every block ranks them): 8 sequences of 50 to 2000
// tokens x 56 heads take 211 us by length and 238 as given, 40 x 32 heads 503 and 504, 250 1060 and 932.
constexpr int kRankSeqs = 32;
struct ChunkShared {
    uint64_t in_full[3], in_free[3];
    uint64_t s_ready, d1_full, q_done, r_ready, d2_full, u_ready, d4_full, o_full, o_free, made, drain;
    uint32_t tmem;
    volatile int bail;
    alignas(16) float dec[2][kD];                             // per channel: exp(G_C), by chunk parity
    int seq, len[kRankSeqs];
    int first, tokens, slot, head, record;                    // the block's stretch, for the roles
};

// Unswizzled K-major descriptors of T and P blocks: 8-row groups 256 bytes apart, their two
// 8-column halves (the leading offset) 128.
constexpr uint32_t kDescTp = (256u >> 4) | (1u << 14);

template <bool kChannel>
__global__ void __launch_bounds__(ChunkShape<kChannel>::threads, 1)
    delta_chunk_kernel(const DeltaArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv)
{
    pdl_wait();
    pdl_trigger();
    using Shape = ChunkShape<kChannel>;
    constexpr int kWarpMma = Shape::warps - 2, kWarpLoad = kWarpMma + 1, kStages = Shape::stages;
    extern __shared__ __align__(1024) uint8_t csm_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(csm_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *made = sm;                                       // per channel
    uint8_t *ring = sm + (kChannel ? kChMade : 0);
    constexpr int kOffV = kChannel ? 0 : kChKq, kOffTp = kOffV + kChV;
    __shared__ ChunkShared sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % a.H;
    int seq = blockIdx.x / a.H;
    if (seq >= a.n_seq) return;                               // the last pair's second block
    if (a.n_seq > 1 && a.n_seq <= kRankSeqs && a.seq_start) {
        // the long sequences first: this block's is the one as many others come before
        for (int i = threadIdx.x; i < a.n_seq; i += Shape::threads) sh.len[i] = a.seq_start[i + 1] - a.seq_start[i];
        __syncthreads();
        for (int i = threadIdx.x; i < a.n_seq; i += Shape::threads) {
            int before = 0;
            for (int j = 0; j < a.n_seq; j++) before += sh.len[j] > sh.len[i] || (sh.len[j] == sh.len[i] && j < i);
            if (before == seq) sh.seq = i;
        }
        __syncthreads();
        seq = sh.seq;
    }
    int first, len, slot;
    if (!delta_seq(a, seq, &first, &len, &slot)) return;
    const size_t sbase = ((size_t)slot * a.H + h) * kD * kD;
    if (len == 0) {
        if (a.chunk0 > 0) return;
        for (int e = threadIdx.x; e < kD * kD / 4; e += Shape::threads)
            reinterpret_cast<float4 *>(a.state_out + sbase)[e] =
                a.state_in ? reinterpret_cast<const float4 *>(a.state_in + sbase)[e] : make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    // this launch's stretch stands for the sequence from here on; the roles read it from shared
    // memory, as what they held in common would be kept in the registers of all
    if (a.chunk0 >= (len + kC - 1) / kC) return;
    if (threadIdx.x == 0) {
        sh.first = first + kC * a.chunk0;
        sh.tokens = a.chunk1 < kAllChunks ? min(len - kC * a.chunk0, kC * (a.chunk1 - a.chunk0)) : len - kC * a.chunk0;
        sh.slot = slot;
        sh.head = h;
        sh.record = first / kC + seq + a.chunk0;
    }
    auto own = [](const int &x) { return *const_cast<const volatile int *>(&x); };
    auto record = [&](int c) {                                // chunk c's
        return a.ws + kCtrOffset + kCtrBytes + ((size_t)(own(sh.record) + c) * a.H + own(sh.head)) * kRecBytes;
    };
    auto stage = [&](int c) { return ring + (size_t)(c % kStages) * Shape::stage; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) { mb_init(&sh.in_full[s], 1); mb_init(&sh.in_free[s], kChOut); }
        mb_init(&sh.s_ready, kChChain);
        mb_init(&sh.d1_full, 1);
        mb_init(&sh.q_done, 1);
        mb_init(&sh.r_ready, kChChain);
        mb_init(&sh.d2_full, 1);
        mb_init(&sh.u_ready, kChChain);
        mb_init(&sh.d4_full, 1);
        mb_init(&sh.o_full, 1);
        mb_init(&sh.o_free, kChOut);
        mb_init(&sh.made, kChMake);
        mb_init(&sh.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.bail = 0;
    }
    if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sh.tmem)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;                              // all 512 columns: the allocation starts at the first
    // A wait of a whole warp; false (with the status bit) when it gave up or another did.
    auto wait = [&](uint64_t &b, int phase) {
        const bool ok = mb_wait_asleep(&b, (uint32_t)phase & 1u);
        if (!ok) {
            set_status(reinterpret_cast<int32_t *>(a.ws), K3MOE_DEV_TIMEOUT);
            sh.bail = 1;
        }
        return (bool)__all_sync(0xffffffffu, ok && !sh.bail);
    };
    // A warp's accesses to tensor memory are done: tell the barrier's waiter.
    auto arrive = [&](uint64_t &b) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mb_arrive(&b);
    };
    if (kChannel) {
        if (warp < kChChain)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChRegsChain));
        else if (warp < kChWarpMake)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChRegsOut));
        else if (warp < kWarpMma)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kChRegsMake));
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kChRegsLast));
    }
    if (warp < kChChain) {
        // ---------------- the chain: value column v, half of the channels or tokens
        const int q = warp & 3, part = warp >> 2, v = 32 * q + lane, t0 = kChPartT * part;
        const int len = own(sh.tokens), nc = (len + kC - 1) / kC;
        auto state_at = [&]() { return ((size_t)own(sh.slot) * a.H + own(sh.head)) * kD * kD + (size_t)(kChPartK * part) * kD + v; };
        const uint32_t la = tmem + ((uint32_t)(32 * q) << 16);
        const uint32_t la_s = la + kTmS + kChPartK * part;
        const uint32_t la_f = la + kTmF + kChPartK * part;
        // 32 channels of the state from b on as two terms
        auto put_terms32 = [&](int b, const float *x) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                uint32_t hi[4], mid[4];
#pragma unroll
                for (int j = 0; j < 4; j++) split2(x[8 * i + 2 * j], x[8 * i + 2 * j + 1], &hi[j], &mid[j]);
                tmem_st4(la_s + b + 4 * i, hi);
                tmem_st4(la_s + b + 16 + 4 * i, mid);
            }
        };
        {
            const float *in = a.chunk0 > 0 ? a.state_out : a.state_in;
            const float *from = in ? in + state_at() : nullptr;
#pragma unroll
            for (int b = 0; b < kChPartK; b += 32) {
                float x[32];
#pragma unroll
                for (int j = 0; j < 32; j++) x[j] = from ? from[(size_t)(b + j) * kD] : 0.0f;
                tmem_st16(la_f + b, &x[0]);
                tmem_st16(la_f + b + 16, &x[16]);
                put_terms32(b, x);
            }
            tmem_wait_st();
            arrive(sh.s_ready);
        }
        for (int c = 0; c < nc; c++) {
            const int n = min(kC, len - kC * c);
            const float *sc = reinterpret_cast<const float *>(stage(c) + kOffTp + kTpBytes) + t0;
            // V[t][v] in its swizzled tile
            const uint8_t *vt = stage(c) + kOffV + (q >> 1) * kChBox + t0 * 128 + (v & 7) * 2;
            const uint32_t v8 = (uint32_t)(v >> 3) & 7u;
            if (!wait(sh.in_full[c % kStages], c / kStages)) break;
            uint32_t vv[kChPartT / 2];                            // two tokens a word
#pragma unroll
            for (int j = 0; j < kChPartT / 2; j++) {
                asm volatile("" : "+l"(vt));
                const uint32_t x = *reinterpret_cast<const uint16_t *>(vt + 2 * j * 128 + ((v8 ^ ((2 * j) & 7u)) << 4));
                const uint32_t y = *reinterpret_cast<const uint16_t *>(vt + 2 * j * 128 + 128 + ((v8 ^ ((2 * j + 1) & 7u)) << 4));
                vv[j] = x | (y << 16);
            }
            if (!wait(sh.d1_full, c)) break;
            tc_fence_after();
            {
                uint32_t d[kChPartT];
                tmem_ld16_nowait(la + kTmR + t0, *reinterpret_cast<uint32_t(*)[16]>(&d[0]));
                tmem_ld16_nowait(la + kTmR + t0 + 16, *reinterpret_cast<uint32_t(*)[16]>(&d[16]));
                tmem_wait_ld();
#pragma unroll
                for (int b = 0; b < kChPartT / 8; b++) {
                    uint32_t hi[4], mid[4];
#pragma unroll
                    for (int j2 = 0; j2 < 4; j2++) {
                        const int j = 8 * b + 2 * j2;
                        const float2 kr = *reinterpret_cast<const float2 *>(&sc[kRecKr + j]);
                        const float2 x = unpack2(fma2(pack2(-kr.x, -kr.y), pack2(__uint_as_float(d[j]), __uint_as_float(d[j + 1])),
                                                     pair_bf16(vv[j >> 1])));
                        split2(t0 + j < n ? x.x : 0.0f, t0 + j + 1 < n ? x.y : 0.0f, &hi[j2], &mid[j2]);
                    }
                    tmem_st4(la + kTmRU + t0 + 4 * b, hi);
                    tmem_st4(la + kTmRU + t0 + 16 + 4 * b, mid);
                }
            }
            tmem_wait_st();
            arrive(sh.r_ready);
            if (!kChannel && n < kC) {
                // K's rows past the sequence's end are another's, or nobody's: U is zero there, but zero times a NaN
                // or an infinity is not.  K S has read them, K^T U has yet to
#pragma unroll 1
                for (int i = threadIdx.x; i < 2 * 8 * (kC - n); i += kChChain * 32)
                    *reinterpret_cast<uint4 *>(stage(c) + (i & 1) * 2 * kChBox + n * 128 + (i >> 1) * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            if (!wait(sh.d2_full, c)) break;
            tc_fence_after();
            {
                uint32_t d[kChPartT];                         // all read: per head U's terms go over them
                tmem_ld16_nowait(la + kTmR + t0, *reinterpret_cast<uint32_t(*)[16]>(&d[0]));
                tmem_ld16_nowait(la + kTmR + t0 + 16, *reinterpret_cast<uint32_t(*)[16]>(&d[16]));
                tmem_wait_ld();
#pragma unroll
                for (int b = 0; b < kChPartT / 8; b++) {
                    uint32_t hi[4], mid[4];
#pragma unroll
                    for (int j2 = 0; j2 < 4; j2++)
                        split2(__uint_as_float(d[8 * b + 2 * j2]), __uint_as_float(d[8 * b + 2 * j2 + 1]), &hi[j2], &mid[j2]);
                    tmem_st4(la + (kChannel ? kTmRU : kTmR) + t0 + 4 * b, hi);
                    tmem_st4(la + (kChannel ? kTmRU : kTmR) + t0 + 16 + 4 * b, mid);
                    if (!kChannel) {
#pragma unroll
                        for (int j2 = 0; j2 < 4; j2++) {
                            const int i = 8 * b + 2 * j2;
                            const float2 kd = *reinterpret_cast<const float2 *>(&sc[kRecKd + i]);
                            split2(mul2(pack2(__uint_as_float(d[i]), __uint_as_float(d[i + 1])), pack2(kd.x, kd.y)), &hi[j2], &mid[j2]);
                        }
                        tmem_st4(la + kTmRU + t0 + 4 * b, hi);
                        tmem_st4(la + kTmRU + t0 + 16 + 4 * b, mid);
                    }
                }
            }
            tmem_wait_st();
            const float dec = kChannel ? 0.0f : sc[kRecDec - t0];     // the stage's last read: it is given back after this arrival
            arrive(sh.u_ready);
            if (!wait(sh.d4_full, c)) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < kChPartK; b += 32) {          // the operand's terms go over the sums they come from
                uint32_t d[32];
                tmem_ld16_nowait(la_s + b, *reinterpret_cast<uint32_t(*)[16]>(&d[0]));
                tmem_ld16_nowait(la_s + b + 16, *reinterpret_cast<uint32_t(*)[16]>(&d[16]));
                float x[32];
#pragma unroll
                for (int b16 = 0; b16 < 32; b16 += 16) {
                    uint32_t f[16];
                    tmem_ld16_nowait(la_f + b + b16, f);
                    tmem_wait_ld();
#pragma unroll
                    for (int j4 = 0; j4 < 4; j4++) {
                        float4 e4 = make_float4(dec, dec, dec, dec);
                        if (kChannel) e4 = *reinterpret_cast<const float4 *>(&sh.dec[c & 1][kChPartK * part + b + b16 + 4 * j4]);
                        const float e[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
                        for (int j = 0; j < 4; j += 2) {
                            const int i = 4 * j4 + j;
                            const float2 z = unpack2(fma2(pack2(e[j], e[j + 1]), pack2(__uint_as_float(f[i]), __uint_as_float(f[i + 1])),
                                                         pack2(__uint_as_float(d[b16 + i]), __uint_as_float(d[b16 + i + 1]))));
                            x[b16 + i] = z.x;
                            x[b16 + i + 1] = z.y;
                        }
                    }
                    if (c + 1 < nc) tmem_st16(la_f + b + b16, &x[b16]);
                }
                if (c + 1 < nc) {
                    put_terms32(b, x);
                } else if (!sh.bail) {
                    float *to = a.state_out + state_at() + (size_t)b * kD;
#pragma unroll
                    for (int j = 0; j < 32; j++) to[(size_t)j * kD] = x[j];
                }
            }
            if (c + 1 < nc) {
                tmem_wait_st();
                arrive(sh.s_ready);
            }
        }
    } else if (warp < kChWarpMake) {
        // ---------------- O: value column v, every token of the chunk
        const int q = warp & 3, v = 32 * q + lane;
        const uint32_t la = tmem + ((uint32_t)(32 * q) << 16);
        const int len = own(sh.tokens), nc = (len + kC - 1) / kC;
        for (int c = 0; c < nc; c++) {
            const int n = min(kC, len - kC * c);
            const float *sc = reinterpret_cast<const float *>(stage(c) + kOffTp + kTpBytes);
            if (!wait(sh.o_full, c)) break;
            tc_fence_after();
            uint32_t w[kC / 2];                               // two tokens a word; all read before any is stored
#pragma unroll
            for (int b = 0; b < kC / 8; b++) {
                uint32_t d[8], p[8];
                tmem_ld8_nowait(la + kTmOq + 8 * b, d);
                tmem_ld8_nowait(la + kTmOp + 8 * b, p);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float2 r = *reinterpret_cast<const float2 *>(&sc[kRecQr + 8 * b + j]);
                    const __nv_bfloat162 x = __floats2bfloat162_rn(fmaf(r.x, __uint_as_float(d[j]), __uint_as_float(p[j])),
                                                                   fmaf(r.y, __uint_as_float(d[j + 1]), __uint_as_float(p[j + 1])));
                    w[4 * b + j / 2] = *reinterpret_cast<const uint32_t *>(&x);
                }
            }
            arrive(sh.o_free);
            if (lane == 0) mb_arrive(&sh.in_free[c % kStages]);
            // neighbouring lanes trade a token each: two columns of one token a store
            const int mine = lane & 1;
            uint32_t *o = reinterpret_cast<uint32_t *>(a.out + ((size_t)(own(sh.first) + kC * c + mine) * a.H + own(sh.head)) * kD + (v & ~1));
            const size_t step = (size_t)a.H * kD;             // words of two tokens
#pragma unroll
            for (int j = 0; j < kC / 2; j++, o += step) {
                asm volatile("" : "+l"(o));                   // one address at a time: all 32 at once would spill
                const uint32_t got = __shfl_xor_sync(0xffffffffu, w[j], 1);
                if (2 * j + mine < n) *o = mine ? __byte_perm(got, w[j], 0x7632) : __byte_perm(w[j], got, 0x5410);
            }
        }
    } else if (kChannel && warp < kChWarpMake + kChMake) {
        // ---------------- per channel: the weighted operands of chunk c, two channels and twice
        // 8 tokens a thread
        const int id = threadIdx.x - kChWarpMake * 32, pair = id & 63, ch = 2 * pair;
        const int len = own(sh.tokens), nc = (len + kC - 1) / kC, first = own(sh.first), h = own(sh.head), hq = h / (a.H / a.Hq);
        for (int c = 0; c < nc; c++) {
            const int n = min(kC, len - kC * c);
            const size_t tok0 = (size_t)(first + kC * c);
            const float *rf = reinterpret_cast<const float *>(record(c) + kTpBytes);
            uint8_t *kq = made + (pair >> 5) * 2 * kChBox;
            uint8_t *late = made + 4 * kChTerm + (c & 1) * 2 * kChTerm + (pair >> 5) * kChBox;
            bool ok = true;
#pragma unroll 1
            for (int part = 0; part < 2; part++) {
                const int e = (id >> 6) + 4 * part, t0 = 8 * e;
                uint32_t k[8], q[8];
                uint64_t g[8];
                {   // a token past the end reads the last one instead, and its decay counts as none; read
                    // from the L2, where they are ahead of time (8192 tokens of one sequence x 56 heads: 659 us,
                    // through the L1 1011)
                    const size_t tok = tok0 + min(t0, n - 1);
                    const uint16_t *pk = a.k + tok * a.k_stride + hq * kD + ch, *pq = a.q + tok * a.q_stride + hq * kD + ch;
                    const float *pg = a.g + (tok * a.H + h) * kD + ch;
                    const int left = n - 1 - t0;              // steps there are after this thread's first token
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        k[i] = __ldcg(reinterpret_cast<const uint32_t *>(pk));
                        q[i] = __ldcg(reinterpret_cast<const uint32_t *>(pq));
                        const float2 x = __ldcg(reinterpret_cast<const float2 *>(pg));
                        g[i] = pack2(x.x, x.y);
                        if (i < left) {
                            pk += a.k_stride;
                            pq += a.q_stride;
                            pg += (size_t)a.H * kD;
                        }
                    }
                }
                float l[8];                                   // log2 of 1 / |k|; minus infinity past the sequence's end
                *reinterpret_cast<float4 *>(&l[0]) = *reinterpret_cast<const float4 *>(&rf[kRecKd + t0]);
                *reinterpret_cast<float4 *>(&l[4]) = *reinterpret_cast<const float4 *>(&rf[kRecKd + t0 + 4]);
                // the decay's sums before and after this thread's tokens
                uint64_t L = pack2(0.0f, 0.0f), E = L;
#pragma unroll
                for (int w = 0; w < 8; w++) {
                    const float2 x = *reinterpret_cast<const float2 *>(&rf[kRecSum + w * kD + ch]);
                    L = add2(L, w < e ? pack2(x.x, x.y) : pack2(0.0f, 0.0f));
                    E = add2(E, w > e ? pack2(x.x, x.y) : pack2(0.0f, 0.0f));
                }
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float2 x = unpack2(g[i]);
                    g[i] = t0 + i < n ? mul2(pack2(clamp_gate(x.x), clamp_gate(x.y)), pack2(kLog2e, kLog2e)) : pack2(0.0f, 0.0f);
                }
                if (part == 0 && c >= 1) ok = wait(sh.q_done, c - 1);      // the last chunk's K and Q are used
                if (!ok) break;
                const uint32_t row = (uint32_t)t0 * 128 + (lane & 3) * 4, c8 = (uint32_t)lane >> 2;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const uint32_t at = row + i * 128 + ((c8 ^ i) << 4);
                    L = add2(L, g[i]);
                    const float2 s = unpack2(L);
                    const uint64_t w = pack2(exp2_fast(s.x), exp2_fast(s.y));
                    uint32_t hi, mid;
                    split2(mul2(pair_bf16(k[i]), w), &hi, &mid);
                    *reinterpret_cast<uint32_t *>(kq + at) = hi;
                    *reinterpret_cast<uint32_t *>(kq + 2 * kChTerm + at) = mid;
                    split2(mul2(pair_bf16(q[i]), w), &hi, &mid);
                    *reinterpret_cast<uint32_t *>(kq + kChBox + at) = hi;
                    *reinterpret_cast<uint32_t *>(kq + 2 * kChTerm + kChBox + at) = mid;
                }
                if (e == 7) {
                    const float2 s = unpack2(L);
                    *reinterpret_cast<float2 *>(&sh.dec[c & 1][ch]) = make_float2(exp2_fast(s.x), exp2_fast(s.y));
                }
#pragma unroll
                for (int i = 7; i >= 0; i--) {                // backwards: exp(G_C - G_t), from the end's sum
                    const uint32_t at = row + i * 128 + ((c8 ^ i) << 4);
                    const float2 s = unpack2(add2(E, pack2(l[i], l[i])));
                    uint32_t hi, mid;
                    split2(mul2(pair_bf16(k[i]), pack2(exp2_fast(s.x), exp2_fast(s.y))), &hi, &mid);
                    *reinterpret_cast<uint32_t *>(late + at) = hi;
                    *reinterpret_cast<uint32_t *>(late + kChTerm + at) = mid;
                    E = add2(E, g[i]);
                }
            }
            if (!ok) break;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mb_arrive(&sh.made);
        }
    } else if (warp == kWarpMma) {
        // ---------------- MMA issue
        const uint32_t idk = idesc(1, kC);                     // 128 x 64, both operands K-major
        const uint32_t idn = idesc(1, 2 * kC) | (1u << 16);    // 128 x 128, B with N contiguous (K^T U: channels)
        // X S^T, X's 64-channel boxes two apart: S hi, S mid, and (per channel) S hi with X mid
        auto with_state = [&](uint32_t d, uint32_t x) {
#pragma unroll 1
            for (int term = 0; term < (kChannel ? 3 : 2); term++)
#pragma unroll
                for (int s = 0; s < 8; s++)
                    umma_ts_warp(d, kTmS + 32 * (s >> 1) + 16 * (term == 1) + 8 * (s & 1),
                                 x + (((term == 2 ? 2 * kChTerm : 0) + (s >> 2) * 2 * kChBox + (s & 3) * 32) >> 4), idk,
                                 term > 0 || s > 0);
        };
        // D[v][t >= 16 j] += X[v][16 tokens j] tile[t][16 tokens j], the tile lower triangular
        // (hi, mid terms), X's terms at columns `x`
        auto tri = [&](uint32_t d, uint32_t x, uint32_t tile) {
            const uint32_t td = desc_lo(tile, 128);
#pragma unroll 1
            for (int term = 0; term < 3; term++)               // hi hi, hi mid, mid hi
#pragma unroll
                for (int j = 0; j < 4; j++)
                    umma_ts_warp<kDescTp>(d + 16 * j, x + 32 * (j >> 1) + (term == 2 ? 16 : 0) + 8 * (j & 1),
                                 td + (((term == 1 ? kTermBytes : 0) + term_block(j)) >> 4), idesc(1, kC - 16 * j),
                                 term > 0 || j > 0);
        };
        // the count and the stages' place as uniform values, so that descriptors are too
        const int chunks = (int)__reduce_max_sync(0xffffffffu, (unsigned)(own(sh.tokens) + kC - 1) / kC);
        int slot_st = 0;
        for (int c = 0; c < chunks; c++, slot_st = slot_st + 1 == kStages ? 0 : slot_st + 1) {
            if (!wait(sh.in_full[c % kStages], c / kStages) || (kChannel && !wait(sh.made, c)) || !wait(sh.s_ready, c)) break;
            tc_fence_after();
            const uint32_t st = saddr(ring) + (uint32_t)(slot_st * Shape::stage), mk0 = saddr(made);
            const uint32_t kq = desc_lo(kChannel ? mk0 : st);
            with_state(kTmR, kq);                              // K S
            umma_commit_warp(&sh.d1_full);
            if (c >= 1 && !wait(sh.o_free, c - 1)) break;      // chunk c - 1's O is read: its columns are free
            tc_fence_after();
            with_state(kTmOq, kq + (kChBox >> 4));             // Q S, under the chain's next step
            if (kChannel) umma_commit_warp(&sh.q_done);
            if (!wait(sh.r_ready, c)) break;
            tc_fence_after();
            const uint32_t tp = st + kOffTp;
            tri(kTmR, kTmRU, tp);
            umma_commit_warp(&sh.d2_full);
            if (!wait(sh.u_ready, c)) break;
            tc_fence_after();
            // B with N contiguous: 64 channels a box, the boxes a leading offset apart
            constexpr int box = kChannel ? kChBox : 2 * kChBox;
            const uint32_t lx = desc_lo(kChannel ? mk0 + 4 * kChTerm + (c & 1) * 2 * kChTerm : st, box);
#pragma unroll 1
            for (int term = 0; term < (kChannel ? 3 : 2); term++)   // K^T U into the state's sums
#pragma unroll
                for (int s = 0; s < 4; s++)
                    umma_ts_warp(kTmS, kTmRU + 32 * (s >> 1) + 16 * (term == 1) + 8 * (s & 1), lx + (((term == 2 ? kChTerm : 0) + s * 16 * 128) >> 4),
                                 idn, term > 0 || s > 0);
            umma_commit_warp(&sh.d4_full);
            tri(kTmOp, kChannel ? kTmRU : kTmR, tp + 2 * kTermBytes);
            umma_commit_warp(&sh.o_full);
        }
        __syncwarp();
        umma_commit_warp(&sh.drain);                           // every issued MMA done before the dealloc
        mb_wait_warp(&sh.drain, 0);
    } else if (warp == kWarpLoad) {
        // ---------------- loads
        const int len = own(sh.tokens), nc = (len + kC - 1) / kC, first = own(sh.first), h = own(sh.head), hq = h / (a.H / a.Hq);
        auto load = [&](int c) {
            uint8_t *p = stage(c);
            uint64_t *bar = &sh.in_full[c % kStages];
            mb_expect_tx(bar, (kChannel ? 0 : kChKq) + kChV + kChTpCopy);
            for (int b = 0; b < 2; b++) {
                if (!kChannel) {
                    tma2d(p + 2 * b * kChBox, &mk, hq * kD + 64 * b, first + kC * c, bar);
                    tma2d(p + 2 * b * kChBox + kChBox, &mq, hq * kD + 64 * b, first + kC * c, bar);
                }
                tma2d(p + kOffV + b * kChBox, &mv, h * kD + 64 * b, first + kC * c, bar);
            }
            bulk_g2s(p + kOffTp, record(c), kChTpCopy, bar);
        };
        // per channel: what the makers of chunk c's operands read, brought to the L2 (from DRAM
        // their loads, a dependent step in every chunk, took three thousand clocks)
        auto ahead = [&](int c) {
            const int t0 = first + kC * c;
            for (int t = lane; t < kC; t += 32)
                if (t0 + t < first + len) prefetch_bulk(a.g + ((size_t)(t0 + t) * a.H + h) * kD, kD * 4);
            if (lane < 2) {
                prefetch2d(&mk, hq * kD + 64 * lane, t0);
                prefetch2d(&mq, hq * kD + 64 * lane, t0);
            }
            if (lane == 0) prefetch_bulk(record(c), kRecBytes);
        };
        int loaded = 0;
        for (; loaded < nc; loaded++) {
            if (loaded >= kStages && !wait(sh.in_free[loaded % kStages], loaded / kStages - 1)) break;
            if (lane == 0) load(loaded);
            if (kChannel && loaded + 1 < nc) ahead(loaded + 1);
            __syncwarp();
        }
        // the block's shared memory stays until its last copies have landed, when another role gave up too
        for (int c = max(0, loaded - kStages); c < loaded; c++) wait(sh.in_full[c % kStages], c / kStages);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(512));
}

// From this many tokens a sequence on average, chunks; `alone` where the recurrent kernel's
// blocks have an SM each.  Recurrent against chunks, us, per head: 64 sequences x 32 heads of 16
// tokens 153, 159 and of 18 173, 161; 8 x 32 heads of 14 23, 24 and of 18 29, 24; alone (one
// sequence, 56 heads) of 22 13.3, 14.3 and of 26 15.5, 14.3.  Per channel: 37 x 56 heads of 26
// tokens 252, 253 and of 28 268, 254; alone of 36 20.2, 20.6.  All of these are sequences of equal
// lengths, and the choice is the call's: with one prompt of 1000 tokens among 95 single ones (32 heads)
// all go token by token, 657 us (per channel 719) where two calls take 69 and 63 (97 and 63); of 4000
// tokens all in chunks, 287 (472), two calls 221 and 63 (323 and 63).
constexpr int chunk_tokens_avg(bool channel, bool alone) { return channel ? (alone ? 37 : 27) : (alone ? 24 : 17); }

// Where the chains leave SMs free, the sequences are walked in stretches: while the chains go
// through one, the SMs that are left prepare the next.  A stretch is as much longer than the
// one before as preparing on those SMs is faster than the chains; the number of stretches is
// the one with the least estimated time (microseconds: a chunk and head prepared on one SM,
// a chain's chunk, and what one stretch more costs), ends[i] the chunk that ends the i-th.
// In one and so, us: one sequence of 8192 tokens x 56 heads 513, 442, x 140 heads 659, 642;
// per channel 841, 658 and 1241, 1205; 512 tokens x 56 heads per channel 61, 63.
constexpr int kMaxStretches = 8;
template <bool kChannel>
int plan_stretches(const DeltaArgs &a, int (&ends)[kMaxStretches])
{
    ends[0] = kAllChunks;
    const long long jobs = (long long)a.n_seq * a.H;
    const int sms = num_sms(), last = (a.T + kC - 1) / kC;
    if (jobs >= sms) return 1;
    constexpr double prepare = kChannel ? 5.5 : 2.3, chain = kChannel ? 4.6 : 3.2;
    constexpr double extra = 8.0;
    const double chunks = (double)last / a.n_seq, grow = chain * (double)(sms - jobs) / (prepare * jobs);
    int n = 1;
    double least = 0.0, first = chunks, sum = 1.0, power = 1.0;
    for (int k = 1; k <= kMaxStretches; k++, sum += power *= grow) {
        const double us = chunks / sum * prepare * jobs / sms + (k - 1) * extra;
        if (k == 1 || us < least) {
            n = k;
            least = us;
            first = chunks / sum;
        }
    }
    if (n == 1) return 1;
    double end = 0.0;
    for (int i = 0; i + 1 < n; i++, first *= grow) {
        end += first;
        ends[i] = std::min(std::max((int)(end + 0.5), 1), last);
    }
    ends[n - 1] = last;
    return n;
}

template <bool kChannel>
cudaError_t launch_chunks(const DeltaArgs &a, cudaStream_t s)
{
    CUtensorMap mq{}, mk{}, mv{};
    const uint64_t cols = (uint64_t)a.Hq * kD;
    if (!map16s(&mq, a.q, (uint64_t)a.T, cols, (uint64_t)a.q_stride, kC) ||
        !map16s(&mk, a.k, (uint64_t)a.T, cols, (uint64_t)a.k_stride, kC) ||
        !map16s(&mv, a.v, (uint64_t)a.T, (uint64_t)a.H * kD, (uint64_t)a.v_stride, kC))
        return cudaErrorInvalidValue;
    using Shape = ChunkShape<kChannel>;
    const cudaError_t allowed = once_a_device([] {
        // the shares of setmaxnreg are of the launch's registers: with another count they would never be there
        cudaFuncAttributes fa{};
        if (kChannel && (cudaFuncGetAttributes(&fa, delta_chunk_kernel<kChannel>) != cudaSuccess || fa.numRegs != kChRegs))
            return cudaErrorInvalidConfiguration;
        const cudaError_t e = cudaFuncSetAttribute(delta_chunk_kernel<kChannel>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::smem);
        return e != cudaSuccess ? e
                                : cudaFuncSetAttribute(delta_prepare_kernel<kChannel>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (int)pp_smem(kChannel));
    });
    if (allowed != cudaSuccess) return allowed;
    int ends[kMaxStretches];
    const int stretches = plan_stretches<kChannel>(a, ends);
    cudaError_t err = cudaSuccess;
    DeltaArgs x = a;
    for (int i = 0; i < stretches && err == cudaSuccess; i++) {
        x.chunk0 = i > 0 ? ends[i - 1] : 0;
        x.chunk1 = ends[i];
        if (x.chunk1 <= x.chunk0) continue;
        const long long units = x.chunk1 < kAllChunks ? (long long)(x.chunk1 - x.chunk0) * a.n_seq : chunk_records(a.n_seq, a.T);
        x.units = (int32_t)(units * a.H);
        // blocks that stay: on every SM, or on those that a later stretch has beside the chains
        const int sms = i > 0 ? std::max(1, num_sms() - ((a.n_seq * a.H + 1) & ~1)) : num_sms();
        const int blocks = kChannel ? x.units : std::min(x.units, sms * kPpBlocks<kChannel>);
        timing_begin("delta_prepare", s);
        err = launch_pdl(delta_prepare_kernel<kChannel>, dim3((unsigned)blocks), dim3(kPpThreads), pp_smem(kChannel), s, x, mq, mk);
        count_launch();
        timing_end("delta_prepare", s);
        if (err != cudaSuccess) return err;
        timing_begin("delta_chunk", s);
        // Beside a prepare the chains go in pairs, a cluster of two on the SMs of a TPC: a chain whose
        // neighbour there runs other code takes a quarter to a half longer (8192 tokens x 56 heads: 442
        // us in pairs, 488 singly; per channel 658, 782; two sequences 304, 331 and 548, 641).
        const bool pairs = stretches > 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(pairs ? (a.n_seq * a.H + 1) & ~1 : a.n_seq * a.H));
        cfg.blockDim = dim3(Shape::threads);
        cfg.dynamicSmemBytes = Shape::smem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 2;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = pairs ? 2 : 1;
        err = cudaLaunchKernelEx(&cfg, delta_chunk_kernel<kChannel>, x, mq, mk, mv);
        count_launch();
        timing_end("delta_chunk", s);
    }
    return err;
}

}  // namespace

size_t delta_workspace(const k3moe_delta_config &dc, int n_seq, int T)
{
    // the most records of any call of at most n_seq sequences and T tokens: chunks need that
    // many tokens a sequence
    size_t bytes = kCtrOffset + kCtrBytes;
    const int avg = chunk_tokens_avg(dc.gate_dim > 1, false);
    if (T >= avg && n_seq > 0) bytes += (size_t)chunk_records(std::min(n_seq, T / avg), T) * dc.n_heads * kRecBytes;
    return bytes;
}

cudaError_t launch_delta(const DeltaArgs &a, cudaStream_t s)
{
    const long long blocks = (long long)a.n_seq * a.H * (kD / kRecCols);
    if (a.T >= (long long)chunk_tokens_avg(a.gate > 1, blocks <= num_sms()) * a.n_seq)
        return a.gate == 1 ? launch_chunks<false>(a, s) : launch_chunks<true>(a, s);
    timing_begin("delta_recurrent", s);
    const cudaError_t err = launch_pdl(delta_recurrent_kernel, dim3((unsigned)blocks), dim3(kRecThreads), 0, s, a);
    count_launch();
    timing_end("delta_recurrent", s);
    return err;
}

}  // namespace k3moe
