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

#include "k3moe_internal.cuh"
#include "k3moe_tc.cuh"

namespace k3moe {
namespace {

constexpr int kD = kDeltaD;
constexpr int kRecThreads = 256, kRecWarps = kRecThreads / 32;

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

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Four bf16 of an 8-byte word.
__device__ __forceinline__ float4 bf4(uint2 w)
{
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}

// One token's vectors as a lane holds them: four channels of q, k and the decay.
struct TokenRaw {
    uint2 q, k;
    float4 g;
    uint2 v;
    float beta;
};

// One block per (sequence, head, CW value columns).  A thread holds RPT key rows x 4 value
// columns of the state; a warp covers 32 / (CW / 4) groups of rows.
template <int CW>
__global__ void __launch_bounds__(kRecThreads) delta_recurrent_kernel(const DeltaArgs a)
{
    pdl_wait();
    pdl_trigger();
    constexpr int kLanes = CW / 4;                       // lanes across the columns
    constexpr int kGroups = kRecThreads / kLanes;        // groups of rows
    constexpr int RPT = kD / kGroups;                    // rows a thread holds
    constexpr int kSplit = kD / CW;
    __shared__ float red[2][kRecWarps][2][CW];           // partial sums of r and W^T q, two tokens' worth
    __shared__ float vec[kRecWarps][3][kD];              // each warp's copy of k, q and exp(g)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cs = blockIdx.x % kSplit, h = (blockIdx.x / kSplit) % a.H, seq = blockIdx.x / (kSplit * a.H);
    int first, len, slot;
    if (!delta_seq(a, seq, &first, &len, &slot)) return;
    const int cl = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
    const int col = cs * CW + 4 * cl, row0 = grp * RPT;
    const size_t sbase = ((size_t)slot * a.H + h) * kD * kD + (size_t)row0 * kD + col;

    float4 S[RPT];
#pragma unroll
    for (int j = 0; j < RPT; j++)
        S[j] = a.state_in ? __ldcs(reinterpret_cast<const float4 *>(a.state_in + sbase + (size_t)j * kD))
                          : make_float4(0.f, 0.f, 0.f, 0.f);

    const int hq = h / (a.H / a.Hq);
    auto fetch = [&](int i) {
        TokenRaw t;
        const size_t tok = (size_t)(first + i);
        t.q = *reinterpret_cast<const uint2 *>(a.q + tok * a.q_stride + hq * kD + 4 * lane);
        t.k = *reinterpret_cast<const uint2 *>(a.k + tok * a.k_stride + hq * kD + 4 * lane);
        t.v = *reinterpret_cast<const uint2 *>(a.v + tok * a.v_stride + h * kD + col);
        if (a.gate == 1) {
            const float g = a.g[tok * a.H + h];
            t.g = make_float4(g, g, g, g);
        } else {
            t.g = *reinterpret_cast<const float4 *>(a.g + (tok * a.H + h) * kD + 4 * lane);
        }
        t.beta = a.beta[tok * a.H + h];
        return t;
    };
    TokenRaw nxt;
    if (len > 0) nxt = fetch(0);
    for (int i = 0; i < len; i++) {
        const TokenRaw cur = nxt;
        if (i + 1 < len) nxt = fetch(i + 1);             // in flight under this token's work
        float4 q = bf4(cur.q), k = bf4(cur.k);
        float qs = a.scale, ks = 1.0f;
        if (a.qk_norm) {
            const float qq = warp_sum(q.x * q.x + q.y * q.y + q.z * q.z + q.w * q.w);
            const float kk = warp_sum(k.x * k.x + k.y * k.y + k.z * k.z + k.w * k.w);
            qs = a.scale / sqrtf(qq + a.eps);
            ks = 1.0f / sqrtf(kk + a.eps);
        }
        q = make_float4(q.x * qs, q.y * qs, q.z * qs, q.w * qs);
        k = make_float4(k.x * ks, k.y * ks, k.z * ks, k.w * ks);
        const float qk = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w);
        __syncwarp();
        reinterpret_cast<float4 *>(vec[warp][0])[lane] = k;
        reinterpret_cast<float4 *>(vec[warp][1])[lane] = q;
        reinterpret_cast<float4 *>(vec[warp][2])[lane] =
            make_float4(expf(cur.g.x), expf(cur.g.y), expf(cur.g.z), expf(cur.g.w));
        __syncwarp();
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f), o = r;
#pragma unroll
        for (int j = 0; j < RPT; j++) {
            const float kj = vec[warp][0][row0 + j], qj = vec[warp][1][row0 + j], dj = vec[warp][2][row0 + j];
            S[j].x *= dj; S[j].y *= dj; S[j].z *= dj; S[j].w *= dj;
            r.x = fmaf(kj, S[j].x, r.x); r.y = fmaf(kj, S[j].y, r.y);
            r.z = fmaf(kj, S[j].z, r.z); r.w = fmaf(kj, S[j].w, r.w);
            o.x = fmaf(qj, S[j].x, o.x); o.y = fmaf(qj, S[j].y, o.y);
            o.z = fmaf(qj, S[j].z, o.z); o.w = fmaf(qj, S[j].w, o.w);
        }
        // over the warp's groups of rows, then over the warps (in warp order)
#pragma unroll
        for (int s = kLanes; s < 32; s <<= 1) {
            r.x += __shfl_xor_sync(0xffffffffu, r.x, s); r.y += __shfl_xor_sync(0xffffffffu, r.y, s);
            r.z += __shfl_xor_sync(0xffffffffu, r.z, s); r.w += __shfl_xor_sync(0xffffffffu, r.w, s);
            o.x += __shfl_xor_sync(0xffffffffu, o.x, s); o.y += __shfl_xor_sync(0xffffffffu, o.y, s);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, s); o.w += __shfl_xor_sync(0xffffffffu, o.w, s);
        }
        float (*rd)[2][CW] = red[i & 1];                 // the other buffer is still being read
        if (lane < kLanes) {
            *reinterpret_cast<float4 *>(&rd[warp][0][4 * cl]) = r;
            *reinterpret_cast<float4 *>(&rd[warp][1][4 * cl]) = o;
        }
        __syncthreads();
        r = o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kRecWarps; w++) {
            const float4 p = *reinterpret_cast<const float4 *>(&rd[w][0][4 * cl]);
            r.x += p.x; r.y += p.y; r.z += p.z; r.w += p.w;
        }
        const float4 v = bf4(cur.v);
        const float4 u = make_float4(cur.beta * (v.x - r.x), cur.beta * (v.y - r.y), cur.beta * (v.z - r.z),
                                     cur.beta * (v.w - r.w));
#pragma unroll
        for (int j = 0; j < RPT; j++) {
            const float kj = vec[warp][0][row0 + j];
            S[j].x = fmaf(kj, u.x, S[j].x); S[j].y = fmaf(kj, u.y, S[j].y);
            S[j].z = fmaf(kj, u.z, S[j].z); S[j].w = fmaf(kj, u.w, S[j].w);
        }
        if (grp == 0) {
#pragma unroll
            for (int w = 0; w < kRecWarps; w++) {
                const float4 p = *reinterpret_cast<const float4 *>(&rd[w][1][4 * cl]);
                o.x += p.x; o.y += p.y; o.z += p.z; o.w += p.w;
            }
            const __nv_bfloat162 lo = __floats2bfloat162_rn(fmaf(qk, u.x, o.x), fmaf(qk, u.y, o.y));
            const __nv_bfloat162 hi = __floats2bfloat162_rn(fmaf(qk, u.z, o.z), fmaf(qk, u.w, o.w));
            uint2 st;
            st.x = *reinterpret_cast<const uint32_t *>(&lo);
            st.y = *reinterpret_cast<const uint32_t *>(&hi);
            *reinterpret_cast<uint2 *>(a.out + ((size_t)(first + i) * a.H + h) * kD + col) = st;
        }
    }
#pragma unroll
    for (int j = 0; j < RPT; j++) __stcs(reinterpret_cast<float4 *>(a.state_out + sbase + (size_t)j * kD), S[j]);
}

// ---------------------------------------------------------------- chunks of 64 tokens
// For a chunk, with G_t the decay's logarithm summed from its start to token t:
//   A_ti = beta_t exp(G_t - G_i) k_t . k_i  (i < t),   P_ti = scale exp(G_t - G_i) q_t . k_i  (i <= t)
//   T = (I + A)^-1 diag(beta),  U = T (V - diag(exp(G)) K S),
//   O = scale diag(exp(G)) Q S + P U,   S <- exp(G_C) S + (diag(exp(G_C - G)) K)^T U.
// A unit lower triangular solve replaces 64 dependent steps, and all else is products on
// the tensor cores.  Every exponent is a later token's sum minus an earlier one's, so no
// factor exceeds one however strong the decay (a logarithm below -200 counts as -200: its
// exponential is zero in float either way).
//
// One block per sequence and head walks its chunks; everything is transposed so that a
// thread owns one value column v (a lane of tensor memory) and the state S^T [v][k] stays
// with it: the A operands (S, R = V - .., U) go from registers to tensor memory and never
// through shared memory, and the B operands (K and Q as they are, T, P) are shared tiles.
// K and Q are exact in bf16; S, R, U, T and P enter as two bf16 terms each (hi + mid, 16
// bits: 2^-18 of the element, where one term's 2^-9 would show in the float state), every
// product of two such as hi hi + hi mid + mid hi.  Sums are float, in tensor memory; the
// state's carry S exp(G_C) + .. is a float in a register.
//
// Warps: 0-7 prepare T and P of the next chunk while the chain of this one runs; 8-23 are
// the chain S -> R -> U -> S; 24-27 write O and compute the next but one chunk's scales; 28
// issues the loads and the MMAs.  A single warp's dependent instructions issue every three
// to five clocks, so each stage has as many warps as the registers allow (64 a thread).
constexpr int kC = 64;                                        // tokens a chunk
constexpr int kChPrep = 8, kChChain = 16, kChOut = 4;
constexpr int kChWarpChain = kChPrep, kChWarpOut = kChWarpChain + kChChain, kChWarpMma = kChWarpOut + kChOut;
constexpr int kChThreads = (kChWarpMma + 1) * 32;             // 928
constexpr int kChStages = 3;
constexpr int kChBox = 2 * kC * 128;                          // 64 channels of K then of Q: 16 KB
constexpr int kChV = 2 * kChBox;                              // after both, V: two boxes of 64 columns
constexpr int kChStageBytes = kChV + kC * kD * 2;             // 48 KB
constexpr int kChTile = kC * 128;                             // one term of T or P: 8 KB
constexpr int kChLd = 68;                                     // row stride of the float scratch
constexpr size_t kChSmem = 1024 + kChStages * kChStageBytes + 6 * kChTile + kC * kChLd * 4;   // T, two P, the scratch
// tensor memory columns
constexpr uint32_t kTmS = 0;      // S^T as an operand, [quarter of k][hi, mid][16]; the new S's sums over it
constexpr uint32_t kTmR = 128;    // K S, then T R
constexpr uint32_t kTmOq = 192;   // Q S
constexpr uint32_t kTmOp = 256;   // P U
constexpr uint32_t kTmRU = 320;   // R, then U scaled for the state, as an operand [hi, mid][32]
constexpr uint32_t kTmU = 384;    // U as an operand [hi, mid][32]
constexpr uint32_t kTmKK = 448;   // K K^T (lanes 0-63) and Q K^T (lanes 64-127) of the next chunk

constexpr int kChScales = 4;
struct ChunkShared {
    uint64_t kq_full[kChStages];
    uint64_t kk_full, kk_free, sc_ready[kChScales], tp_ready, s_ready, d1_full, r_ready, d2_full, u_ready, d4_full, o_full, o_free,
        drain;
    uint32_t tmem;
    volatile int bail;
    // a chunk's scales (of the chunk's number modulo kChScales), with G_t the decay's sum and
    // r = 1 / |k_t| (1 without qk_norm):
    //   g2 = log2(e) G_t, gk = g2 - log2 r, kb = beta_t r, kr = r exp(G_t), kd = r exp(G_C - G_t),
    //   qn = scale / |q_t|, qr = qn exp(G_t), dec = exp(G_C); 0 (gk: infinity) past the end
    struct Scales {
        alignas(16) float g2[kC], gk[kC], beta[kC], kb[kC], kr[kC], kd[kC], qn[kC], qr[kC];
        float dec, pad[3];
    } sc[kChScales];
};

constexpr float kLog2e = 1.4426950408889634f;
// 2^x, x <= 0, within 2 ulp; volatile so that a select of its result stays a select (as a
// branch around it, each of a row's 64 would be waited for by itself).
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (x, y) as two packed bf16 terms: hi rounded to nearest, mid the rounded remainder.
__device__ __forceinline__ void split2(float x, float y, uint32_t *hi, uint32_t *mid)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const uint32_t u = *reinterpret_cast<const uint32_t *>(&h);
    const __nv_bfloat162 m = __floats2bfloat162_rn(x - __uint_as_float(u << 16), y - __uint_as_float(u & 0xFFFF0000u));
    *hi = u;
    *mid = *reinterpret_cast<const uint32_t *>(&m);
}
// Eight values of row t, columns 8 c8.., as two terms of a swizzled tile.
__device__ __forceinline__ void put_terms(uint8_t *tile, int t, int c8, const float (&x)[8])
{
    uint32_t h[4], m[4];
#pragma unroll
    for (int j = 0; j < 4; j++) split2(x[2 * j], x[2 * j + 1], &h[j], &m[j]);
    uint8_t *p = tile + t * 128 + ((c8 ^ (t & 7)) << 4);
    *reinterpret_cast<uint4 *>(p) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(p + kChTile) = make_uint4(m[0], m[1], m[2], m[3]);
}
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
__device__ __forceinline__ void prep_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kChPrep * 32) : "memory"); }

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// A warp's 16 x 8 tile of X Y over K, X and Y in shared memory with rows kChLd floats apart:
// tf32 MMAs on two terms each (hi + lo, 22 bits; hi hi + hi lo + lo hi), which read an
// element once a tile where plain FMAs, at four outputs a thread, read it once a thread
// (the whole inverse: 7.4 thousand clocks of shared-memory reads, against 2).
template <int K>
__device__ __forceinline__ void block_product(float (&d)[4], const float *X, const float *Y, int lane)
{
    const int g = lane >> 2, t = lane & 3;
    d[0] = d[1] = d[2] = d[3] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; k += 8) {
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
        mma_tf32(d, al, bh);
        mma_tf32(d, ah, bl);
        mma_tf32(d, ah, bh);
    }
}
__device__ __forceinline__ void store_tile(float *D, const float (&d)[4], float sign, int lane)
{
    const int g = lane >> 2, t = (lane & 3) * 2;
    *reinterpret_cast<float2 *>(&D[g * kChLd + t]) = make_float2(sign * d[0], sign * d[1]);
    *reinterpret_cast<float2 *>(&D[(g + 8) * kChLd + t]) = make_float2(sign * d[2], sign * d[3]);
}

// A <- (I + A)^-1 of a strictly lower triangular 64 x 64 A (rows kChLd floats apart), in
// place and by blocks: the 16 x 16 diagonal blocks by substitution, then twice
// [X11 0; -X22 A21 X11, X22].  Above the diagonal blocks is scratch.  256 threads.
__device__ __forceinline__ void invert64(float *A, int tid)
{
    const int warp = tid >> 5, lane = tid & 31;
    if (warp < 4) {   // column `lane` of diagonal block `warp` (lanes from 16 on repeat the others' work)
        float *a = A + (16 * warp) * (kChLd + 1);
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
        if (lane < 16)
#pragma unroll
            for (int t = 0; t < 16; t++) a[t * kChLd + col] = x[t];       // zero above the diagonal
    }
    prep_sync();
    {   // 16 -> 32: two pairs of blocks, two tiles of 16 x 8 each, a tile for each of four warps
        float *a = A + 32 * (warp >> 1) * (kChLd + 1);
        const int n0 = (warp & 1) * 8;
        float w[4];
        if (warp < 4) {
            block_product<16>(w, &a[16 * kChLd], &a[n0], lane);           // A21 X11
            store_tile(&a[16 + n0], w, 1.0f, lane);
        }
        prep_sync();
        if (warp < 4) {
            block_product<16>(w, &a[16 * kChLd + 16], &a[16 + n0], lane); // X22 (A21 X11)
            store_tile(&a[16 * kChLd + n0], w, -1.0f, lane);
        }
        prep_sync();
        const int r = (tid & 127) >> 3, c = (tid & 7) * 2;
        *reinterpret_cast<float2 *>(&A[(32 * (tid >> 7) + r) * kChLd + 32 * (tid >> 7) + 16 + c]) = make_float2(0.f, 0.f);
    }
    prep_sync();
    {   // 32 -> 64: eight tiles of 16 x 8, one a warp
        const int m0 = 16 * (warp >> 2), n0 = 8 * (warp & 3);
        float w[4];
        block_product<32>(w, &A[(32 + m0) * kChLd], &A[n0], lane);
        store_tile(&A[m0 * kChLd + 32 + n0], w, 1.0f, lane);
        prep_sync();
        block_product<32>(w, &A[(32 + m0) * kChLd + 32], &A[32 + n0], lane);
        store_tile(&A[(32 + m0) * kChLd + n0], w, -1.0f, lane);
    }
    prep_sync();
}

__global__ void __launch_bounds__(kChThreads, 1) delta_chunk_kernel(const DeltaArgs a,
                                                                    const __grid_constant__ CUtensorMap mq,
                                                                    const __grid_constant__ CUtensorMap mk,
                                                                    const __grid_constant__ CUtensorMap mv)
{
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(1024) uint8_t csm_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(csm_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *tT = sm + kChStages * kChStageBytes, *tP = tT + 2 * kChTile;
    float *As = reinterpret_cast<float *>(tP + 4 * kChTile);
    __shared__ ChunkShared sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % a.H, seq = blockIdx.x / a.H;
    int first, len, slot;
    if (!delta_seq(a, seq, &first, &len, &slot)) return;
    const size_t sbase = ((size_t)slot * a.H + h) * kD * kD;
    if (len == 0) {
        for (int e = threadIdx.x; e < kD * kD / 4; e += kChThreads)
            reinterpret_cast<float4 *>(a.state_out + sbase)[e] =
                a.state_in ? reinterpret_cast<const float4 *>(a.state_in + sbase)[e] : make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    const int hq = h / (a.H / a.Hq), nc = (len + kC - 1) / kC;
    int32_t *status = reinterpret_cast<int32_t *>(a.ws);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kChStages; s++) mb_init(&sh.kq_full[s], 1);
        mb_init(&sh.kk_full, 1);
        mb_init(&sh.kk_free, kChPrep);
        for (int p = 0; p < kChScales; p++) mb_init(&sh.sc_ready[p], kChOut);
        mb_init(&sh.tp_ready, kChPrep);
        mb_init(&sh.s_ready, kChChain);
        mb_init(&sh.d1_full, 1);
        mb_init(&sh.r_ready, kChChain);
        mb_init(&sh.d2_full, 1);
        mb_init(&sh.u_ready, kChChain);
        mb_init(&sh.d4_full, 1);
        mb_init(&sh.o_full, 1);
        mb_init(&sh.o_free, kChOut);
        mb_init(&sh.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.bail = 0;
    }
    if (warp == kChWarpMma) {
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
            set_status(status, K3MOE_DEV_TIMEOUT);
            sh.bail = 1;
        }
        return ok && !sh.bail;
    };
    // A warp's accesses to tensor memory are done: tell the barrier's waiter.
    auto arrive = [&](uint64_t &b) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mb_arrive(&b);
    };

    if (warp < kChPrep) {
        // ---------------- T and P of chunk c: lanes 0-63 of tensor memory hold A's rows, 64-127
        // P's; a warp takes 32 rows of one of the two, half of their columns
        const int row = 32 * (warp & 3) + lane, t = row & (kC - 1), i00 = 32 * (warp >> 2);
        const bool is_a = row < kC;
        for (int c = 0; c < nc; c++) {
            const int n = min(kC, len - kC * c);
            if (!wait(sh.sc_ready[c % kChScales], c / kChScales) || !wait(sh.kk_full, c)) break;
            tc_fence_after();                                 // chunk c - 2's P is used: the MMAs' issue saw to it
            const ChunkShared::Scales &sc = sh.sc[c % kChScales];
            const float rowf = is_a ? sc.kb[t] : sc.qn[t], g2 = sc.g2[t];
            const int last = t < n ? (is_a ? t - 1 : t) : -1;          // the row's last token
            uint8_t *tPc = tP + (c & 1) * 2 * kChTile;
#pragma unroll 1
            for (int i0 = i00; i0 < i00 + 32; i0 += 16) {
                float v[16];
                tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kTmKK + i0, v);
#pragma unroll
                for (int j4 = 0; j4 < 4; j4++) {
                    const float4 gk4 = *reinterpret_cast<const float4 *>(&sc.gk[i0 + 4 * j4]);
                    const float gk[4] = {gk4.x, gk4.y, gk4.z, gk4.w};
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float x = v[4 * j4 + j] * (rowf * exp2_approx(g2 - gk[j]));
                        v[4 * j4 + j] = i0 + 4 * j4 + j <= last ? x : 0.0f;
                    }
                }
                if (is_a) {
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        *reinterpret_cast<float4 *>(&As[t * kChLd + i0 + 4 * j]) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                } else {
                    const float(*v8)[8] = reinterpret_cast<const float(*)[8]>(v);
                    put_terms(tPc, t, i0 / 8, v8[0]);
                    put_terms(tPc, t, i0 / 8 + 1, v8[1]);
                }
            }
            arrive(sh.kk_free);
            prep_sync();
            invert64(As, threadIdx.x);
            if (c >= 1 && !wait(sh.d2_full, c - 1)) break;    // T of chunk c - 1 is used
            {
                const int r = threadIdx.x >> 2, c0 = (threadIdx.x & 3) * 16;
#pragma unroll
                for (int j8 = 0; j8 < 2; j8++) {
                    float x[8], b[8];
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        *reinterpret_cast<float4 *>(&x[j]) = *reinterpret_cast<const float4 *>(&As[r * kChLd + c0 + 8 * j8 + j]);
                        *reinterpret_cast<float4 *>(&b[j]) = *reinterpret_cast<const float4 *>(&sc.beta[c0 + 8 * j8 + j]);
                    }
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const float y = x[j] * b[j];
                        x[j] = c0 + 8 * j8 + j <= r ? y : 0.0f;
                    }
                    put_terms(tT, r, c0 / 8 + j8, x);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mb_arrive(&sh.tp_ready);
            prep_sync();                                      // the scratch is free again
        }
    } else if (warp < kChWarpOut) {
        // ---------------- the chain: value column v, a quarter of the channels or tokens
        const int q = warp & 3, part = (warp - kChWarpChain) >> 2, v = 32 * q + lane;
        const uint32_t la = tmem + ((uint32_t)(32 * q) << 16);
        float S[32];
#pragma unroll
        for (int j = 0; j < 32; j++)
            S[j] = a.state_in ? a.state_in[sbase + (size_t)(32 * part + j) * kD + v] : 0.0f;
        auto put_state = [&]() {
#pragma unroll
            for (int b = 0; b < 4; b++) {
                uint32_t hi[4], mid[4];
#pragma unroll
                for (int j = 0; j < 4; j++) split2(S[8 * b + 2 * j], S[8 * b + 2 * j + 1], &hi[j], &mid[j]);
                tmem_st4(la + kTmS + 32 * part + 4 * b, hi);
                tmem_st4(la + kTmS + 32 * part + 16 + 4 * b, mid);
            }
            tmem_wait_st();
            arrive(sh.s_ready);
        };
        put_state();
        for (int c = 0; c < nc; c++) {
            const int n = min(kC, len - kC * c), t0 = 16 * part;
            const int st = c % kChStages;
            const ChunkShared::Scales &sc = sh.sc[c % kChScales];
            // V[t][v] in its swizzled tile
            const uint8_t *vt = sm + (size_t)st * kChStageBytes + kChV + (q >> 1) * kC * 128 + t0 * 128 + (v & 7) * 2;
            const uint32_t v8 = (uint32_t)(v >> 3) & 7u;
            if (!wait(sh.kq_full[st], c / kChStages)) break;
            uint32_t vv[8];                                       // two tokens a word
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t x = *reinterpret_cast<const uint16_t *>(vt + 2 * j * 128 + ((v8 ^ ((2 * j) & 7u)) << 4));
                const uint32_t y = *reinterpret_cast<const uint16_t *>(vt + 2 * j * 128 + 128 + ((v8 ^ ((2 * j + 1) & 7u)) << 4));
                vv[j] = x | (y << 16);
            }
            if (!wait(sh.sc_ready[c % kChScales], c / kChScales) || !wait(sh.d1_full, c)) break;
            tc_fence_after();
            {
                uint32_t d[16];
                tmem_ld16_nowait(la + kTmR + t0, d);
                tmem_wait_ld();
#pragma unroll
                for (int b = 0; b < 2; b++) {
                    uint32_t hi[4], mid[4];
#pragma unroll
                    for (int j2 = 0; j2 < 4; j2++) {
                        const int j = 8 * b + 2 * j2;
                        const float2 kr = *reinterpret_cast<const float2 *>(&sc.kr[t0 + j]);
                        const float x = fmaf(-kr.x, __uint_as_float(d[j]), __uint_as_float(vv[j >> 1] << 16));
                        const float y = fmaf(-kr.y, __uint_as_float(d[j + 1]), __uint_as_float(vv[j >> 1] & 0xFFFF0000u));
                        split2(t0 + j < n ? x : 0.0f, t0 + j + 1 < n ? y : 0.0f, &hi[j2], &mid[j2]);
                    }
                    tmem_st4(la + kTmRU + 8 * part + 4 * b, hi);
                    tmem_st4(la + kTmRU + 32 + 8 * part + 4 * b, mid);
                }
            }
            tmem_wait_st();
            arrive(sh.r_ready);
            if (!wait(sh.d2_full, c)) break;
            tc_fence_after();
            {
                uint32_t d[16];
                tmem_ld16_nowait(la + kTmR + t0, d);
                tmem_wait_ld();
#pragma unroll
                for (int b = 0; b < 2; b++) {
                    uint32_t hi[4], mid[4];
#pragma unroll
                    for (int j2 = 0; j2 < 4; j2++) {
                        const int j = 8 * b + 2 * j2;
                        const float2 kd = *reinterpret_cast<const float2 *>(&sc.kd[t0 + j]);
                        split2(__uint_as_float(d[j]) * kd.x, __uint_as_float(d[j + 1]) * kd.y, &hi[j2], &mid[j2]);
                    }
                    tmem_st4(la + kTmRU + 8 * part + 4 * b, hi);
                    tmem_st4(la + kTmRU + 32 + 8 * part + 4 * b, mid);
#pragma unroll
                    for (int j2 = 0; j2 < 4; j2++)
                        split2(__uint_as_float(d[8 * b + 2 * j2]), __uint_as_float(d[8 * b + 2 * j2 + 1]), &hi[j2], &mid[j2]);
                    tmem_st4(la + kTmU + 8 * part + 4 * b, hi);
                    tmem_st4(la + kTmU + 32 + 8 * part + 4 * b, mid);
                }
            }
            tmem_wait_st();
            arrive(sh.u_ready);
            const float dec = sc.dec;
            if (!wait(sh.d4_full, c)) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; b++) {
                uint32_t d[16];
                tmem_ld16_nowait(la + kTmS + 32 * part + 16 * b, d);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; j++) S[16 * b + j] = fmaf(dec, S[16 * b + j], __uint_as_float(d[j]));
            }
            if (c + 1 < nc) put_state();
        }
        if (!sh.bail)
#pragma unroll
            for (int j = 0; j < 32; j++) a.state_out[sbase + (size_t)(32 * part + j) * kD + v] = S[j];
    } else if (warp < kChWarpMma) {
        // ---------------- O: value column v, every token of the chunk; and the scales
        const int q = warp & 3, v = 32 * q + lane;
        const uint32_t la = tmem + ((uint32_t)(32 * q) << 16);
        // The scales of chunk c, a thread a row of K (0-63) or Q (64-127).
        auto scales = [&](int c) {
            const int n = min(kC, len - kC * c), t = v & (kC - 1), st = c % kChStages;
            const bool is_k = v < kC;
            const size_t tok = (size_t)(first + kC * c);
            float g0 = lane < n ? a.g[(tok + lane) * a.H + h] : 0.0f;
            float g1 = lane + 32 < n ? a.g[(tok + lane + 32) * a.H + h] : 0.0f;
            const float bt = t < n ? a.beta[(tok + t) * a.H + h] : 0.0f;
            g0 = g0 < -200.0f ? -200.0f : g0;
            g1 = g1 < -200.0f ? -200.0f : g1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float p0 = __shfl_up_sync(0xffffffffu, g0, o), p1 = __shfl_up_sync(0xffffffffu, g1, o);
                if (lane >= o) { g0 += p0; g1 += p1; }
            }
            g1 += __shfl_sync(0xffffffffu, g0, 31);
            const float G = (q & 1) ? g1 : g0, GC = __shfl_sync(0xffffffffu, g1, 31);
            if (!wait(sh.kq_full[st], c / kChStages)) return false;
            uint8_t *x = sm + (size_t)st * kChStageBytes + v * 128;
            float norm = 1.0f;
            if (a.qk_norm) {
                float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                for (int j = 0; j < 16; j++) {                // chunk order is the swizzle's: a sum does not mind
                    const uint4 w = *reinterpret_cast<const uint4 *>(x + (j >> 3) * kChBox + (((j & 7) ^ (v & 7)) << 4));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int r = 0; r < 4; r++) {
                        const float lo = __uint_as_float(u[r] << 16), hi = __uint_as_float(u[r] & 0xFFFF0000u);
                        s0 = fmaf(lo, lo, s0);
                        s1 = fmaf(hi, hi, s1);
                    }
                }
                norm = 1.0f / sqrtf(s0 + s1 + a.eps);
            }
            const bool in = t < n;
            if (!in && is_k)                                  // the rows past the sequence's end take no part in K^T U
#pragma unroll
                for (int j = 0; j < 16; j++)
                    *reinterpret_cast<uint4 *>(x + (j >> 3) * kChBox + ((j & 7) << 4)) = make_uint4(0, 0, 0, 0);
            ChunkShared::Scales &sc = sh.sc[c % kChScales];
            const float eG = expf(G);
            if (is_k) {
                sc.g2[t] = G * kLog2e;
                sc.gk[t] = in ? G * kLog2e - log2f(norm) : __int_as_float(0x7f800000);
                sc.beta[t] = bt;
                sc.kb[t] = in ? bt * norm : 0.0f;
                sc.kr[t] = in ? norm * eG : 0.0f;
                sc.kd[t] = in ? norm * expf(GC - G) : 0.0f;
                if (t == 0) sc.dec = expf(GC);
            } else {
                sc.qn[t] = in ? a.scale * norm : 0.0f;
                sc.qr[t] = in ? a.scale * norm * eG : 0.0f;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mb_arrive(&sh.sc_ready[c % kChScales]);
            return true;
        };
        bool ok = scales(0) && (nc < 2 || scales(1));
        for (int c = 0; c < nc && ok; c++) {
            const int n = min(kC, len - kC * c);
            const ChunkShared::Scales &sc = sh.sc[c % kChScales];
            if (!wait(sh.o_full, c)) break;
            tc_fence_after();
            // neighbouring lanes trade a token each: two columns of one token a store
            const int mine = lane & 1;
            uint32_t *o = reinterpret_cast<uint32_t *>(a.out + ((size_t)(first + kC * c + mine) * a.H + h) * kD + (v & ~1));
            const size_t step = (size_t)a.H * kD;             // words of two tokens
#pragma unroll 1
            for (int b = 0; b < 8; b++) {
                uint32_t d[8], p[8];
                tmem_ld8_nowait(la + kTmOq + 8 * b, d);
                tmem_ld8_nowait(la + kTmOp + 8 * b, p);
                tmem_wait_ld();
#pragma unroll
                for (int j4 = 0; j4 < 2; j4++) {
                    const float4 qr = *reinterpret_cast<const float4 *>(&sc.qr[8 * b + 4 * j4]);
                    const float r[4] = {qr.x, qr.y, qr.z, qr.w};
                    float x[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) x[j] = fmaf(r[j], __uint_as_float(d[4 * j4 + j]), __uint_as_float(p[4 * j4 + j]));
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const float got = __shfl_xor_sync(0xffffffffu, mine ? x[2 * j] : x[2 * j + 1], 1);
                        const __nv_bfloat162 w = __floats2bfloat162_rn(mine ? got : x[2 * j], mine ? x[2 * j + 1] : got);
                        if (8 * b + 4 * j4 + 2 * j + mine < n) *o = *reinterpret_cast<const uint32_t *>(&w);
                        o += step;
                    }
                }
            }
            arrive(sh.o_free);
            if (c + 2 < nc) ok = scales(c + 2);
        }
    } else if (warp == kChWarpMma) {
        // ---------------- loads and MMA issue
        const uint32_t idk = idesc(1, kC);                     // 128 x 64, both operands K-major
        const uint32_t idn = idk | (1u << 16);                 // B with N contiguous (K^T U: channels)
        const uint32_t aT = saddr(tT), aP = saddr(tP);
        // K K^T and Q K^T of chunk c: rows of K over rows of Q, against K
        auto kk = [&](int c) {
            const uint32_t b = saddr(sm + (size_t)(c % kChStages) * kChStageBytes);
            const uint64_t bd = sdesc(b);
#pragma unroll
            for (int s = 0; s < 8; s++) {
                const uint64_t at = bd + (((s >> 2) * kChBox + (s & 3) * 32) >> 4);
                umma_warp(kTmKK, at, at, idk, s > 0);
            }
        };
        // D[v][t >= 16 j] += X[v][16 tokens j] tile[t][16 tokens j], the tile lower triangular:
        // the terms of X at columns `x`, of the tile kChTile apart
        auto tri = [&](uint32_t d, uint32_t x, uint32_t tile) {
            const uint64_t td = sdesc(tile);
#pragma unroll
            for (int term = 0; term < 3; term++)               // hi hi, hi mid, mid hi
#pragma unroll
                for (int j = 0; j < 4; j++)
                    umma_ts_warp(d + 16 * j, x + (term == 2 ? 32 : 0) + 8 * j,
                            td + (((term == 1 ? kChTile : 0) + 16 * j * 128 + j * 32) >> 4), idesc(1, kC - 16 * j),
                            term > 0 || j > 0);
        };
        auto load = [&](int c) {
            uint8_t *p = sm + (size_t)(c % kChStages) * kChStageBytes;
            uint64_t *bar = &sh.kq_full[c % kChStages];
            mb_expect_tx(bar, kChStageBytes);
            for (int b = 0; b < 2; b++) {
                tma2d(p + b * kChBox, &mk, hq * kD + 64 * b, first + kC * c, bar);
                tma2d(p + b * kChBox + kC * 128, &mq, hq * kD + 64 * b, first + kC * c, bar);
                tma2d(p + kChV + b * kC * 128, &mv, h * kD + 64 * b, first + kC * c, bar);
            }
        };
        if (lane == 0)
            for (int c = 0; c < min(nc, 2); c++) load(c);
        __syncwarp();
        bool ok = wait(sh.kq_full[0], 0);
        if (ok) {
            kk(0);
            umma_commit_warp(&sh.kk_full);
        }
        for (int c = 0; c < nc && ok; c++) {
            const uint64_t kq = sdesc(saddr(sm + (size_t)(c % kChStages) * kChStageBytes));
            if (!wait(sh.s_ready, c)) break;
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 16; s++)                       // K S, hi and mid
                umma_ts_warp(kTmR, kTmS + 32 * ((s >> 1) & 3) + 16 * (s >> 3) + 8 * (s & 1),
                             kq + ((((s >> 2) & 1) * kChBox + (s & 3) * 32) >> 4), idk, s > 0);
            umma_commit_warp(&sh.d1_full);
            if (c + 1 < nc) {
                // the wait for chunk c - 1's O lets the preparation of chunk c + 1 write over that chunk's scales and P
                if (!wait(sh.kq_full[(c + 1) % kChStages], (c + 1) / kChStages) || !wait(sh.kk_free, c) ||
                    (c >= 1 && !wait(sh.o_free, c - 1)))
                    break;
                tc_fence_after();
                kk(c + 1);
                umma_commit_warp(&sh.kk_full);
            }
            if (c + 2 < nc && lane == 0) load(c + 2);          // chunk c - 1 is done with its stage: its state was here
            __syncwarp();
            if (!wait(sh.tp_ready, c) || !wait(sh.r_ready, c)) break;
            tc_fence_after();
            tri(kTmR, kTmRU, aT);
            umma_commit_warp(&sh.d2_full);
            if (c >= 1 && c + 1 == nc && !wait(sh.o_free, c - 1)) break;   // the last chunk has not waited above
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 16; s++)                       // Q S
                umma_ts_warp(kTmOq, kTmS + 32 * ((s >> 1) & 3) + 16 * (s >> 3) + 8 * (s & 1),
                             kq + ((((s >> 2) & 1) * kChBox + kC * 128 + (s & 3) * 32) >> 4), idk, s > 0);
            if (!wait(sh.u_ready, c)) break;
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 16; s++)                       // K^T U into the state's sums, a half of k at a time
                umma_ts_warp(kTmS + 64 * (s >> 3), kTmRU + 32 * ((s >> 2) & 1) + 8 * (s & 3),
                             kq + (((s >> 3) * kChBox + (s & 3) * 16 * 128) >> 4), idn, (s & 7) > 0);
            umma_commit_warp(&sh.d4_full);
            tri(kTmOp, kTmU, aP + (c & 1) * 2 * kChTile);
            umma_commit_warp(&sh.o_full);
        }
        __syncwarp();
        umma_commit_warp(&sh.drain);                           // every issued MMA done before the dealloc
        mb_wait_warp(&sh.drain, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kChWarpMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(512));
}

}  // namespace

size_t delta_workspace(const k3moe_delta_config &dc, int n_seq, int T)
{
    (void)dc;
    (void)n_seq;
    (void)T;
    return kCtrOffset + kCtrBytes;
}

static cudaError_t launch_chunks(const DeltaArgs &a, cudaStream_t s)
{
    CUtensorMap mq{}, mk{}, mv{};
    const uint64_t cols = (uint64_t)a.Hq * kD;
    if (!map16s(&mq, a.q, (uint64_t)a.T, cols, (uint64_t)a.q_stride, kC) ||
        !map16s(&mk, a.k, (uint64_t)a.T, cols, (uint64_t)a.k_stride, kC) ||
        !map16s(&mv, a.v, (uint64_t)a.T, (uint64_t)a.H * kD, (uint64_t)a.v_stride, kC))
        return cudaErrorInvalidValue;
    static bool smem_set = false;
    if (!smem_set) {
        cudaFuncSetAttribute(delta_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kChSmem);
        smem_set = true;
    }
    timing_begin("delta_chunk", s);
    const cudaError_t err =
        launch_pdl(delta_chunk_kernel, dim3((unsigned)(a.n_seq * a.H)), dim3(kChThreads), kChSmem, s, a, mq, mk, mv);
    count_launch();
    timing_end("delta_chunk", s);
    return err;
}

cudaError_t launch_delta(const DeltaArgs &a, cudaStream_t s)
{
    if (a.gate == 1 && a.T >= 24 * a.n_seq) return launch_chunks(a, s);
    // one block per head while they fill the GPU twice over; else 32 columns a block
    const long long blocks = (long long)a.n_seq * a.H;
    timing_begin("delta_recurrent", s);
    const cudaError_t err = blocks >= 2 * 152
        ? launch_pdl(delta_recurrent_kernel<128>, dim3((unsigned)blocks), dim3(kRecThreads), 0, s, a)
        : launch_pdl(delta_recurrent_kernel<32>, dim3((unsigned)blocks * 4), dim3(kRecThreads), 0, s, a);
    count_launch();
    timing_end("delta_recurrent", s);
    return err;
}

}  // namespace k3moe
