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
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"

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

}  // namespace

size_t delta_workspace(const k3moe_delta_config &dc, int n_seq, int T)
{
    (void)dc;
    (void)n_seq;
    (void)T;
    return kCtrOffset + kCtrBytes;
}

cudaError_t launch_delta(const DeltaArgs &a, cudaStream_t s)
{
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
