// k3moe_attend.cu -- latent attention in the absorbed form: every query head attends the same
// cached rows [c, r] of 576 columns, whose first 512 are the values too.
//
// A block has up to 64 query rows (heads of one token, or of a few) of one sequence and walks cached rows in tiles
// of 64.  Scores are taken transposed, S^T [row of the cache][query] = cache Q^T, so that the tile is the A operand whatever
// the number of heads, and the outputs likewise, O^T [c][query] += C^T P^T with the same tile in shared memory read along
// c.  Softmax in powers of two as in the expanded form; a query's maximum moves only when it is outdone by 2^8, so that a
// tile mostly needs no more than a vote.
//
// Bound by the cache's bytes: 1152 a row against 64 x 2176 flops.  A tile is 72 KB, and beside the queries (72 KB) there is
// room for two: with tiles of 128 rows nothing could be loaded under a tile's softmax, all SMs loaded and computed in
// step, and the DRAM was idle half of the time (96 sequences: 158 us).  All tiles of all sequences are one line that is cut
// into as many even parts as there are SMs; a query block that a cut goes through leaves its parts' sums (float) in the
// workspace, and a second kernel joins them.
//
// Measured, both kernels, 56 heads: 96 tokens of up to 8192 rows 99.5 us (489 MB: 4.9 TB/s over all, 5.6 in the middle), one token of
// 131071 rows 42.8 (26 of them loads), of 777 rows 12.1 (every step's latency once).  40 drafted tokens of 11 sequences,
// 16 heads, pages of 16: 24.2; with cuts that count nothing ahead of a query block some SMs had four of its starts (29.4
// against 27.0 then).  A tile is in its place for about 8000 clocks: 4300 until its first boxes have landed, 700 to 2400 of scores,
// 900 of weights, 250 to 1100 of outputs.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>

#include "k3moe_internal.cuh"
#include "k3moe_latent.cuh"

namespace k3moe {
namespace {

constexpr int kAtRows = 64, kAtTile = 64;                     // queries of a block, cached rows of a tile
constexpr int kAtBoxes = kLatRow / 64;                        // 64-column boxes of a tile: c's eight, then r's
constexpr int kAtBox = kAtTile * 128;                         // 8 KB
constexpr int kAtSlots = 2 * kAtBoxes;                        // c of even and of odd tiles, then r of both
// Boxes of c are loaded, waited for and freed in pairs, the first with r: the scores of what has landed are taken while the rest
// is on its way, and the next tile but one is asked for pair by pair as the outputs get done
constexpr int kAtPairs = kLatC / 128;
constexpr int kAtQBox = kAtRows * 128;
constexpr int kAtQ = kAtBoxes * kAtQBox, kAtP = kAtTile * kAtRows * 2;
constexpr int kAtSmem = 1024 + kAtQ + kAtP + kAtSlots * kAtBox;
// Warps: two groups of four share the softmax (32 queries each), two issue the products, scores and outputs, and two the
// cache's loads, of half of c each and r
constexpr int kAtThreads = 384, kAtWarpS = 8, kAtWarpV = 9, kAtWarpLoad = 10;
constexpr uint32_t kAtTmS = 0, kAtTmO = 128;                  // S^T of two tiles, and O^T in four blocks of 128 of c
constexpr float kAtSlack = 8.0f;
// A query block's queries, first product and output take about as long as this many tiles: the cuts count it so
constexpr int kAtAhead = 2;

// A part's sums in the workspace: O [query][c], then the maxima and the sums of the weights.
constexpr size_t kAtPart = kLatPart;
// A query block that cuts leave to join: its first part is share `first`'s last (its first or second), the others are the
// first ones of the shares after it.  Each share writes down the one that begins in it and the one that goes on there.
struct AttendJoin {
    int t0, row0, rows, first, second, parts;                 // rows = 0: none
};

// Sequence i: its queries, cached rows, blocks of 1 << shift queries and tiles of each; false when something does not fit.
struct AttendSeq {
    int t0, n, len, blocks, tiles, each;                      // units of a query block: what comes ahead of its tiles, and they
    __device__ bool set(const AttendArgs &a, int from, int to, int kv, int shift)
    {
        t0 = from;
        n = to - from;
        len = kv;
        const bool ok = from >= 0 && to >= from && to <= a.T && len >= 0 && len <= a.max_pages << a.page_shift;
        blocks = ok ? (n * a.H + (1 << shift) - 1) >> shift : 0;
        tiles = max(1, (len + kAtTile - 1) / kAtTile);        // one that has nothing where no row is cached
        each = a.whole ? 1 : kAtAhead + tiles;
        return ok;
    }
    __device__ static int start(const AttendArgs &a, int i)
    {
        return a.seq_start ? a.seq_start[i] : a.n_seq == 1 ? i * a.T : i;
    }
    __device__ bool read(const AttendArgs &a, int i, int shift) { return set(a, start(a, i), start(a, i + 1), a.kv_len[i], shift); }
};

// The walk of a block's share of units, query block by query block.
template <typename I> struct AttendWalk {
    I u, end, base;                                           // next unit, the share's end, the sequence's first unit
    int seq, shift;
    AttendSeq s;
    int row0, tile0, tile1;                                   // the query block and its tiles here
    __device__ bool next(const AttendArgs &a)
    {
        if (u >= end) return false;
        while (u >= base + (I)s.blocks * s.each) {
            base += (I)s.blocks * s.each;
            s.read(a, ++seq, shift);
        }
        const I at = u - base;
        const int block = (int)quotient(at, s.each), from = (int)(at - (I)block * s.each), to = (int)min((I)s.each, from + (end - u));
        row0 = block << shift;
        tile0 = a.whole ? 0 : max(0, from - kAtAhead);
        tile1 = a.whole ? s.tiles : max(0, to - kAtAhead);
        u += to - from;
        return tile1 > 0;                                     // a share that ends ahead of the first tile leaves the block to the next
    }
    __device__ I unit(int tile) const { return base + (I)(row0 >> shift) * s.each + kAtAhead + tile; }
    __device__ int rows(const AttendArgs &a) const { return min(1 << shift, s.n * a.H - row0); }
    __device__ bool whole() const { return tile0 == 0 && tile1 == s.tiles; }
};

// Even shares of all units, the first `more` of them a unit longer; where there are fewer than shares the last are empty.
template <typename I> struct AttendShares {
    I each, more;
    __device__ void cut(I all, int n)
    {
        each = quotient(all, n);
        more = all - each * n;
    }
    __device__ I begin(int i) const { return i * each + min((I)i, more); }
    __device__ int of(I unit) const                           // the share that has it
    {
        return (int)(unit < more * (each + 1) ? unit / (each + 1) : more + (unit - more * (each + 1)) / each);
    }
};

template <typename I> struct AttendShared {
    uint64_t q_full, full[2][kAtPairs], empty[2][kAtPairs], r_empty[2], s_full[2], p_ready[2], pv_done, drain[2];    // by the tile's turn, pairs of c's boxes
    uint32_t tmem;
    volatile int bail;
    int spoiled[2];                                           // by the query block's turn
    union {                                                   // (one after the other)
        struct {
            UnitSearch<I> search;
            AttendWalk<I> walk;
            AttendShares<I> shares;
            int have;
        } first;
        float top[2][4][32], sum[2][4][32];
    };
    float m[kAtRows];
    union {
        float f[kAtRows], inv[kAtRows];
    };
    int lim[2][32];
};
static_assert(sizeof(AttendShared<long long>) <= 2048 && kAtSmem + 2048 <= 227 * 1024, "an SM's shared memory");

// The block's share and its first query block, into shared memory.  Up to 128 sequences are one warp's, four a lane, and with few
// tiles the query blocks get smaller, so that more SMs have one.
constexpr int kAtPlanSeqs = 128;
template <typename I> __device__ __forceinline__ void attend_plan(const AttendArgs &a, AttendShared<I> &sh, int32_t *status)
{
    const int lane = threadIdx.x & 31;
    AttendShares<I> shares;
    AttendWalk<I> w;
    w.shift = 6;
    bool mine = false;                                        // this thread has found the share's first tile
    I before = 0;
    if (a.n_seq <= kAtPlanSeqs) {
        int from[5], kv[4];                                   // all asked for before any is looked at
#pragma unroll
        for (int k = 0; k < 5; k++) {
            const int i = 4 * lane + k;
            from[k] = i <= a.n_seq ? AttendSeq::start(a, i) : 0;
            if (k < 4) kv[k] = i < a.n_seq ? a.kv_len[i] : 0;
        }
        AttendSeq s[4];
        bool bad = false;
        I all = 0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            s[k].blocks = 0;
            if (4 * lane + k < a.n_seq) bad = !s[k].set(a, from[k], from[k + 1], kv[k], 6) || bad;
            all += s[k].blocks ? (I)s[k].blocks * (a.whole ? 1 : s[k].tiles) : 0;
        }
        if (bad) set_status(status, K3MOE_DEV_BAD_OFFSETS);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        const int n = gridDim.x;
        if (all <= n / 2) w.shift = all <= n / 4 ? 4 : 5;
        I units[4], each = 0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            if (s[k].blocks) s[k].blocks = (s[k].n * a.H + (1 << w.shift) - 1) >> w.shift;
            each += units[k] = s[k].blocks ? (I)s[k].blocks * s[k].each : 0;
        }
        const I upto = warp_scan(each, lane);
        shares.cut(__shfl_sync(0xffffffffu, upto, 31), gridDim.x);
        w.u = shares.begin(blockIdx.x);
        before = w.u - (upto - each);
        mine = before >= 0 && before < each;
        w.seq = 4 * lane;
        w.s = s[0];
#pragma unroll
        for (int k = 0; k < 3; k++)
            if (mine && w.seq == 4 * lane + k && before >= units[k]) {
                before -= units[k];
                w.seq++;
                w.s = s[k + 1];
            }
    } else {
        I all;
        w.seq = find_unit<kAtThreads, I>(
            sh.first.search, a.n_seq, &before, &all,
            [&](int i) -> I {
                AttendSeq s;
                if (!s.read(a, i, 6)) set_status(status, K3MOE_DEV_BAD_OFFSETS);
                return (I)s.blocks * s.each;
            },
            [&](I all) {
                shares.cut(all, gridDim.x);
                return shares.begin(blockIdx.x);
            });
        w.u = shares.begin(blockIdx.x);
        mine = w.seq >= 0 && threadIdx.x == 0;
    }
    w.end = shares.begin(blockIdx.x + 1);
    if (w.u >= w.end) {
        if ((threadIdx.x & 31) == 0) sh.first.have = 0;
        return;
    }
    if (!mine) return;
    w.base = w.u - before;
    if (a.n_seq > kAtPlanSeqs) w.s.read(a, w.seq, w.shift);
    const bool any = w.next(a);
    if (any) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.pages + (size_t)w.seq * a.max_pages + min(kAtTile * w.tile0 >> a.page_shift, a.max_pages - 1)));
    sh.first.have = any;
    sh.first.walk = w;
    sh.first.shares = shares;
}

static_assert(2 * sizeof(AttendJoin) * kMaxShares <= kLatJoinBytes && kAtRows == 64, "as the workspace is laid out");

// S^T's 16 lanes of a warp, 32 columns: v[4 k + 2 i + j] is row lane / 4 + 8 i, column 8 k + 2 (lane % 4) + j.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Over the lanes that have the same columns: eight values each.
template <typename F> __device__ __forceinline__ void over_rows(float (&v)[8], F f)
{
#pragma unroll
    for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = f(v[j], __shfl_xor_sync(0xffffffffu, v[j], o));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }
__device__ __forceinline__ bool group_any(int group, bool p)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)p), "r"(1 + group)
        : "memory");
    return r != 0;
}
template <typename I>
__global__ void __launch_bounds__(kAtThreads, 1)
    attend_kernel(const AttendArgs a, const __grid_constant__ CUtensorMap m2, const __grid_constant__ CUtensorMap m1, float *parts, AttendJoin *joins)
{
    extern __shared__ __align__(1024) uint8_t asm_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(asm_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sm_p = sm + kAtQ, *ring = sm_p + kAtP;
    __shared__ AttendShared<I> sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *status = reinterpret_cast<int32_t *>(a.ws);
    if (threadIdx.x == 0) {
        mb_init(&sh.q_full, 8);
        for (int i = 0; i < 2; i++) {
            for (int j = 0; j < kAtPairs; j++) {
                mb_init(&sh.full[i][j], 1);
                mb_init(&sh.empty[i][j], 1);
            }
            mb_init(&sh.r_empty[i], 1);
            mb_init(&sh.s_full[i], 1);
            mb_init(&sh.p_ready[i], 8);
            mb_init(&sh.drain[i], 1);
        }
        mb_init(&sh.pv_done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.bail = 0;
        sh.spoiled[0] = sh.spoiled[1] = 0;
        prefetch_map(&m2);
        prefetch_map(&m1);
    }
    pdl_wait();
    pdl_trigger();
    if (warp == kAtWarpS) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sh.tmem)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (a.n_seq > kAtPlanSeqs || warp == kAtWarpLoad) attend_plan<I>(a, sh, status);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const bool have = sh.first.have;
    AttendWalk<I> w = sh.first.walk;
    const AttendShares<I> shares = sh.first.shares;
    const int shift = w.shift;
    __syncthreads();                                          // what is read here is written over by the softmax
    if (!have) {
        if (threadIdx.x < 2) joins[2 * blockIdx.x + threadIdx.x].rows = 0;
        if (warp == kAtWarpS) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(512));
        return;
    }
    constexpr uint32_t tmem = 0;                              // all 512 columns: the allocation starts at the first
    auto wait = [&](uint64_t &b, int phase) { return role_wait(&b, phase, status, &sh.bail); };
    // the same for the warps that meet at barriers: after a wait that gave up they go on without waiting, to the end
    auto go_on = [&](uint64_t &b, int phase) { return !sh.bail && wait(b, phase); };

    if (warp < kAtWarpS) {
        // ---------------- queries, softmax and output: cached rows 16 q + lane / 4 and 8 more of a tile, queries 32 g ..
        const int g = warp >> 2, q = warp & 3, row = 16 * q + (lane >> 2), col = 2 * (lane & 3);
        const uint32_t la = tmem + ((uint32_t)(32 * q) << 16);
        const float c = a.scale * kLatLog2e;
        // the next query block's rows, in the order the tensor core reads: 64 columns of 64 rows a box, 128-byte swizzle
        auto load_q = [&]() {
            const int r = threadIdx.x >> 2, rows = w.rows(a), gr = w.row0 + (r < rows ? r : 0);
            if (r >= 1 << shift) return;
            const uint16_t *src = a.q + (size_t)(w.s.t0 + gr / a.H) * a.q_stride + (size_t)(gr % a.H) * a.q_head;
            const uint32_t dst = saddr(sm) + (uint32_t)(r * 128);
#pragma unroll
            for (int j = 0; j < kLatRow / 8 / 4; j++) {
                const int x = 4 * j + (threadIdx.x & 3);
                cp_async16(dst + (uint32_t)((x >> 3) * kAtQBox + (((x & 7) ^ (r & 7)) << 4)), src + 8 * x, r < rows);
            }
        };
        auto q_loaded = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mb_arrive(&sh.q_full);
        };
        int tile = 0;                                         // so far
        bool more = true;
        load_q();
        q_loaded();
        const bool idle = 32 * g >= 1 << shift;               // no query of this group's
        for (int seg = 0; more; seg++) {
            const AttendWalk<I> now = w;
            const int rows = w.rows(a);
            // rows of the cache that each query sees
            auto limit = [&](int r) { return a.causal ? max(0, now.s.len - (now.s.n - 1 - (now.row0 + r) / a.H)) : now.s.len; };
            const int least = limit(0);                       // of all its queries
            int *lim = sh.lim[g];
            if (q == 0) lim[lane] = 32 * g + lane < rows ? limit(32 * g + lane) : 0;
            float m[8], l[8];                                 // maxima (minus; 0 where there is none) and sums of columns 8 k + col, + 1
#pragma unroll
            for (int j = 0; j < 8; j++) m[j] = l[j] = 0.0f;
            if (q == 0) sh.m[32 * g + lane] = 32 * g + lane < rows ? -INFINITY : 0.0f;
            group_sync(g);
            // none: a query of this thread's columns has had no score above minus infinity yet, so that its weights' exponents are
            // not of a maximum; one is looked for tile by tile until it has (rows of the cache whose scores are infinite may come first)
            bool first = true, none = true;
            for (int t = now.tile0; t < now.tile1; t++, tile++) {
                go_on(sh.s_full[tile & 1], tile >> 1);
                tc_fence_after();
                uint32_t u[16];
                tmem_ld_16x256(la + kAtTmS + 64 * (tile & 1) + 32 * g, u);
                float v[16];
                const int at = kAtTile * t + row;             // of the sequence's rows
#pragma unroll
                for (int j = 0; j < 16; j++) v[j] = fmaf(__uint_as_float(u[j]), c, m[(j >> 2) * 2 + (j & 1)]);     // the weights' exponents
                if (kAtTile * (t + 1) > least)
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        const int see = lim[8 * (j >> 2) + col + (j & 1)];
                        v[j] = at + 4 * (j & 2) < see ? v[j] : -INFINITY;
                    }
                if (idle || shift == 4)                       // columns that no product has written
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (idle || j >= 8) v[j] = -INFINITY;
                const bool free = role_done(sh.pv_done, tile - 1);      // asked ahead of where it is needed
                float over = v[0];
#pragma unroll
                for (int j = 1; j < 15; j += 2) over = max3(over, v[j], v[j + 1]);
                over = fmaxf(over, v[15]);
                if (group_any(g, none || over > kAtSlack)) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; j++) x[j] = fmaxf(v[4 * (j >> 1) + (j & 1)], v[4 * (j >> 1) + 2 + (j & 1)]) - m[j];
                    over_rows(x, [](float p, float r) { return fmaxf(p, r); });
                    if (lane < 4)
#pragma unroll
                        for (int j = 0; j < 8; j++) sh.top[g][q][8 * (j >> 1) + col + (j & 1)] = x[j];
                    group_sync(g);
                    if (q == 0) {                             // lane j query j's
                        const float all = fmaxf(fmaxf(sh.top[g][0][lane], sh.top[g][1][lane]), fmaxf(sh.top[g][2][lane], sh.top[g][3][lane]));
                        const float m0 = sh.m[32 * g + lane], m1 = all > m0 + kAtSlack ? all : m0;
                        sh.m[32 * g + lane] = m1;
                        sh.f[32 * g + lane] = m1 == -INFINITY || first ? 1.0f : exp2_fast(m0 - m1);
                    }
                    group_sync(g);
                    none = false;
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const int at = 32 * g + 8 * (j >> 1) + col + (j & 1);
                        const bool has = sh.m[at] != -INFINITY;
                        const float to = has ? -sh.m[at] : 0.0f, by = to - m[j];
                        none = none || !has;
                        m[j] = to;
                        l[j] *= sh.f[at];
                        v[4 * (j >> 1) + (j & 1)] += by;
                        v[4 * (j >> 1) + 2 + (j & 1)] += by;
                    }
                    if (!first) {
                        go_on(sh.pv_done, tile - 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int b = 0; b < 8; b++) {
                            const uint32_t o_at = la + kAtTmO + 64 * (b >> 1) + 32 * g + 16 * (b & 1);
                            float o[16];
                            tmem_ld16(o_at, o);
#pragma unroll
                            for (int j = 0; j < 16; j++) o[j] *= sh.f[32 * g + 16 * (b & 1) + j];
                            tmem_st16(o_at, o);
                        }
                        tmem_wait_st();
                    }
                }
                first = false;
                // the sums are of the weights in float; the product takes them in bf16, as it takes c, each off by 2^-8 of itself at most
                uint32_t p[8];
#pragma unroll
                for (int k = 0; k < 4; k++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float x = exp2_fast(v[4 * k + 2 * i]), y = exp2_fast(v[4 * k + 2 * i + 1]);
                        l[2 * k] += x;
                        l[2 * k + 1] += y;
                        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
                        p[2 * k + i] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                // a row's weights of 64 queries are 128 bytes of P, 128-byte swizzle; the product before has read its own
                if (!__all_sync(0xffffffffu, free)) go_on(sh.pv_done, tile - 1);
#pragma unroll
                for (int k = 0; k < 4; k++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const int r = row + 8 * i;
                        *reinterpret_cast<uint32_t *>(sm_p + r * 128 + (((4 * g + k) ^ (r & 7)) << 4) + 2 * col) = p[2 * k + i];
                    }
                if (kAtTile * (t + 1) > least) {
                    // rows behind the last are cleared, and of rows that some query does not see what is infinite or NaN: a
                    // weight of zero would not keep it out (queries that see it add it at the end)
                    const int r = threadIdx.x & 63, at = kAtTile * t + r;
                    bool any = false;
                    if (at >= least)
#pragma unroll 1
                        for (int n = 0; n < 2; n++) {
                            const int b = 8 * (tile & 1) + 2 * (threadIdx.x >> 6) + n;
                            uint4 *x = reinterpret_cast<uint4 *>(ring + b * kAtBox + r * 128);
#pragma unroll 1
                            for (int j = 0; j < 8; j++) {
                                uint4 y = x[j];
                                if (at >= now.s.len) {
                                    x[j] = make_uint4(0, 0, 0, 0);
                                } else if (clear_spoiled(y)) {
                                    x[j] = y;
                                    any = true;
                                }
                            }
                        }
                    if (any) atomicOr(&sh.spoiled[seg & 1], 1);
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mb_arrive(&sh.p_ready[tile & 1]);
            }
            // the last scores are there: the queries' place is free for the next block's
            more = w.next(a);
            if (more) load_q();
            over_rows(l, [](float x, float y) { return x + y; });
            if (lane < 4)
#pragma unroll
                for (int j = 0; j < 8; j++) sh.sum[g][q][8 * (j >> 1) + col + (j & 1)] = l[j];
            group_sync(g);
            const bool whole = now.whole();
            // a share's first query block leaves its part in the block's first place, a later one in the second
            float *part = parts + (size_t)(2 * blockIdx.x + (seg > 0)) * kAtPart;
            if (q == 0) {
                const int mine = 32 * g + lane;
                const float sum = (sh.sum[g][0][lane] + sh.sum[g][1][lane]) + (sh.sum[g][2][lane] + sh.sum[g][3][lane]);
                sh.inv[mine] = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
                if (!whole) {
                    part[kAtRows * kLatC + mine] = isnan(sum) && sh.m[mine] == -INFINITY ? 0.0f : sh.m[mine];    // not one without keys
                    part[kAtRows * kLatC + kAtRows + mine] = sum;
                } else if (a.lse && mine < rows) {
                    a.lse[(size_t)now.s.t0 * a.H + now.row0 + mine] = (sh.m[mine] + log2f(sum)) * kLatLn2;
                }
            }
            if (more) q_loaded();
            group_sync(g);
            const bool ok = go_on(sh.pv_done, tile - 1);
            tc_fence_after();
            const bool spoiled = *const_cast<volatile int *>(&sh.spoiled[seg & 1]) != 0;
            const int count = ok ? min(32, rows - 32 * g) : 0;
            // 16 queries at a time, a thread four columns of c
#pragma unroll 1
            for (int b = 0; b < 2; b++) {
                const int r0 = 32 * g + 16 * b, left = min(16, count - 16 * b);
                if (left <= 0) break;
                uint32_t o[4][16];
#pragma unroll
                for (int k = 0; k < 4; k++) tmem_ld16_nowait(la + kAtTmO + 64 * k + r0, o[k]);
                tmem_wait_ld();
                if (spoiled)
#pragma unroll 1
                    for (int at = max(least, kAtTile * now.tile0); at < min(now.s.len, kAtTile * now.tile1); at++) {
                        const int page = a.pages[(size_t)now.seq * a.max_pages + (at >> a.page_shift)];
                        if (page < 0 || page >= a.n_pages) continue;
                        const uint16_t *from = a.cache + ((size_t)page * a.page + (at & (a.page - 1))) * kLatRow + 32 * q + lane;
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const uint32_t x = from[128 * k];
                            if ((x & 0x7F80u) != 0x7F80u) continue;
#pragma unroll
                            for (int j = 0; j < 16; j++)
                                if (at < lim[16 * b + j]) o[k][j] = __float_as_uint(__uint_as_float(o[k][j]) + bf16_bits_to_f32(x));
                        }
                    }
                if (whole) {
                    __nv_bfloat16 *to = reinterpret_cast<__nv_bfloat16 *>(a.out) + ((size_t)now.s.t0 * a.H + now.row0 + r0) * kLatC + 32 * q + lane;
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        const float inv = sh.inv[r0 + j];
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            if (j < left) to[j * kLatC + 128 * k] = __float2bfloat16_rn(inv == 0.0f ? 0.0f : __uint_as_float(o[k][j]) * inv);
                    }
                } else {
                    uint32_t *to = reinterpret_cast<uint32_t *>(part) + (size_t)r0 * kLatC + 32 * q + lane;
#pragma unroll
                    for (int j = 0; j < 16; j++)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            if (j < left) to[j * kLatC + 128 * k] = o[k][j];
                }
            }
            tc_fence_before();                                // the next query block's first product is after its weights
            // the next query block has its flag cleared, and both groups are done with this one
            if (threadIdx.x == 0) sh.spoiled[~seg & 1] = 0;
            asm volatile("bar.sync 3, 256;" ::: "memory");
        }
    } else if (warp == kAtWarpS) {
        // ---------------- scores, a tile ahead of the products with c where its boxes have landed
        const uint32_t id = (idesc(1, 1 << uniform(shift)) & ~(31u << 24)) | (4u << 24);              // M = 64 rows of the cache
        const uint32_t q0 = desc_lo(saddr(sm)), c0 = desc_lo(saddr(ring));
        constexpr uint32_t box = kAtBox >> 4, q_box = kAtQBox >> 4;
        int tile = 0;
        bool ok = true;
        for (int seg = 0; ok && (seg == 0 || w.next(a)); seg++) {
            if (!(ok = wait(sh.q_full, seg))) break;
            const int n = uniform(w.tile1 - w.tile0);
#pragma unroll 1
            for (int t = 0; t < n; t++, tile++) {
                const uint32_t turn = (uint32_t)uniform(tile & 1), D = kAtTmS + 64 * turn;
                // the weights of the tile before the last are made of what was here
                if (tile >= 2 && !(ok = wait(sh.p_ready[turn], (tile >> 1) - 1))) break;
                auto product = [&](uint32_t A, uint32_t B, bool first) {
#pragma unroll
                    for (int k = 0; k < 4; k++) umma_warp(D, A + 2 * k, B + 2 * k, id, !first || k > 0);
                };
                bool there = false;                           // looked for under the products before
#pragma unroll
                for (int j = 0; j < kAtPairs; j++) {
                    if (!__all_sync(0xffffffffu, there) && !(ok = wait(sh.full[turn][j], tile >> 1))) break;
                    if (j == 0) tc_fence_after();
                    there = j + 1 < kAtPairs && role_done(sh.full[turn][j + 1], tile >> 1);
                    if (j == 0) {
                        product(c0 + (16 + turn) * box, q0 + 8 * q_box, true);
                        umma_commit_warp(&sh.r_empty[turn]);
                    }
                    product(c0 + (8 * turn + 2 * j) * box, q0 + 2 * j * q_box, false);
                    product(c0 + (8 * turn + 2 * j + 1) * box, q0 + (2 * j + 1) * q_box, false);
                }
                if (!ok) break;
                umma_commit_warp(&sh.s_full[turn]);
            }
        }
        __syncwarp();
        umma_commit_warp(&sh.drain[0]);                        // every issued MMA done before the dealloc
        mb_wait_warp(&sh.drain[0], 0);
    } else if (warp == kAtWarpV) {
        // ---------------- products of the weights with c
        const uint32_t id = idesc(1, 1 << uniform(shift)) | (1u << 15) | (1u << 16);                  // both with M, N contiguous
        const uint32_t p0 = desc_lo(saddr(sm_p)), c0 = desc_lo(saddr(ring), kAtBox);
        constexpr uint32_t box = kAtBox >> 4;
        int tile = 0;
        bool ok = true;
        for (bool more = true; ok && more; more = ok && w.next(a)) {
            const int n = uniform(w.tile1 - w.tile0);
#pragma unroll 1
            for (int t = 0; t < n; t++, tile++) {
                const uint32_t turn = (uint32_t)uniform(tile & 1);
                if (!(ok = wait(sh.p_ready[turn], tile >> 1))) break;
                tc_fence_after();
                const uint32_t A = c0 + 8 * turn * box;
#pragma unroll 1
                for (int b = 0; b < kAtPairs; b++) {
#pragma unroll
                    for (int k = 0; k < kAtTile / 16; k++)
                        umma_warp(kAtTmO + 64 * b, A + 2 * b * box + (uint32_t)(k * 16 * 128 >> 4), p0 + (uint32_t)(k * 16 * 128 >> 4), id, t > 0 || k > 0);
                    umma_commit_warp(&sh.empty[turn][b]);
                }
                umma_commit_warp(&sh.pv_done);
            }
        }
        __syncwarp();
        umma_commit_warp(&sh.drain[1]);
        mb_wait_warp(&sh.drain[1], 0);
    } else {
        // ---------------- the cache's rows: every other pair of boxes of c, of a page's rows each, a lane a page; the first warp loads r
        const int box_rows = min(a.page, kAtTile), pieces = kAtTile >> min(a.page_shift, 6), half = uniform(warp - kAtWarpLoad);
        int tile = 0;
        bool ok = true;
        int asked = 0;                                        // pairs, two of a tile
        if (half == 0 && lane < 2) joins[2 * blockIdx.x + lane].rows = 0;
        __syncwarp();
        for (int seg = 0; ok && (seg == 0 || w.next(a)); seg++) {
            const int begun = w.tile0, left = w.s.tiles - w.tile1;
            const int n_tiles = uniform(w.tile1 - w.tile0), len = w.s.len, tile0 = w.tile0;
            const int32_t *pages = a.pages + (size_t)w.seq * a.max_pages;
#pragma unroll 1
            for (int t = 0; t < n_tiles; t++, tile++) {
                const int at = kAtTile * (tile0 + t) + lane * box_rows, turn = uniform(tile & 1), phase = tile >> 1;
                int row = -1;                                 // nothing to load
                if (lane < pieces && at < len) {
                    const int page = pages[at >> a.page_shift];
                    if (page < 0 || page >= a.n_pages) {
                        set_status(status, K3MOE_DEV_BAD_INDEX);
                        row = a.n_pages * a.page;             // past the cache: zeros
                    } else {
                        row = page * a.page + (at & (a.page - 1));
                    }
                }
                const int n = uniform(__popc(__ballot_sync(0xffffffffu, row >= 0)));
                const int row0 = uniform(__shfl_sync(0xffffffffu, row, 0));
                const uint32_t rows_bytes = (uint32_t)(box_rows * 128);
                auto load = [&](int slot, int group, uint64_t *full) {
                    uint8_t *dst = ring + slot * kAtBox;
                    if (n > 0) tma3d_warp(dst, &m1, 0, row0, group, full);
#pragma unroll 1
                    for (int j = 1; j < n; j++) tma3d_warp(dst + j * rows_bytes, &m1, 0, uniform(__shfl_sync(0xffffffffu, row, j)), group, full);
                };
#pragma unroll 1
                for (int j = half; j < kAtPairs; j += 2) {
                    uint64_t *full = &sh.full[turn][j];
                    if (tile >= 2 && (!(ok = wait(sh.empty[turn][j], phase - 1)) || (j == 0 && !(ok = wait(sh.r_empty[turn], phase - 1))))) break;
                    mb_expect_tx_warp(full, (j == 0 ? 3 : 2) * n * rows_bytes);
                    if (j == 0) load(16 + turn, 8, full);
                    if (box_rows == kAtTile) {                // a pair is one copy
                        if (n > 0) tma3d_warp(ring + (8 * turn + 2 * j) * kAtBox, &m2, 0, row0, 2 * j, full);
                    } else {
#pragma unroll 1
                        for (int b = 2 * j; b < 2 * j + 2; b++) load(8 * turn + b, b, full);
                    }
                    asked++;
                }
                if (!ok) break;
            }
            // the query blocks that cuts leave unfinished, for the second kernel
            if (half == 0 && lane == 0 && (begun > 0 || left > 0)) {
                const int first = begun > 0 ? shares.of(w.unit(0)) : blockIdx.x;
                const bool second = shares.begin(first) < w.unit(-kAtAhead);      // another one's last tile comes before it there
                joins[2 * blockIdx.x + (begun > 0)] = AttendJoin{w.s.t0, w.row0, w.rows(a), first, second, shares.of(w.unit(w.s.tiles - 1)) - first + 1};
            }
        }
        // the block's shared memory stays until its last copies have landed, when another role gave up too
        for (int i = max(0, asked - 4); i < asked; i++) mb_wait_warp(&sh.full[(i >> 1) & 1][half + 2 * (i & 1)], (uint32_t)(i >> 2) & 1u);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kAtWarpS) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(512));
}

// ---------------------------------------------------------------- joining
// out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i over the parts i, M the largest m.  Blocks (x, y) for share x: of a query
// block with few parts, the share's that begins it have eight queries each, a warp a query, a lane 16 columns; with many, all its
// shares' have a quarter of a query's columns at a time, two, four or eight warps on it by the parts, so that a warp has asked for all
// of its own, or a good many, before it looks at the first.  Its loads' latency is what it takes: two blocks an SM that go on to
// their next piece, rather than eight that wait for a place (draft of 11: 24.5 us for both kernels then; a block a piece with barriers
// for the factors 27.0).
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kJoinBlocks = 4, kJoinMany = 8, kJoinDeep = 10;
static_assert(kMaxShares <= 64 * kJoinWarps, "two factors a lane");

// Where a join's parts begin in the workspace, in floats.
struct JoinParts {
    uint32_t p0, p1;                                          // the first part, and the second
    __device__ JoinParts(int share, int second) : p0((2 * share + second) * (uint32_t)kAtPart), p1((2 * share + 2) * (uint32_t)kAtPart) {}
    __device__ uint32_t operator()(int p) const { return p == 0 ? p0 : p1 + (uint32_t)(p - 1) * (uint32_t)(2 * kAtPart); }
};
static_assert((2 * kMaxShares + 2) * kAtPart < 1ull << 32, "in 32 bits");
__device__ __forceinline__ void join_add(float4 &o, float f, const float4 &x)
{
    o.x = fmaf(f, x.x, o.x);
    o.y = fmaf(f, x.y, o.y);
    o.z = fmaf(f, x.z, o.z);
    o.w = fmaf(f, x.w, o.w);
}
__device__ __forceinline__ void join_put(uint16_t *to, const float4 &o, float inv)
{
    const __nv_bfloat162 w[2] = {__floats2bfloat162_rn(o.x * inv, o.y * inv), __floats2bfloat162_rn(o.z * inv, o.w * inv)};
    *reinterpret_cast<uint2 *>(to) = *reinterpret_cast<const uint2 *>(w);
}
__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__global__ void __launch_bounds__(kJoinThreads, 2)
    attend_join_kernel(const AttendArgs a, const float *parts, const AttendJoin *joins)
{
    pdl_wait();
    pdl_trigger();
    __shared__ float4 sum[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const AttendJoin j = joins[2 * blockIdx.x], on = joins[2 * blockIdx.x + 1];
    auto row_of = [&](const AttendJoin &j, int r) { return (size_t)j.t0 * a.H + j.row0 + r; };
    auto inverse = [](float L) { return L == 0.0f ? 0.0f : 1.0f / L; };
    for (int r = kJoinWarps * blockIdx.y + warp; j.parts < kJoinMany && r < j.rows; r += kJoinWarps * kJoinBlocks) {
        const JoinParts part(j.first, j.second);
        float m = -INFINITY, l = 0.0f;
        float4 x[2][4];
        const uint32_t at = r * kLatC + 4 * lane;
        auto load = [&](int p) {
#pragma unroll
            for (int i = 0; i < 4; i++) x[p & 1][i] = __ldcg(reinterpret_cast<const float4 *>(parts + (part(p) + at + 128 * i)));
        };
        load(0);
        load(1);                                              // a join has two parts at least
        if (lane < j.parts) {
            m = parts[part(lane) + kAtRows * kLatC + r];
            l = parts[part(lane) + kAtRows * kLatC + kAtRows + r];
        }
        const float M = warp_max(m), f = m == -INFINITY ? 0.0f : exp2_fast(m - M), L = warp_sum(f == 0.0f ? 0.0f : f * l), inv = inverse(L);
        float4 o[4] = {};
#pragma unroll 2
        for (int p = 0; p < j.parts; p++) {
            const float w = __shfl_sync(0xffffffffu, f, p);
#pragma unroll
            for (int i = 0; i < 4; i++) join_add(o[i], w, x[p & 1][i]);
            if (p + 2 < j.parts) load(p + 2);
        }
        uint16_t *to = a.out + row_of(j, r) * kLatC + 4 * lane;
#pragma unroll
        for (int i = 0; i < 4; i++) join_put(to + 128 * i, o[i], inv);
        if (a.lse && lane == 0) a.lse[row_of(j, r)] = (M + log2f(L)) * kLatLn2;
    }
    // pieces of a join: quarters of rows
    auto many = [&](const AttendJoin &j) {
        if (j.rows == 0 || j.parts < kJoinMany) return;
        const JoinParts part(j.first, j.second);
        const int share = j.parts <= 20 ? 2 : j.parts <= 40 ? 4 : kJoinWarps, sets = kJoinWarps / share;      // warps of a piece
        const int mine = warp % share, pieces = 4 * j.rows;
        for (int p0 = (blockIdx.y * j.parts + blockIdx.x - j.first) * sets; p0 < pieces; p0 += j.parts * kJoinBlocks * sets) {
            const int piece = p0 + warp / share, r = min(piece, pieces - 1) >> 2, quarter = 128 * (piece & 3);
            const uint32_t at = r * kLatC + quarter + 4 * lane;
            float4 x[kJoinDeep];
            auto load = [&](int i0) {
#pragma unroll
                for (int i = 0; i < kJoinDeep; i++)
                    if (mine + share * (i0 + i) < j.parts) x[i] = __ldcg(reinterpret_cast<const float4 *>(parts + (part(mine + share * (i0 + i)) + at)));
            };
            load(0);
            auto max_of = [&](int p) { return p < j.parts ? parts[part(p) + kAtRows * kLatC + r] : -INFINITY; };
            const float m0 = max_of(mine + share * lane), m1 = share == kJoinWarps ? max_of(mine + share * (lane + 32)) : -INFINITY;
            float M = -INFINITY, L = 0.0f;                    // of the parts lane, lane + 32 ..
#pragma unroll 4
            for (int p = lane; p < j.parts; p += 32) {
                const float m = max_of(p), l = parts[part(p) + kAtRows * kLatC + kAtRows + r];
                if (m == -INFINITY) continue;
                const float top = fmaxf(m, M);
                L = fmaf(L, exp2_fast(M - top), l * exp2_fast(m - top));
                M = top;
            }
            const float top = warp_max(M);
            L = warp_sum(M == -INFINITY ? 0.0f : L * exp2_fast(M - top));
            const float f0 = m0 == -INFINITY ? 0.0f : exp2_fast(m0 - top), f1 = m1 == -INFINITY ? 0.0f : exp2_fast(m1 - top);
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int i0 = 0; mine + share * i0 < j.parts; i0 += kJoinDeep) {
                if (i0 > 0) load(i0);
#pragma unroll
                for (int i = 0; i < kJoinDeep; i++) {
                    const float f = __shfl_sync(0xffffffffu, i0 + i < 32 ? f0 : f1, (i0 + i) & 31);
                    if (mine + share * (i0 + i) < j.parts) join_add(o, f, x[i]);
                }
            }
            if (mine > 0) sum[warp][lane] = o;
            __syncthreads();
            if (mine == 0 && piece < pieces) {
                for (int k = 1; k < share; k++) join_add(o, 1.0f, sum[warp + k][lane]);
                join_put(a.out + row_of(j, r) * kLatC + quarter + 4 * lane, o, inverse(L));
                if (a.lse && lane == 0 && quarter == 0) a.lse[row_of(j, r)] = (top + log2f(L)) * kLatLn2;
            }
            __syncthreads();
        }
    };
    many(j);
    many(on);
}

int attend_shares() { return std::min(num_sms(), kMaxShares); }

}  // namespace

size_t latent_workspace(const k3moe_latent_config &lc, int n_seq, int T)
{
    (void)lc;
    const size_t base = kCtrOffset + kCtrBytes;
    return n_seq > 0 && T > 0 ? base + kLatJoinBytes + (size_t)attend_shares() * 2 * kAtPart * 4 : base;
}

cudaError_t launch_attend(const AttendArgs &args, cudaStream_t s)
{
    AttendArgs a = args;
    // the cache as [9 boxes of columns][rows][64]: boxes of a page's or a tile's rows, two of columns at once or one
    CUtensorMap m2{}, m1{};
    const uint64_t rows = (uint64_t)a.n_pages * a.page;
    const uint32_t box_rows = (uint32_t)std::min(a.page, kAtTile);
    if (!map16x3(&m2, a.cache, kAtBoxes, 64, rows, kLatRow, 64, box_rows, 2) || !map16x3(&m1, a.cache, kAtBoxes, 64, rows, kLatRow, 64, box_rows, 1))
        return cudaErrorInvalidValue;
    const cudaError_t allowed = once_a_device([] {
        const cudaError_t e = cudaFuncSetAttribute(attend_kernel<int>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAtSmem);
        return e != cudaSuccess ? e : cudaFuncSetAttribute(attend_kernel<long long>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAtSmem);
    });
    if (allowed != cudaSuccess) return allowed;
    // whether every count of tiles fits 32 bits, whatever the offsets and lengths are: each sequence may claim all tokens
    const double most = (double)a.n_seq * ((double)a.T * a.H / 16 + 1) * ((double)a.max_pages * a.page / kAtTile + 1 + kAtAhead);
    const int shares = attend_shares();
    // With short tables a query block is one SM's, whole, and nothing is joined: that saves the second kernel and costs the tiles by which
    // the busiest SM has more than its even part, here of sequences half as long as the tables on average; six and a half of them
    // are even (one token x 56 heads behind 250 rows 10.1 us either way, behind 60 7.0 against 8.9, 380 12.1 against 10.7; 96 tokens behind
    // 500 18.6 against 22.4).
    const double blocks = std::ceil((double)a.T * a.H / kAtRows), tiles = std::ceil((double)a.max_pages * a.page / kAtTile);
    a.whole = tiles * (std::ceil(blocks / shares) - 0.5 * blocks / shares) <= 6.5;
    AttendJoin *joins = reinterpret_cast<AttendJoin *>(a.ws + kCtrOffset + kCtrBytes);
    float *parts = latent_parts(a.ws);
    timing_begin("latent_attend", s);
    cudaError_t err = launch_pdl(most < INT32_MAX ? attend_kernel<int> : attend_kernel<long long>, dim3((unsigned)shares), dim3(kAtThreads), kAtSmem, s, a,
                                 m2, m1, parts, joins);
    count_launch();
    timing_end("latent_attend", s);
    if (err != cudaSuccess || a.whole) return err;
    timing_begin("latent_attend_join", s);
    err = launch_pdl(attend_join_kernel, dim3((unsigned)shares, kJoinBlocks), dim3(kJoinThreads), 0, s, a, (const float *)parts, (const AttendJoin *)joins);
    count_launch();
    timing_end("latent_attend_join", s);
    return err;
}

}  // namespace k3moe
