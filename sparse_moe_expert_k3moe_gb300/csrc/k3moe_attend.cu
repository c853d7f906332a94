// k3moe_attend.cu -- latent attention in the absorbed form: every query head attends the same
// cached rows [c, r] of 576 columns, whose first 512 are the values too.
//
// A block has up to 64 query rows (heads of one token, or of a few) of one sequence and walks cached rows in tiles
// of 64.  Scores are taken transposed, S^T [row of the cache][query] = cache Q^T, so that the tile is the A operand whatever
// the number of heads, and the outputs likewise, O^T [c][query] += C^T P^T with the same tile in shared memory read along
// c.  Softmax in powers of two as in the expanded form; a query's maximum moves only when it is outdone by 2^8, so that a
// tile mostly needs no more than a vote.
//
// Bound by the cache's bytes: 1152 a row against 64 x 2176 flops.  A tile is 72 KB, and the ring beside the queries (72 KB)
// holds not quite two: with tiles of 128 rows nothing could be loaded under a tile's softmax, all SMs loaded and computed in
// step, and the DRAM was idle half of the time (96 sequences: 158 us).  All tiles of all sequences are one line that is cut
// into as many even parts as there are SMs; a query block that a cut goes through leaves its parts' sums (float) in the
// workspace, and a second kernel joins them.
#include <cuda.h>
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"
#include "k3moe_latent.cuh"

namespace k3moe {
namespace {

constexpr int kAtRows = 64, kAtTile = 64;                     // queries of a block, cached rows of a tile
constexpr int kAtBoxes = kLatRow / 64;                        // 64-column boxes of a tile: c's eight, then r's
constexpr int kAtBox = kAtTile * 128;                         // 8 KB
constexpr int kAtSlots = 17;                                  // c of even tiles, c of odd tiles, r of either
constexpr int kAtQBox = kAtRows * 128;
constexpr int kAtQ = kAtBoxes * kAtQBox, kAtP = kAtTile * kAtRows * 2;
constexpr int kAtSmem = 1024 + kAtQ + kAtP + kAtSlots * kAtBox;
// Warps: two groups of four share the softmax (32 queries each), two issue the products, scores and outputs, and two the
// cache's loads, of half of c each and r
constexpr int kAtThreads = 384, kAtWarpS = 8, kAtWarpV = 9, kAtWarpLoad = 10;
constexpr uint32_t kAtTmS = 0, kAtTmO = 128;                  // S^T of two tiles, and O^T in four blocks of 128 of c
constexpr float kAtSlack = 8.0f;

// A part's sums in the workspace: O [query][c], then the maxima and the sums of the weights.
constexpr size_t kAtPart = (size_t)kAtRows * kLatC + 2 * kAtRows;
// What a cut leaves to join: the query block's first part is share i's last (its first or second), the others
// are the first ones of the shares after it.
struct AttendJoin {
    int t0, row0, rows, second, parts;                        // its queries; rows = 0: nothing to join
};

struct AttendShared {
    uint64_t q_full, full[2][2], empty[2][4], r_empty, s_full[2], p_ready[2], pv_done, drain[2];    // by the tile's turn: half of c; its pairs
    uint32_t tmem;
    volatile int bail;
    int spoiled[2];                                           // by the query block's turn
    float top[2][4][32], m[kAtRows], f[kAtRows], sum[2][4][32], inv[kAtRows];
    int lim[2][kAtRows];
    UnitSearch search;
};

// Sequence i: its queries, cached rows, blocks of queries and tiles of each; false when something does not fit.
struct AttendSeq {
    int t0, n, len, blocks, tiles;
    __device__ bool read(const AttendArgs &a, int i)
    {
        bool ok = latent_queries(a.seq_start, a.n_seq, a.T, i, &t0, &n);
        len = a.kv_len[i];
        ok = ok && len >= 0 && len <= a.max_pages * a.page;
        blocks = ok ? (int)(((long long)n * a.H + kAtRows - 1) / kAtRows) : 0;
        tiles = max(1, (len + kAtTile - 1) / kAtTile);        // one that has nothing where no row is cached
        return ok;
    }
    __device__ long long units() const { return (long long)blocks * tiles; }
};

// The walk of a block's share of tiles, query block by query block.
struct AttendWalk {
    long long u, end, base;                                   // next tile, the share's end, the sequence's first tile
    int seq;
    AttendSeq s;
    int row0, tile0, tile1;                                   // the query block and its tiles here
    __device__ void begin(const AttendArgs &a, int i, long long before, long long from, long long to)
    {
        u = from;
        end = to;
        seq = i;
        base = from - before;
        if (u < end) s.read(a, i);
    }
    __device__ __noinline__ bool next(const AttendArgs &a)
    {
        if (u >= end) return false;
        while (u >= base + s.units()) {
            base += s.units();
            s.read(a, ++seq);
        }
        const long long at = u - base;
        const int block = (int)(at / s.tiles);
        row0 = block * kAtRows;
        tile0 = (int)(at - (long long)block * s.tiles);
        tile1 = (int)min((long long)s.tiles, tile0 + (end - u));
        u += tile1 - tile0;
        return true;
    }
    __device__ int rows(const AttendArgs &a) const { return (int)min((long long)kAtRows, (long long)s.n * a.H - row0); }
    __device__ bool whole() const { return tile0 == 0 && tile1 == s.tiles; }
};

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
__global__ void __launch_bounds__(kAtThreads, 1)
    attend_kernel(const AttendArgs a, const __grid_constant__ CUtensorMap mc, float *parts, AttendJoin *joins)
{
    extern __shared__ __align__(1024) uint8_t asm_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(asm_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sm_p = sm + kAtQ, *ring = sm_p + kAtP;
    __shared__ AttendShared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *status = reinterpret_cast<int32_t *>(a.ws);
    if (threadIdx.x == 0) {
        mb_init(&sh.q_full, 8);
        for (int i = 0; i < 2; i++) {
            for (int j = 0; j < 2; j++) mb_init(&sh.full[i][j], 1);
            for (int j = 0; j < 4; j++) mb_init(&sh.empty[i][j], 1);
            mb_init(&sh.s_full[i], 1);
            mb_init(&sh.p_ready[i], 8);
            mb_init(&sh.drain[i], 1);
        }
        mb_init(&sh.r_empty, 1);
        mb_init(&sh.pv_done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.bail = 0;
        sh.spoiled[0] = sh.spoiled[1] = 0;
        prefetch_map(&mc);
    }
    pdl_wait();
    pdl_trigger();
    long long before, units;
    // even shares, fewer of them than blocks where there are fewer tiles
    const auto share = [&](long long i, long long all) {
        if (all <= gridDim.x) return min(i, all);
        const long long each = all / gridDim.x, more = all - each * gridDim.x;
        return i * each + min(i, more);
    };
    const int seq0 = find_unit<kAtThreads>(
        sh.search, a.n_seq, &before, &units,
        [&](int i) -> long long {
            AttendSeq s;
            if (!s.read(a, i)) set_status(status, K3MOE_DEV_BAD_OFFSETS);
            return s.units();
        },
        [&](long long all) { return share(blockIdx.x, all); });
    const long long from = share(blockIdx.x, units), to = share(blockIdx.x + 1, units);
    if (from >= to) {
        if (threadIdx.x == 0) joins[blockIdx.x].rows = 0;
        return;
    }
    if (warp == kAtWarpS) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sh.tmem)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;                              // all 512 columns: the allocation starts at the first
    auto wait = [&](uint64_t &b, int phase) {
        const bool ok = mb_wait_warp(&b, (uint32_t)phase & 1u);
        if (!ok) {
            set_status(status, K3MOE_DEV_TIMEOUT);
            sh.bail = 1;
        }
        return ok;
    };
    // the same for the warps that meet at barriers: after a wait that gave up they go on without waiting, to the end
    auto go_on = [&](uint64_t &b, int phase) { return !sh.bail && wait(b, phase); };
    AttendWalk w;
    w.begin(a, seq0, before, from, to);

    if (warp < kAtWarpS) {
        // ---------------- queries, softmax and output: cached rows 16 q + lane / 4 and 8 more of a tile, queries 32 g ..
        const int g = warp >> 2, q = warp & 3, row = 16 * q + (lane >> 2), col = 2 * (lane & 3);
        const uint32_t la = tmem + ((uint32_t)(32 * q) << 16);
        const float c = a.scale * kLatLog2e;
        // the next query block's rows, in the order the tensor core reads: 64 columns of 64 rows a box, 128-byte swizzle
        auto load_q = [&]() {
            const int r = threadIdx.x >> 2, rows = w.rows(a), gr = w.row0 + (r < rows ? r : 0);
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
        bool more = w.next(a);
        load_q();
        q_loaded();
        for (int seg = 0; more; seg++) {
            const AttendWalk now = w;
            const int rows = w.rows(a);
            // rows of the cache that each query sees
            auto limit = [&](int r) { return a.causal ? max(0, now.s.len - (now.s.n - 1 - (now.row0 + r) / a.H)) : now.s.len; };
            const int least = limit(0);                       // of all its queries
            int *lim = sh.lim[g];
            if (q == 0) lim[lane] = 32 * g + lane < rows ? limit(32 * g + lane) : 0;
            float m[8], l[8];                                 // maxima (minus; 0 where there is none) and sums of columns 8 k + col, + 1
#pragma unroll
            for (int j = 0; j < 8; j++) m[j] = l[j] = 0.0f;
            if (q == 0) sh.m[32 * g + lane] = -INFINITY;
            group_sync(g);
            bool first = true;
            for (int t = now.tile0; t < now.tile1; t++, tile++) {
                go_on(sh.s_full[tile & 1], tile >> 1);
                tc_fence_after();
                uint32_t u[16];
                tmem_ld_16x256(la + kAtTmS + 64 * (tile & 1) + 32 * g, u);
                float v[16];
                const int at = kAtTile * t + row;             // of the sequence's rows
#pragma unroll
                for (int j = 0; j < 16; j++) v[j] = __uint_as_float(u[j]) * c;
                if (kAtTile * (t + 1) > least)
#pragma unroll
                    for (int j = 0; j < 16; j++) {
                        const int see = lim[8 * (j >> 2) + col + (j & 1)];
                        v[j] = at + 4 * (j & 2) < see ? v[j] : -INFINITY;
                    }
                float over = -INFINITY;
#pragma unroll
                for (int j = 0; j < 16; j++) over = fmaxf(over, v[j] + m[(j >> 2) * 2 + (j & 1)]);
                if (group_any(g, first || over > kAtSlack)) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; j++) x[j] = fmaxf(v[4 * (j >> 1) + (j & 1)], v[4 * (j >> 1) + 2 + (j & 1)]);
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
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const int at = 32 * g + 8 * (j >> 1) + col + (j & 1);
                        m[j] = sh.m[at] == -INFINITY ? 0.0f : -sh.m[at];
                        l[j] *= sh.f[at];
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
                uint32_t p[8];
#pragma unroll
                for (int k = 0; k < 4; k++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float x = exp2_fast(v[4 * k + 2 * i] + m[2 * k]), y = exp2_fast(v[4 * k + 2 * i + 1] + m[2 * k + 1]);
                        l[2 * k] += x;
                        l[2 * k + 1] += y;
                        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
                        p[2 * k + i] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                // a row's weights of 64 queries are 128 bytes of P, 128-byte swizzle; the product before has read its own
                if (tile > 0) go_on(sh.pv_done, tile - 1);
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
                    part[kAtRows * kLatC + mine] = sh.m[mine];
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
#pragma unroll 1
            for (int b = 0; b < 8; b++) {
                const int at_c = 128 * (b >> 1) + 32 * q + lane, r0 = 32 * g + 16 * (b & 1);   // of c; the first of 16 queries
                float o[16];
                tmem_ld16(la + kAtTmO + 64 * (b >> 1) + r0, o);
                if (spoiled)
#pragma unroll 1
                    for (int at = max(least, kAtTile * now.tile0); at < min(now.s.len, kAtTile * now.tile1); at++) {
                        const int page = a.pages[(size_t)now.seq * a.max_pages + at / a.page];
                        if (page < 0 || page >= a.n_pages) continue;
                        const uint32_t x = a.cache[((size_t)page * a.page + at % a.page) * kLatRow + at_c];
                        if ((x & 0x7F80u) != 0x7F80u) continue;
#pragma unroll
                        for (int j = 0; j < 16; j++)
                            if (at < lim[16 * (b & 1) + j]) o[j] += bf16_bits_to_f32(x);
                    }
                const int left = min(16, count - 16 * (b & 1));
                if (whole) {
                    __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(a.out) + ((size_t)now.s.t0 * a.H + now.row0 + r0) * kLatC + at_c;
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (j < left) p[(size_t)j * kLatC] = __float2bfloat16_rn(sh.inv[r0 + j] == 0.0f ? 0.0f : o[j] * sh.inv[r0 + j]);
                } else {
                    float *p = part + (size_t)r0 * kLatC + at_c;
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (j < left) p[(size_t)j * kLatC] = o[j];
                }
            }
            tc_fence_before();                                // the next query block's first product is after its weights
            // the next query block has its flag cleared, and both groups are done with this one
            if (threadIdx.x == 0) sh.spoiled[~seg & 1] = 0;
            asm volatile("bar.sync 3, 256;" ::: "memory");
        }
    } else if (warp == kAtWarpS) {
        // ---------------- scores, a tile ahead of the products with c where its boxes have landed
        const uint32_t id = (idesc(1, kAtRows) & ~(31u << 24)) | (4u << 24);                          // M = 64 rows of the cache
        const uint32_t q0 = desc_lo(saddr(sm)), c0 = desc_lo(saddr(ring));
        constexpr uint32_t box = kAtBox >> 4, q_box = kAtQBox >> 4;
        int tile = 0;
        bool ok = true;
        for (int seg = 0; ok && w.next(a); seg++) {
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
                if (!(ok = wait(sh.full[turn][0], tile >> 1))) break;
                tc_fence_after();
                product(c0 + 16 * box, q0 + 8 * q_box, true);
                umma_commit_warp(&sh.r_empty);
#pragma unroll
                for (int b = 0; b < 4; b++) product(c0 + (8 * turn + b) * box, q0 + b * q_box, false);
                if (!(ok = wait(sh.full[turn][1], tile >> 1))) break;
                tc_fence_after();
#pragma unroll
                for (int b = 4; b < 8; b++) product(c0 + (8 * turn + b) * box, q0 + b * q_box, false);
                umma_commit_warp(&sh.s_full[turn]);
            }
        }
        __syncwarp();
        umma_commit_warp(&sh.drain[0]);                        // every issued MMA done before the dealloc
        mb_wait_warp(&sh.drain[0], 0);
    } else if (warp == kAtWarpV) {
        // ---------------- products of the weights with c
        const uint32_t id = idesc(1, kAtRows) | (1u << 15) | (1u << 16);                              // both with M, N contiguous
        const uint32_t p0 = desc_lo(saddr(sm_p)), c0 = desc_lo(saddr(ring), kAtBox);
        constexpr uint32_t box = kAtBox >> 4;
        int tile = 0;
        bool ok = true;
        while (ok && w.next(a)) {
            const int n = uniform(w.tile1 - w.tile0);
#pragma unroll 1
            for (int t = 0; t < n; t++, tile++) {
                const uint32_t turn = (uint32_t)uniform(tile & 1);
                if (!(ok = wait(sh.p_ready[turn], tile >> 1))) break;
                tc_fence_after();
                const uint32_t A = c0 + 8 * turn * box;
#pragma unroll
                for (int b = 0; b < 4; b++) {
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
        // ---------------- the cache's rows: half of c, of a page's rows each box, a lane a page; the first half's warp loads r
        const int box_rows = min(a.page, kAtTile), pieces = kAtTile / box_rows, half = uniform(warp - kAtWarpLoad);
        int tile = 0;
        bool ok = true, last = false;
        for (int seg = 0; ok && w.next(a); seg++) {
            const int n_tiles = uniform(w.tile1 - w.tile0), len = w.s.len, tile0 = w.tile0;
            const int32_t *pages = a.pages + (size_t)w.seq * a.max_pages;
#pragma unroll 1
            for (int t = 0; t < n_tiles; t++, tile++) {
                const int at = kAtTile * (tile0 + t) + lane * box_rows, turn = uniform(tile & 1), phase = tile >> 1;
                int row = -1;                                 // nothing to load
                if (lane < pieces && at < len) {
                    const int page = pages[at / a.page];
                    if (page < 0 || page >= a.n_pages) {
                        set_status(status, K3MOE_DEV_BAD_INDEX);
                        row = a.n_pages * a.page;             // past the cache: zeros
                    } else {
                        row = page * a.page + at % a.page;
                    }
                }
                const int n = uniform(__popc(__ballot_sync(0xffffffffu, row >= 0)));
                const int row0 = uniform(__shfl_sync(0xffffffffu, row, 0));
                uint64_t *full = &sh.full[turn][half];
                auto load = [&](int slot, int col) {
                    uint8_t *dst = ring + slot * kAtBox;
                    if (n > 0) tma2d_warp(dst, &mc, col, row0, full);
#pragma unroll 1
                    for (int j = 1; j < n; j++)
                        tma2d_warp(dst + j * box_rows * 128, &mc, col, uniform(__shfl_sync(0xffffffffu, row, j)), full);
                };
                if (tile >= 2 && !(ok = wait(sh.empty[turn][2 * half], phase - 1))) break;
                mb_expect_tx_warp(full, (uint32_t)((half == 0 ? 5 : 4) * n * box_rows * 128));
                load(8 * turn + 4 * half, 256 * half);
                load(8 * turn + 4 * half + 1, 256 * half + 64);
                if (tile >= 2 && !(ok = wait(sh.empty[turn][2 * half + 1], phase - 1))) break;
                load(8 * turn + 4 * half + 2, 256 * half + 128);
                load(8 * turn + 4 * half + 3, 256 * half + 192);
                if (half == 0) {
                    if (tile >= 1 && !(ok = wait(sh.r_empty, tile - 1))) break;
                    load(16, kLatC);
                }
            }
            // the query block that a cut leaves unfinished, for the second kernel: its first part writes it down
            last = w.u >= w.end && w.tile0 == 0 && w.tile1 < w.s.tiles;
            if (last && half == 0 && lane == 0) {
                const long long done = w.u + (w.s.tiles - w.tile1);
                int parts = 1;
                while (share(blockIdx.x + parts, units) < done) parts++;
                joins[blockIdx.x] = AttendJoin{w.s.t0, w.row0, w.rows(a), seg > 0, parts};
            }
        }
        if (!last && half == 0 && lane == 0) joins[blockIdx.x].rows = 0;
        // the block's shared memory stays until its last copies have landed, when another role gave up too (boxes that a
        // wait cut short do not complete: that wait is bounded as well)
        for (int f = max(0, tile - 2 + !ok); f < tile + !ok; f++) mb_wait_warp(&sh.full[f & 1][half], (uint32_t)(f >> 1) & 1u);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kAtWarpS) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(512));
}

// ---------------------------------------------------------------- joining
// out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i over the parts i in order, M the largest m.  A block takes one query at
// a time, a thread four columns, sixteen parts' loads in flight.
constexpr int kJoinThreads = 128, kJoinDeep = 16, kMaxShares = 512;

__global__ void __launch_bounds__(kJoinThreads)
    attend_join_kernel(const AttendArgs a, const float *parts, const AttendJoin *joins, const int shares)
{
    pdl_wait();
    pdl_trigger();
    __shared__ int upto[kMaxShares];                          // queries of the joins up to each
    __shared__ float weight[kMaxShares], sums[kMaxShares];
    __shared__ int warp_sum[kJoinThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int total = 0;
    for (int i0 = 0; i0 < shares; i0 += kJoinThreads) {
        const int i = i0 + threadIdx.x;
        int v = i < shares ? joins[i].rows : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        if (lane == 31) warp_sum[warp] = v;
        __syncthreads();
        int before = total;
        for (int k = 0; k < kJoinThreads / 32; k++) {
            if (k < warp) before += warp_sum[k];
            total += warp_sum[k];
        }
        if (i < shares) upto[i] = before + v;
        __syncthreads();
    }
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
        int lo = 0, hi = shares - 1;                          // the first share with upto > unit
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (upto[mid] > unit)
                hi = mid;
            else
                lo = mid + 1;
        }
        const AttendJoin j = joins[lo];
        const int r = unit - (upto[lo] - j.rows);
        const float *p0 = parts + (size_t)(2 * lo + j.second) * kAtPart, *p1 = parts + (size_t)(2 * lo + 2) * kAtPart;
        auto part = [&](int p) { return p == 0 ? p0 : p1 + (size_t)(p - 1) * 2 * kAtPart; };
        for (int p = threadIdx.x; p < j.parts; p += kJoinThreads) {
            weight[p] = part(p)[kAtRows * kLatC + r];
            sums[p] = part(p)[kAtRows * kLatC + kAtRows + r];
        }
        __syncthreads();
        float M = -INFINITY, L = 0.0f;
        for (int p = 0; p < j.parts; p++) M = fmaxf(M, weight[p]);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const size_t at = (size_t)r * kLatC + 4 * threadIdx.x;
        for (int p = 0; p < j.parts; p += kJoinDeep) {
            float4 x[kJoinDeep];
#pragma unroll
            for (int k = 0; k < kJoinDeep; k++)
                if (p + k < j.parts) x[k] = __ldcg(reinterpret_cast<const float4 *>(part(p + k) + at));
#pragma unroll
            for (int k = 0; k < kJoinDeep; k++)
                if (p + k < j.parts && weight[p + k] != -INFINITY) {
                    const float f = exp2_fast(weight[p + k] - M);
                    L = fmaf(f, sums[p + k], L);
                    o.x = fmaf(f, x[k].x, o.x);
                    o.y = fmaf(f, x[k].y, o.y);
                    o.z = fmaf(f, x[k].z, o.z);
                    o.w = fmaf(f, x[k].w, o.w);
                }
        }
        const size_t row = (size_t)j.t0 * a.H + j.row0 + r;
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        const __nv_bfloat162 w[2] = {__floats2bfloat162_rn(o.x * inv, o.y * inv), __floats2bfloat162_rn(o.z * inv, o.w * inv)};
        *reinterpret_cast<uint2 *>(a.out + row * kLatC + 4 * threadIdx.x) = *reinterpret_cast<const uint2 *>(w);
        if (a.lse && threadIdx.x == 0) a.lse[row] = (M + log2f(L)) * kLatLn2;
        __syncthreads();
    }
}

int attend_shares() { return std::min(num_sms(), kMaxShares); }

}  // namespace

size_t latent_workspace(const k3moe_latent_config &lc, int n_seq, int T)
{
    (void)lc;
    const size_t base = kCtrOffset + kCtrBytes;
    return n_seq > 0 && T > 0 ? base + align256((size_t)attend_shares() * sizeof(AttendJoin)) + (size_t)attend_shares() * 2 * kAtPart * 4 : base;
}

cudaError_t launch_attend(const AttendArgs &a, cudaStream_t s)
{
    CUtensorMap mc{};
    if (!map16s(&mc, a.cache, (uint64_t)a.n_pages * a.page, kLatRow, kLatRow, (uint32_t)std::min(a.page, kAtTile))) return cudaErrorInvalidValue;
    const cudaError_t allowed =
        once_a_device([] { return cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAtSmem); });
    if (allowed != cudaSuccess) return allowed;
    const int shares = attend_shares();
    AttendJoin *joins = reinterpret_cast<AttendJoin *>(a.ws + kCtrOffset + kCtrBytes);
    float *parts = reinterpret_cast<float *>(a.ws + kCtrOffset + kCtrBytes + align256((size_t)shares * sizeof(AttendJoin)));
    timing_begin("latent_attend", s);
    cudaError_t err = launch_pdl(attend_kernel, dim3((unsigned)shares), dim3(kAtThreads), kAtSmem, s, a, mc, parts, joins);
    count_launch();
    timing_end("latent_attend", s);
    if (err != cudaSuccess) return err;
    timing_begin("latent_attend_join", s);
    err = launch_pdl(attend_join_kernel, dim3((unsigned)(shares * 8)), dim3(kJoinThreads), 0, s, a, (const float *)parts, (const AttendJoin *)joins, shares);
    count_launch();
    timing_end("latent_attend_join", s);
    return err;
}

}  // namespace k3moe
