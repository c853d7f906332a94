// k3moe_attend.cu -- latent attention in the absorbed form: every query head attends the same
// cached rows [c, r] of 576 columns, whose first 512 are the values too.
//
// A block has up to 64 query rows (heads of one token, or of a few) of one sequence and walks cached rows in tiles
// of 128.  Scores are taken transposed, S^T [row of the cache][query] = cache Q^T, so that the cache's 128 rows fill the
// tensor core's M side whatever the number of heads, and the outputs likewise, O^T [c][query] += C^T P^T with the tile in
// shared memory as the A operand of both (read along c the second time).  Softmax in powers of two as in the
// expanded form; a query's maximum moves only when it is outdone by 2^8, so that a tile mostly needs no more than a vote.
//
// Bound by the cache's bytes: 1152 a row against 64 x 2176 flops.  All tiles of all sequences are one line that is cut into
// as many even parts as there are SMs; a query block that a cut goes through leaves its parts' sums (float) in the workspace,
// and a second kernel joins them.
#include <cuda.h>
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"
#include "k3moe_latent.cuh"

namespace k3moe {
namespace {

constexpr int kAtRows = 64, kAtTile = 128;                    // queries of a block, cached rows of a tile
constexpr int kAtBoxes = kLatRow / 64;                        // 64-column boxes of a tile: r first, then c
constexpr int kAtBox = kAtTile * 128;                         // 16 KB
constexpr int kAtSlots = 8;
constexpr int kAtQBox = kAtRows * 128;
constexpr int kAtQ = kAtBoxes * kAtQBox, kAtP = kAtTile * kAtRows * 2;
constexpr int kAtSmem = 1024 + kAtQ + kAtP + kAtSlots * kAtBox;
// Warps: two groups of four share the softmax (32 queries each), then MMA issue, the cache's loads, two for the queries'
constexpr int kAtThreads = 384, kAtWarpMma = 8, kAtWarpLoad = 9, kAtWarpQ = 10;
constexpr uint32_t kAtTmS = 0, kAtTmO = 64;                   // S^T, and O^T in four blocks of 128 of c
constexpr float kAtSlack = 8.0f;

// A part's sums in the workspace: O [query][c], then the maxima and the sums of the weights.
constexpr size_t kAtPart = (size_t)kAtRows * kLatC + 2 * kAtRows;
// What a cut leaves to join: the query block's first part is share i's last (its first or second), the others
// are the first ones of the shares after it.
struct AttendJoin {
    int t0, row0, rows, second, parts;                        // its queries; rows = 0: nothing to join
};

struct AttendShared {
    uint64_t q_full, q_free, full[kAtSlots], empty[kAtSlots], s_full, p_ready, o_full, o_free, drain;
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
    __device__ bool next(const AttendArgs &a)
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

// Column sums or maxima of 32 values a lane over the warp: lane i ends with column i's.
template <typename F> __device__ __forceinline__ float over_lanes(float (&v)[32], int lane, F f)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o; j++) {
            const float keep = up ? v[j + o] : v[j], give = up ? v[j] : v[j + o];
            v[j] = f(keep, __shfl_xor_sync(0xffffffffu, give, o));
        }
    }
    return v[0];
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
// Columns a box of the tile has: r's, then c's; of a pair that wraps around the ring the lower slot takes the first.
__device__ __forceinline__ int box_column(int count, int b)
{
    if (b == 0) return kLatC;
    const int first = (b - 1) & ~1;                           // of the pair
    const int s = (count + b) % kAtSlots, other = (count + ((b - 1) & 1 ? b - 1 : b + 1)) % kAtSlots;
    return 64 * (first + (s > other));
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
    pdl_wait();
    pdl_trigger();
    long long before, units;
    // even shares, fewer of them than blocks where there are fewer tiles
    const auto shares = [&](long long all) { return min(all, (long long)gridDim.x); };
    const auto share = [&](long long i, long long all) { return i < shares(all) ? all * i / shares(all) : all; };
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
    if (threadIdx.x == 0) {
        mb_init(&sh.q_full, 2);
        mb_init(&sh.q_free, 1);
        for (int i = 0; i < kAtSlots; i++) {
            mb_init(&sh.full[i], 1);
            mb_init(&sh.empty[i], 1);
        }
        mb_init(&sh.s_full, 1);
        mb_init(&sh.p_ready, 8);
        mb_init(&sh.o_full, 1);
        mb_init(&sh.o_free, 8);
        mb_init(&sh.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.bail = 0;
        sh.spoiled[0] = sh.spoiled[1] = 0;
        prefetch_map(&mc);
    }
    if (warp == kAtWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sh.tmem)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;                              // all 512 columns: the allocation starts at the first
    auto wait = [&](uint64_t &b, int phase) {
        const bool ok = mb_wait_asleep(&b, (uint32_t)phase & 1u);
        if (!ok) {
            set_status(status, K3MOE_DEV_TIMEOUT);
            sh.bail = 1;
        }
        return (bool)__all_sync(0xffffffffu, ok && !sh.bail);
    };
    // the same for the warps that meet at barriers: after a wait that gave up they go on without waiting, to the end
    auto go_on = [&](uint64_t &b, int phase) { return !sh.bail && wait(b, phase); };
    AttendWalk w;
    w.begin(a, seq0, before, from, to);

    if (warp < kAtWarpMma) {
        // ---------------- softmax and output: cached row 32 q + lane of a tile, queries 32 g ..
        const int g = warp >> 2, q = warp & 3;
        const uint32_t la = tmem + ((uint32_t)(32 * q) << 16);
        const float c = a.scale * kLatLog2e;
        int tile = 0;                                         // so far
        for (int seg = 0; w.next(a); seg++) {
            const int rows = w.rows(a);
            // rows of the cache that each query sees
            auto limit = [&](int r) { return a.causal ? max(0, w.s.len - (w.s.n - 1 - (w.row0 + r) / a.H)) : w.s.len; };
            const int least = limit(0);                       // of all its queries
            int *lim = sh.lim[g];
            if (q == 0) lim[lane] = 32 * g + lane < rows ? limit(32 * g + lane) : 0;
            float m = -INFINITY;                              // of query 32 g + lane, the same in the group's warps
            float nm[32], l[32];
#pragma unroll
            for (int j = 0; j < 32; j++) nm[j] = l[j] = 0.0f;
            group_sync(g);
            bool first = true;
            for (int t = w.tile0; t < w.tile1; t++, tile++) {
                go_on(sh.s_full, tile);
                tc_fence_after();
                uint32_t u[32];
                tmem_ld16_nowait(la + kAtTmS + 32 * g, *reinterpret_cast<uint32_t(*)[16]>(&u[0]));
                tmem_ld16_nowait(la + kAtTmS + 32 * g + 16, *reinterpret_cast<uint32_t(*)[16]>(&u[16]));
                tmem_wait_ld();
                float v[32];
                const int at = kAtTile * t + 32 * q + lane;   // of the sequence's rows
#pragma unroll
                for (int j = 0; j < 32; j++) v[j] = __uint_as_float(u[j]) * c;
                if (kAtTile * (t + 1) > least)
#pragma unroll
                    for (int j = 0; j < 32; j++) v[j] = at < lim[j] ? v[j] : -INFINITY;
                float over = -INFINITY;
#pragma unroll
                for (int j = 0; j < 32; j++) over = fmaxf(over, v[j] + nm[j]);
                if (group_any(g, first || over > kAtSlack)) {
                    // the tile's maxima: lane j query j's
                    float x[32];
#pragma unroll
                    for (int j = 0; j < 32; j++) x[j] = v[j];
                    const float top = over_lanes(x, lane, [](float p, float r) { return fmaxf(p, r); });
                    sh.top[g][q][lane] = top;
                    group_sync(g);
                    const float all = fmaxf(fmaxf(sh.top[g][0][lane], sh.top[g][1][lane]), fmaxf(sh.top[g][2][lane], sh.top[g][3][lane]));
                    const float m1 = first || all > (m == -INFINITY ? -INFINITY : m + kAtSlack) ? fmaxf(m, all) : m;
                    const float f = m1 == -INFINITY || first ? 1.0f : exp2_fast(m - m1);
                    m = m1;
                    if (q == 0) {
                        sh.m[32 * g + lane] = m1 == -INFINITY ? 0.0f : -m1;
                        sh.f[32 * g + lane] = f;
                    }
                    group_sync(g);
#pragma unroll
                    for (int j = 0; j < 32; j++) {
                        nm[j] = sh.m[32 * g + j];
                        l[j] *= sh.f[32 * g + j];
                    }
                    if (!first) {
                        // in order behind S: the product before is done with O
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
                uint32_t p[16];
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    const float x = exp2_fast(v[2 * j] + nm[2 * j]), y = exp2_fast(v[2 * j + 1] + nm[2 * j + 1]);
                    l[2 * j] += x;
                    l[2 * j + 1] += y;
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
                    p[j] = *reinterpret_cast<const uint32_t *>(&h);
                }
                const int row = 32 * q + lane;
#pragma unroll
                for (int j = 0; j < 4; j++)
                    *reinterpret_cast<uint4 *>(sm_p + row * 128 + (((4 * g + j) ^ (row & 7)) << 4)) =
                        make_uint4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
                if (at >= least) {
                    // rows behind the last are cleared, and of rows that some query does not see what is infinite or NaN: a
                    // weight of zero would not keep it out (queries that see it add it at the end)
                    bool any = false;
#pragma unroll 1
                    for (int b = 1 + 4 * g; b < 5 + 4 * g; b++) {
                        uint4 *x = reinterpret_cast<uint4 *>(ring + (tile * kAtBoxes + b) % kAtSlots * kAtBox + row * 128);
#pragma unroll 1
                        for (int j = 0; j < 8; j++) {
                            uint4 y = x[j];
                            if (at >= w.s.len) {
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
                if (lane == 0) mb_arrive(&sh.p_ready);
            }
            // the weights' sums: lane j query j's
            sh.sum[g][q][lane] = over_lanes(l, lane, [](float x, float y) { return x + y; });
            group_sync(g);
            const float sum = (sh.sum[g][0][lane] + sh.sum[g][1][lane]) + (sh.sum[g][2][lane] + sh.sum[g][3][lane]);
            const bool whole = w.whole();
            const int mine = 32 * g + lane;
            // a share's first query block leaves its part in the block's first place, a later one in the second
            float *part = parts + (size_t)(2 * blockIdx.x + (seg > 0)) * kAtPart;
            if (q == 0) {
                sh.inv[mine] = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
                if (!whole) {
                    part[kAtRows * kLatC + mine] = m;
                    part[kAtRows * kLatC + kAtRows + mine] = sum;
                } else if (a.lse && mine < rows) {
                    a.lse[(size_t)w.s.t0 * a.H + w.row0 + mine] = (m + log2f(sum)) * kLatLn2;
                }
            }
            group_sync(g);
            const bool ok = go_on(sh.o_full, seg);
            tc_fence_after();
            const bool spoiled = *const_cast<volatile int *>(&sh.spoiled[seg & 1]) != 0;
            const int count = ok ? min(32, rows - 32 * g) : 0;
#pragma unroll 1
            for (int b = 0; b < 8; b++) {
                const int col = 128 * (b >> 1) + 32 * q + lane, r0 = 32 * g + 16 * (b & 1);   // of c; the first of 16 queries
                float o[16];
                tmem_ld16(la + kAtTmO + 64 * (b >> 1) + r0, o);
                if (spoiled)
                    for (int at = max(least, kAtTile * w.tile0); at < min(w.s.len, kAtTile * w.tile1); at++) {
                        const int page = a.pages[(size_t)w.seq * a.max_pages + at / a.page];
                        if (page < 0 || page >= a.n_pages) continue;
                        const uint32_t x = a.cache[((size_t)page * a.page + at % a.page) * kLatRow + col];
                        if ((x & 0x7F80u) != 0x7F80u) continue;
#pragma unroll
                        for (int j = 0; j < 16; j++)
                            if (at < lim[16 * (b & 1) + j]) o[j] += bf16_bits_to_f32(x);
                    }
                const int left = min(16, count - 16 * (b & 1));
                if (whole) {
                    __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(a.out) + ((size_t)w.s.t0 * a.H + w.row0 + r0) * kLatC + col;
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (j < left) p[(size_t)j * kLatC] = __float2bfloat16_rn(sh.inv[r0 + j] == 0.0f ? 0.0f : o[j] * sh.inv[r0 + j]);
                } else {
                    float *p = part + (size_t)r0 * kLatC + col;
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        if (j < left) p[(size_t)j * kLatC] = o[j];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mb_arrive(&sh.o_free);
            // the next query block has its flag cleared, and both groups are done with this one
            if (threadIdx.x == 0) sh.spoiled[~seg & 1] = 0;
            asm volatile("bar.sync 3, 256;" ::: "memory");
        }
    } else if (warp == kAtWarpMma) {
        // ---------------- products
        const uint32_t ids = idesc(1, kAtRows), idv = idesc(1, kAtRows) | (1u << 15) | (1u << 16);    // both with M, N contiguous
        const uint32_t q0 = desc_lo(saddr(sm)), p0 = desc_lo(saddr(sm_p)), r0 = saddr(ring);
        int tile = 0;
        bool ok = true;
        for (int seg = 0; ok && w.next(a); seg++) {
            if (!(ok = wait(sh.q_full, seg))) break;
            for (int t = w.tile0; t < w.tile1; t++, tile++) {
                const int count = tile * kAtBoxes;
                for (int b = 0; b < kAtBoxes; b++) {
                    const int s = (count + b) % kAtSlots;
                    if (!(ok = wait(sh.full[s], (count + b) / kAtSlots))) break;
                    tc_fence_after();
                    const uint32_t A = desc_lo(r0 + (uint32_t)(s * kAtBox)), B = q0 + (uint32_t)(box_column(count, b) / 64 * kAtQBox >> 4);
#pragma unroll
                    for (int k = 0; k < 4; k++) umma_warp(kAtTmS, A + 2 * k, B + 2 * k, ids, b > 0 || k > 0);
                    if (b == 0) umma_commit_warp(&sh.empty[s]);
                }
                if (!ok) break;
                umma_commit_warp(&sh.s_full);
                if (t == w.tile1 - 1) umma_commit_warp(&sh.q_free);
                if (!(ok = wait(sh.p_ready, tile))) break;
                if (t == w.tile0 && seg > 0 && !(ok = wait(sh.o_free, seg - 1))) break;
                tc_fence_after();
#pragma unroll 1
                for (int b = 1; b < kAtBoxes; b += 2) {
                    const int s0 = (count + b) % kAtSlots, s1 = (count + b + 1) % kAtSlots, lo = min(s0, s1);
                    const uint32_t A = desc_lo(r0 + (uint32_t)(lo * kAtBox), (uint32_t)((max(s0, s1) - lo) * kAtBox));
#pragma unroll
                    for (int k = 0; k < kAtTile / 16; k++)
                        umma_warp(kAtTmO + 32 * (b - 1), A + (uint32_t)(k * 16 * 128 >> 4), p0 + (uint32_t)(k * 16 * 128 >> 4), idv,
                                  t > w.tile0 || k > 0);
                    umma_commit_warp(&sh.empty[s0]);
                    umma_commit_warp(&sh.empty[s1]);
                }
            }
            if (ok) umma_commit_warp(&sh.o_full);
        }
        __syncwarp();
        umma_commit_warp(&sh.drain);                           // every issued MMA done before the dealloc
        mb_wait_warp(&sh.drain, 0);
    } else if (warp == kAtWarpLoad) {
        // ---------------- the cache's rows: boxes of a page's rows, a lane a page
        const int box_rows = min(a.page, kAtTile), pieces = kAtTile / box_rows;
        int loaded = 0;
        bool ok = true;
        while (ok && w.next(a)) {
            for (int t = w.tile0; ok && t < w.tile1; t++) {
                const int at = kAtTile * t + lane * box_rows;
                int row = -1;                                 // nothing to load
                if (lane < pieces && at < w.s.len) {
                    const int page = a.pages[(size_t)w.seq * a.max_pages + at / a.page];
                    if (page < 0 || page >= a.n_pages) {
                        set_status(status, K3MOE_DEV_BAD_INDEX);
                        row = a.n_pages * a.page;             // past the cache: zeros
                    } else {
                        row = page * a.page + at % a.page;
                    }
                }
                const int n = __popc(__ballot_sync(0xffffffffu, row >= 0)), count = loaded;
                for (int b = 0; b < kAtBoxes; b++, loaded++) {
                    const int s = loaded % kAtSlots;
                    if (loaded >= kAtSlots && !(ok = wait(sh.empty[s], loaded / kAtSlots - 1))) break;
                    mb_expect_tx_warp(&sh.full[s], (uint32_t)(n * box_rows * 128));
                    const int col = box_column(count, b);
                    for (int i = 0; i < n; i++)
                        tma2d_warp(ring + s * kAtBox + i * box_rows * 128, &mc, col, __shfl_sync(0xffffffffu, row, i), &sh.full[s]);
                }
            }
        }
        // the block's shared memory stays until its last copies have landed, when another role gave up too
        for (int f = max(0, loaded - kAtSlots); f < loaded; f++) mb_wait_warp(&sh.full[f % kAtSlots], (uint32_t)(f / kAtSlots) & 1u);
    } else {
        // ---------------- the queries, in the order the tensor core reads: 64 columns of 64 rows a box, 128-byte swizzle
        const int id = threadIdx.x - 32 * kAtWarpQ;
        bool last = false;
        for (int seg = 0; w.next(a); seg++) {
            const int rows = w.rows(a);
            if (seg > 0 && !wait(sh.q_free, seg - 1)) break;
            for (int e = id; e < kAtRows * (kLatRow / 8); e += 64) {
                const int r = e / (kLatRow / 8), x = e % (kLatRow / 8), gr = w.row0 + (r < rows ? r : 0);
                const uint16_t *src = a.q + (size_t)(w.s.t0 + gr / a.H) * a.q_stride + (size_t)(gr % a.H) * a.q_head + 8 * x;
                cp_async16(saddr(sm) + (uint32_t)((x >> 3) * kAtQBox + r * 128 + (((x & 7) ^ (r & 7)) << 4)), src, r < rows);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mb_arrive(&sh.q_full);
            // the query block that a cut leaves unfinished, for the second kernel: its first part writes it down
            last = w.u >= w.end && w.tile0 == 0 && w.tile1 < w.s.tiles;
            if (last && id == 0) {
                const long long done = w.u + (w.s.tiles - w.tile1);
                int parts = 1;
                while (share(blockIdx.x + parts, units) < done) parts++;
                joins[blockIdx.x] = AttendJoin{w.s.t0, w.row0, rows, seg > 0, parts};
            }
        }
        if (!last && id == 0) joins[blockIdx.x].rows = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kAtWarpMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(512));
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
