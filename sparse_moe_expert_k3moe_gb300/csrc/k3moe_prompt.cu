// k3moe_prompt.cu -- latent attention in the expanded form: every head has keys [k, r] of 192
// columns (r shared by all heads) and values of 128, packed sequences, causal or not.
//
// One pass over the keys with a running maximum m and sum l (softmax in powers of two):
//   p_j = 2^(c s_j - m),  l = sum p_j,  O = sum p_j v_j,  out = O / l,  lse = (m + log2 l) ln 2,
// c = scale log2 e.  A block has 256 queries of one head in two halves of 128 and walks its keys in tiles of
// 128.  The scores S = Q K^T go to tensor memory, a thread owns a row of one half: it reads its 128 scores, and
// its weights go back over them as the A operand of O += P V, so that the softmax of one half runs
// beside the products of the other.
//
// m need not be the maximum, only not far below it: the weights are taken with the m of the keys before, and their sum,
// which is needed anyway, says whether they have grown beyond 2^30; only then (and for a row's first keys) is the maximum
// looked for, O scaled down and the weights taken again.  A product's chain of steps, scores, weights, values, is
// what a tile takes, and a maximum ahead of the exponentials was a quarter of the weights' part.
//
// Measured: 8192 tokens x 56 heads 770 us (1.56 PFLOP/s; the tensor cores, and their power); 7 ragged prompts, 3001 tokens x 16 heads,
// 34.9 us (two blocks an SM, 3 us until the first scores, 1.8 a tile, 1.5 from the last to the end).
#include <cuda.h>
#include <cuda_bf16.h>

#include "k3moe_internal.cuh"
#include "k3moe_latent.cuh"

namespace k3moe {
namespace {

constexpr int kPrRows = 128, kPrTile = 128;                   // rows of a half; keys of a tile
constexpr int kPrBox = kPrTile * 128;                         // 64 columns of 128 rows: 16 KB
constexpr int kPrQBoxes = (kLatK + kLatR) / 64;               // boxes of a half's queries, and of a tile's keys
constexpr int kPrTileBoxes = kPrQBoxes + kLatV / 64;          // with its values
constexpr int kPrSlots = 8;                                   // the ring of key and value boxes
constexpr int kPrSmem = 1024 + (2 * kPrQBoxes + kPrSlots) * kPrBox;
// Warps: four of softmax for each half, then one each that issues its products, and one of loads (whole warpgroups:
// registers move)
constexpr int kPrThreads = 384, kPrWarpMma = 8, kPrWarpLoad = 10;
// Registers a thread: 168 at launch, moved from the last warpgroup to the rows' threads
constexpr int kPrRegs = 168, kPrRegsRows = 216, kPrRegsLast = 72;
static_assert(2 * kPrRegsRows + kPrRegsLast <= 3 * kPrRegs, "shares within the launch's");
// Tensor memory: S (P over its first half) and O of both halves
constexpr uint32_t kPrTmS = 0, kPrTmO = 2 * kPrTile;
constexpr float kPrLimit = 1073741824.0f;                     // 2^30: a sum of 64 weights that calls for a new m

// Few queries against many keys: `splits` blocks have an even part of the key tiles each, leave their sums in the
// workspace, O [16 columns][row] in float and then m and l of the rows, and a second kernel joins them.
constexpr int kPrBlock = 2 * kPrRows, kPrGroups = kLatV / 16, kPrMaxSplits = 16;
constexpr size_t kPrPart = (size_t)kPrBlock * kLatV + 2 * kPrBlock;
static_assert(kPrPart <= 2 * kLatPart, "a part a block, in the room of two of the absorbed form's");
// Few query blocks of unlike lengths: the longest of all sequences first, every head's, so that what is begun last is short.
// Their order is each block's own reckoning; only while all keys stay in the L2, which else wants a head's blocks together.
// 7 prompts x 16 heads, 3001 tokens: 38.4 us, head by head 44.7.
constexpr int kPrSorted = 128;
constexpr size_t kPrSortedBytes = 64u << 20;
struct PromptPlace {
    int token, rows;                                          // a block's first query, and how many
};

struct PromptShared {
    // by the tile's turn: keys and values there, and free again; by the half: its queries, scores, weights (of the first and
    // the last 64 keys of a tile), its product with the first 64 values and its output
    uint64_t k_full[2], v_full[2], k_empty[2], v_empty[2], q_full[2], s_full[2], p_ready[2][2], first_done[2], o_full[2], turn[2], drain[2];
    uint32_t tmem;
    volatile int bail, spoiled;
    int pick;
    union {
        UnitSearch<int> search;
        uint32_t order[kPrSorted];                            // work << 14 | sequence << 7 | query block
    };
};
static_assert(kPrSmem + sizeof(PromptShared) <= 227 * 1024, "an SM's shared memory");

// Queries [first, first + n) of sequence i; false when its offsets are not ascending within 0 .. T.
__device__ __forceinline__ bool latent_queries(const int32_t *start, int n_seq, int T, int i, int *first, int *n)
{
    if (!start) {
        const int each = n_seq == 1 ? T : 1;
        *first = i * each;
        *n = each;
        return true;
    }
    const int s0 = start[i], s1 = start[i + 1];
    *first = s0;
    *n = s1 - s0;
    return s0 >= 0 && s1 >= s0 && s1 <= T;
}

// 64 of a row's scores become weights in tensor memory, packed; returns their sum, of the weights as they are in float.  The
// product takes them in bf16, as it takes the values: each is off by 2^-8 of itself at most, whatever m is, and in f32 they would not
// fit over the scores.  Single floats: pairs of them cost more moves than they save here (5.7 instructions a weight, 4 this way).
__device__ __forceinline__ float weigh(const uint32_t *v, uint32_t taddr, float c, float m)
{
    const float minus = m == -INFINITY ? 0.0f : -m;
    float sum[4] = {};
#pragma unroll
    for (int b = 0; b < 2; b++) {
        float w[16];
#pragma unroll
        for (int j = 0; j < 16; j++) {
            const int i = 32 * b + 2 * j;
            const float x = exp2_fast(fmaf(__uint_as_float(v[i]), c, minus)), y = exp2_fast(fmaf(__uint_as_float(v[i + 1]), c, minus));
            sum[2 * (j & 1)] += x;
            sum[2 * (j & 1) + 1] += y;
            const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
            w[j] = __uint_as_float(*reinterpret_cast<const uint32_t *>(&h));
        }
        tmem_st16(taddr + 16 * b, w);
    }
    return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

template <bool kParts>
__global__ void __launch_bounds__(kPrThreads, 1)
    prompt_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkv,
                  const __grid_constant__ CUtensorMap mr, const int blocks, const int sorted, float *parts, PromptPlace *places)
{
    extern __shared__ __align__(1024) uint8_t psm_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(psm_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *ring = sm + 2 * kPrQBoxes * kPrBox;
    __shared__ PromptShared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *status = reinterpret_cast<int32_t *>(a.ws);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; i++) {
            mb_init(&sh.k_full[i], 1);
            mb_init(&sh.v_full[i], 1);
            mb_init(&sh.k_empty[i], 2);
            mb_init(&sh.v_empty[i], 2);
            mb_init(&sh.q_full[i], 1);
            mb_init(&sh.s_full[i], 1);
            mb_init(&sh.p_ready[i][0], 4);
            mb_init(&sh.p_ready[i][1], 4);
            mb_init(&sh.o_full[i], 1);
            mb_init(&sh.first_done[i], 1);
            mb_init(&sh.turn[i], 1);
            mb_init(&sh.drain[i], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sh.bail = 0;
        sh.spoiled = 0;
        prefetch_map(&mq);
        prefetch_map(&mkv);
        prefetch_map(&mr);
    }
    // Ahead of the wait for the kernel before, and held through it.  That one's blocks have all begun by then, so one of them that has
    // yet to take tensor memory has its SM already; it cannot be this block's SM, whose shared memory leaves 2 KB beside a block,
    // and every kernel that takes tensor memory has tens of KB.
    if (warp == kPrWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&sh.tmem)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    pdl_trigger();
    // ---- the block's queries: all blocks of a head together, so that its keys stay in the L2, the longest first; or sorted
    const int h = !kParts && sorted ? blockIdx.x % a.H : blockIdx.x / blocks;
    auto queries = [&](int i, int *t0, int *n, int *k0, int *nk) {
        bool ok = latent_queries(a.seq_start, a.n_seq, a.T, i, t0, n);
        if (a.kv_start) {
            const int s0 = a.kv_start[i], s1 = a.kv_start[i + 1];
            *k0 = s0;
            *nk = s1 - s0;
            ok = ok && s0 >= 0 && s1 >= s0 && s1 <= a.S;
        } else if (!a.seq_start && a.n_seq == 1) {
            *k0 = 0;
            *nk = a.S;
        } else {
            *k0 = *t0;
            *nk = *n;
        }
        return ok;
    };
    int t0 = 0, n = 0, k0 = 0, nk = 0;
    auto count = [&](int i, int *t0, int *n, int *k0, int *nk) {      // its query blocks
        if (!queries(i, t0, n, k0, nk)) {
            set_status(status, K3MOE_DEV_BAD_OFFSETS);
            return 0;
        }
        return (*n + 2 * kPrRows - 1) / (2 * kPrRows);
    };
    int seq, block;
    if (!kParts && sorted) {
        if (threadIdx.x < kPrSorted) sh.order[threadIdx.x] = 0;
        __syncthreads();
        if (warp == 0) {
            int all = 0;
            for (int i0 = 0; i0 < a.n_seq; i0 += 32) {
                const int mine = i0 + lane < a.n_seq ? count(i0 + lane, &t0, &n, &k0, &nk) : 0, upto = all + warp_scan(mine, lane);
                for (int b = 0, at = upto - mine; b < mine && at < blocks; b++, at++) {
                    const int rows = min(n, (b + 1) * kPrBlock), most = a.causal ? min(nk, max(0, nk - n + rows)) : nk;
                    const int work = 1 + (most + kPrTile - 1) / kPrTile;      // a tile takes one half's queries as long as both's
                    sh.order[at] = (uint32_t)(work << 14 | (i0 + lane) << 7 | b);
                }
                all = __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        __syncthreads();
        if ((int)threadIdx.x < blocks) {
            const uint32_t mine = sh.order[threadIdx.x];
            int rank = 0;
            for (int i = 0; i < blocks; i++) rank += sh.order[i] > mine || (sh.order[i] == mine && i < (int)threadIdx.x);
            if (rank == (int)blockIdx.x / a.H) sh.pick = (int)mine;
        }
        __syncthreads();
        seq = sh.pick ? sh.pick >> 7 & (kPrSorted - 1) : -1;
        block = sh.pick & (kPrSorted - 1);
    } else {
        int before, total;
        seq = find_unit<kPrThreads, int>(
            sh.search, a.n_seq, &before, &total,
            [&](int i) -> int {
                int t0, n, k0, nk;
                return count(i, &t0, &n, &k0, &nk);
            },
            [&](int) { return (int)(blockIdx.x % blocks); });
        block = -1 - before;
    }
    const int splits = kParts ? gridDim.y : 1;
    if (seq < 0) {
        if (kParts && blockIdx.y == 0 && threadIdx.x == 0) places[blockIdx.x].rows = 0;
        __syncwarp();
        if (warp == kPrWarpMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(0), "r"(512));    // as below: all
        return;
    }
    queries(seq, &t0, &n, &k0, &nk);
    if (block < 0) block += (n + kPrBlock - 1) / kPrBlock;    // counted from the last
    const int row0 = block * kPrBlock;
    // keys that row r of the sequence sees: nk + ahead + r of them, within the nk of this block's part
    int ahead = a.causal ? 1 - n : n;
    if (kParts) {
        if (blockIdx.y == 0 && threadIdx.x == 0) places[blockIdx.x] = PromptPlace{t0 + row0, min(n - row0, kPrBlock)};
        const int most = min(nk, max(0, nk + ahead + min(n, row0 + kPrBlock) - 1)), tiles = (most + kPrTile - 1) / kPrTile;
        const int first = tiles * (int)blockIdx.y / splits * kPrTile, end = min(nk, tiles * (int)(blockIdx.y + 1) / splits * kPrTile);
        k0 += first;
        ahead += nk - end;                                    // as many keys are left out at the part's end ..
        nk = max(0, end - first);                             // .. and the others before it
    }
    // the tiles of each half, and the first tile that some row does not see whole
    auto limit = [&](int r) { return min(max(nk + ahead + r, 0), nk); };
    auto tiles_of = [&](int half) {
        const int first = row0 + kPrRows * half;
        return first < n ? (limit(min(n, first + kPrRows) - 1) + kPrTile - 1) / kPrTile : 0;
    };
    const int tiles0 = tiles_of(0), tiles1 = tiles_of(1), tiles = max(tiles0, tiles1), least = limit(row0), whole = least / kPrTile;

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
    // the ring's slot of a tile's box: keys, r, values
    auto slot_of = [](int tile, int box) { return (uint32_t)(kPrTileBoxes * tile + box) % (uint32_t)kPrSlots; };

    if (warp < kPrWarpMma) {
        // ---------------- softmax and output of a half
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPrRegsRows));
        const int half = warp >> 2, q = warp & 3, r = row0 + kPrRows * half + 32 * q + lane;
        const int mine = half ? tiles1 : tiles0;
        const uint32_t la = tmem + ((uint32_t)(32 * q) << 16), la_s = la + kPrTmS + kPrTile * half, la_o = la + kPrTmO + kLatV * half;
        const int lim = r < n ? limit(r) : nk;
        const float c = a.scale * kLatLog2e;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < mine; i++) {
            if (!(ok = wait(sh.s_full[half], i))) break;
            tc_fence_after();
            uint32_t v[128];
#pragma unroll
            for (int b = 0; b < 8; b++) tmem_ld16_nowait(la_s + 16 * b, *reinterpret_cast<uint32_t(*)[16]>(&v[16 * b]));
            tmem_wait_ld();
            if (i >= whole) {
                const int left = lim - kPrTile * i;
#pragma unroll
                for (int j = 0; j < 128; j++) v[j] = j < left ? v[j] : 0xFF800000u;
            }
            if (i >= whole) {
                // of keys that not every row sees the values that are infinite or NaN are cleared, which a weight of zero would not
                // keep out (rows that see them add them at the end)
                if (!(ok = wait(sh.v_full[i & 1], i >> 1))) break;
                const int from = 8 * max(0, least - kPrTile * i) + (threadIdx.x & 127);
                for (int box = 0; box < 2; box++) {
                    uint4 *p = reinterpret_cast<uint4 *>(ring + slot_of(i, kPrQBoxes + box) * kPrBox);
#pragma unroll 1
                    for (int e = from; e < 8 * kPrTile; e += 4 * 128) {
                        uint4 w[4];
                        uint32_t any = 0;
#pragma unroll
                        for (int k = 0; k < 4; k++) w[k] = e + 128 * k < 8 * kPrTile ? p[e + 128 * k] : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int k = 0; k < 4; k++) any |= spoiled_in(w[k]);
                        if (!any) continue;
                        sh.spoiled = 1;
                        __threadfence_block();
#pragma unroll 1
                        for (int at = e; at < 8 * kPrTile && at < e + 4 * 128; at += 128) {
                            uint4 x = p[at];
                            if (clear_spoiled(x)) p[at] = x;
                        }
                    }
                }
                fence_async_smem();
            }
#pragma unroll
            for (int b = 0; b < 2; b++) {                     // the product of the first 64 keys begins under the last
                float sum = 0.0f;
                if (b > 0 || i > 0) sum = weigh(&v[64 * b], la_s + 32 * b, c, m);
                const bool grown = sum > kPrLimit || m == -INFINITY;      // of this row: the others' stay as they are, bit for bit
                if (__any_sync(0xffffffffu, grown)) {
                    float mx[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) mx[k] = __uint_as_float(v[64 * b + k]);
#pragma unroll
                    for (int j = 4; j < 60; j += 8)
#pragma unroll
                        for (int k = 0; k < 4; k++) mx[k] = max3(mx[k], __uint_as_float(v[64 * b + j + 2 * k]), __uint_as_float(v[64 * b + j + 2 * k + 1]));
#pragma unroll
                    for (int k = 0; k < 4; k++) mx[k] = fmaxf(mx[k], __uint_as_float(v[64 * b + 60 + k]));
                    const float m1 = grown ? fmaxf(m, max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * c) : m, f = m1 == -INFINITY ? 1.0f : exp2_fast(m - m1);
                    m = m1;
                    l *= f;
                    if (i > 0 || b > 0) {
                        // the products so far are done: those of the tile before in order ahead of S
                        if (b > 0 && !(ok = wait(sh.first_done[half], i))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int d = 0; d < kLatV; d += 16) {
                            float o[16];
                            tmem_ld16(la_o + d, o);
#pragma unroll
                            for (int j = 0; j < 16; j++) o[j] *= f;
                            tmem_st16(la_o + d, o);
                        }
                    }
                    sum = weigh(&v[64 * b], la_s + 32 * b, c, m);
                }
                l += sum;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mb_arrive(&sh.p_ready[half][b]);
            }
            if (!ok) break;
        }
        if (ok && mine > 0) ok = wait(sh.o_full[half], 0);
        if (ok && __any_sync(0xffffffffu, r < n)) {
            tc_fence_after();
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const bool spoiled = sh.spoiled != 0;
            float *part = kParts ? parts + ((size_t)blockIdx.x * splits + blockIdx.y) * kPrPart + (r - row0) * 16 : nullptr;
            // 32 columns at a time; rows of out go through where the queries were, so that a warp stores whole ones
            uint4 *stage = reinterpret_cast<uint4 *>(sm + half * kPrQBoxes * kPrBox) + 512 * q;
#pragma unroll 1
            for (int b = 0; b < kLatV; b += 32) {
                uint32_t o[32];
#pragma unroll
                for (int j = 0; j < 32; j++) o[j] = 0;
                if (mine > 0) {
                    tmem_ld16_nowait(la_o + b, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
                    tmem_ld16_nowait(la_o + b + 16, *reinterpret_cast<uint32_t(*)[16]>(&o[16]));
                    tmem_wait_ld();
                }
                if (spoiled && r < n)                         // what was cleared, for the rows that see it
#pragma unroll 1
                    for (int k = least; k < lim; k++) {
                        const uint16_t *p = a.kv + (size_t)(k0 + k) * a.kv_stride + (size_t)h * a.kv_head + kLatK + b;
#pragma unroll
                        for (int j = 0; j < 32; j++) {
                            const uint32_t u = p[j];
                            if ((u & 0x7F80u) == 0x7F80u) o[j] = __float_as_uint(__uint_as_float(o[j]) + bf16_bits_to_f32(u));
                        }
                    }
                if (kParts) {
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (r < n)
                            *reinterpret_cast<uint4 *>(part + (size_t)(b + (j & 4) * 4) * kPrBlock + 4 * (j & 3)) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const float x = __uint_as_float(o[8 * j + 2 * k]) * inv, y = __uint_as_float(o[8 * j + 2 * k + 1]) * inv;
                            const __nv_bfloat162 z = l == 0.0f ? __floats2bfloat162_rn(0.0f, 0.0f) : __floats2bfloat162_rn(x, y);
                            w[k] = *reinterpret_cast<const uint32_t *>(&z);
                        }
                        stage[16 * lane + ((b / 8 + j) ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
            }
            if (!kParts) {
                uint4 *to = reinterpret_cast<uint4 *>(a.out + ((size_t)(t0 + r - lane) * a.H + h) * kLatV) + (lane & 15);
#pragma unroll 4
                for (int i = lane >> 4; i < min(32, n - (r - lane)); i += 2) to[(size_t)i * a.H * (kLatV / 8)] = stage[16 * i + ((lane & 15) ^ (i & 7))];
            }
            if (kParts && r < n) {
                part += (size_t)kPrBlock * kLatV - (r - row0) * 15;
                part[0] = isnan(l) && m == -INFINITY ? 0.0f : m;      // not one without keys
                part[kPrBlock] = l;
            } else if (a.lse && r < n) {
                a.lse[(size_t)(t0 + r) * a.H + h] = (m + log2f(l)) * kLatLn2;
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPrRegsLast));
        if (warp < kPrWarpLoad) {
            // ---------------- products of a half: with values, then its scores of the tile after, in order, so that the weights
            // may lie over the scores.  A warp a half: while one looks for its next operands the other's products run
            // (one warp for both 949 us, 8192 tokens x 56 heads).
            const uint32_t ids = idesc(1, kPrTile), idv = idesc(1, kLatV) | (1u << 16);     // V with its columns contiguous
            const int half = uniform(warp - kPrWarpMma), mine = uniform(half ? tiles1 : tiles0), others = uniform(half ? tiles0 : tiles1);
            constexpr uint32_t box = kPrBox >> 4;
            const uint32_t sm_q = desc_lo(saddr(sm)) + (uint32_t)half * kPrQBoxes * box, sm_kv = desc_lo(saddr(ring), 0);
            const uint32_t S = kPrTmS + kPrTile * half, O = kPrTmO + kLatV * half;
            // a tile's keys or values are free when both halves are done with them; this one speaks for one that has no such tile
            auto done = [&](uint64_t *b, int i) {
                umma_commit_warp(b);
                if (i >= others) umma_commit_warp(b);
            };
            if (mine > 0 && wait(sh.q_full[half], 0)) {
                bool ok = true;
#pragma unroll 1
                for (int i = -1; ok && i < mine; i++) {
                    // in turn, the first half first: in step both would wait for products, then both for exponentials
                    const int turn = half ? i + 1 : i;        // the other's that has to be through
                    if (turn >= 0 && others > 0 && turn <= others && !(ok = wait(sh.turn[half], turn))) break;
                    if (i >= 0) {
                        const uint32_t s0 = slot_of(i, kPrQBoxes), s1 = slot_of(i, kPrQBoxes + 1), lo = min(s0, s1);
                        const uint32_t B = sm_kv + lo * box + ((max(s0, s1) - lo) * box << 16);
                        if (!(ok = wait(sh.v_full[i & 1], i >> 1))) break;
#pragma unroll
                        for (int b = 0; b < 2; b++) {
                            if (!(ok = wait(sh.p_ready[half][b], i))) break;
                            tc_fence_after();
#pragma unroll
                            for (int k = 0; k < 4; k++)
                                umma_ts_warp(O, S + 32 * b + 8 * k, B + (uint32_t)((4 * b + k) * 16 * 128 >> 4), idv, i > 0 || b > 0 || k > 0);
                            if (b == 0) umma_commit_warp(&sh.first_done[half]);
                        }
                        if (!ok) break;
                        done(&sh.v_empty[i & 1], i);
                        if (i == mine - 1) {
                            umma_commit_warp(&sh.o_full[half]);
                            if (lane == 0) mb_arrive(&sh.turn[half ^ 1]);
                            break;
                        }
                    }
                    const int j = i + 1;
                    uint32_t B[kPrQBoxes];
#pragma unroll
                    for (int b = 0; b < kPrQBoxes; b++) B[b] = sm_kv + slot_of(j, b) * box;
                    if (!(ok = wait(sh.k_full[j & 1], j >> 1))) break;
                    tc_fence_after();
#pragma unroll
                    for (int b = 0; b < kPrQBoxes; b++) {
                        if (b == kPrQBoxes - 1 && lane == 0) mb_arrive(&sh.turn[half ^ 1]);     // the other gets ready under the last ones
#pragma unroll
                        for (int k = 0; k < 4; k++) umma_warp(S, sm_q + b * box + 2 * k, B[b] + 2 * k, ids, b > 0 || k > 0);
                    }
                    umma_commit_warp(&sh.s_full[half]);
                    done(&sh.k_empty[j & 1], j);
                }
            }
            __syncwarp();
            umma_commit_warp(&sh.drain[half]);                 // every issued MMA done before the dealloc
            mb_wait_warp(&sh.drain[half], 0);
        } else if (warp == kPrWarpLoad) {
            // ---------------- loads
            auto load_q = [&](int half) {
                mb_expect_tx_warp(&sh.q_full[half], kPrQBoxes * kPrBox);
                for (int b = 0; b < kPrQBoxes; b++)
                    tma3d_warp(sm + (half * kPrQBoxes + b) * kPrBox, &mq, 64 * b, h, t0 + row0 + kPrRows * half, &sh.q_full[half]);
            };
            const int n = uniform(tiles), tok0 = uniform(k0);
            int k_loads = 0, v_loads = 0;
            if (tiles0 > 0) load_q(0);
#pragma unroll 1
            for (int i = 0; i < n; i++) {
                // slots: the keys' were the last of the keys and the values of the tile before the last, the values' the first two
                // of the keys of the last
                if (i >= 2 && !wait(sh.v_empty[i & 1], (i >> 1) - 1)) break;
                const int tok = tok0 + kPrTile * i;
                mb_expect_tx_warp(&sh.k_full[i & 1], kPrQBoxes * kPrBox);
#pragma unroll
                for (int b = 0; b < kLatK / 64; b++) tma3d_warp(ring + slot_of(i, b) * kPrBox, &mkv, 64 * b, h, tok, &sh.k_full[i & 1]);
                tma2d_warp(ring + slot_of(i, kLatK / 64) * kPrBox, &mr, 0, tok, &sh.k_full[i & 1]);
                k_loads++;
                if (i == 0 && tiles1 > 0) load_q(1);
                if (i >= 1 && !wait(sh.k_empty[(i - 1) & 1], (i - 1) >> 1)) break;
                // the values' first columns to the lower slot of the two
                const int s0 = slot_of(i, kPrQBoxes), s1 = slot_of(i, kPrQBoxes + 1);
                mb_expect_tx_warp(&sh.v_full[i & 1], 2 * kPrBox);
                tma3d_warp(ring + min(s0, s1) * kPrBox, &mkv, kLatK, h, tok, &sh.v_full[i & 1]);
                tma3d_warp(ring + max(s0, s1) * kPrBox, &mkv, kLatK + 64, h, tok, &sh.v_full[i & 1]);
                v_loads++;
            }
            // the block's shared memory stays until its last copies have landed, when another role gave up too
            for (int i = max(0, k_loads - 2); i < k_loads; i++) mb_wait_warp(&sh.k_full[i & 1], (uint32_t)(i >> 1) & 1u);
            for (int i = max(0, v_loads - 2); i < v_loads; i++) mb_wait_warp(&sh.v_full[i & 1], (uint32_t)(i >> 1) & 1u);
            if (tiles0 > 0) mb_wait_warp(&sh.q_full[0], 0);
            if (tiles1 > 0 && k_loads > 0) mb_wait_warp(&sh.q_full[1], 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kPrWarpMma) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(512));
}

// The join of a block's parts: a thread 16 columns of a row.
__global__ void __launch_bounds__(kPrBlock) prompt_join_kernel(const PromptArgs a, const int blocks, const int splits, const float *parts, const PromptPlace *places)
{
    pdl_wait();
    pdl_trigger();
    const PromptPlace place = places[blockIdx.x];
    const int r = threadIdx.x, group = blockIdx.y;
    if (r >= place.rows) return;
    const float *from = parts + (size_t)blockIdx.x * splits * kPrPart, *ml = from + (size_t)kPrBlock * kLatV + r;
    float m[kPrMaxSplits], l[kPrMaxSplits], M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int p = 0; p < kPrMaxSplits; p++) {
        m[p] = p < splits ? ml[p * kPrPart] : -INFINITY;
        l[p] = p < splits ? ml[p * kPrPart + kPrBlock] : 0.0f;
        M = fmaxf(M, m[p]);
    }
    float o[16] = {};
#pragma unroll
    for (int p = 0; p < kPrMaxSplits; p++) {
        if (p >= splits) break;
        const float f = m[p] == -INFINITY ? 0.0f : exp2_fast(m[p] - M);
        L = fmaf(f, l[p], L);
        const float4 *x = reinterpret_cast<const float4 *>(from + p * kPrPart + ((size_t)group * kPrBlock + r) * 16);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float4 v = x[j];
            o[4 * j] = fmaf(f, v.x, o[4 * j]);
            o[4 * j + 1] = fmaf(f, v.y, o[4 * j + 1]);
            o[4 * j + 2] = fmaf(f, v.z, o[4 * j + 2]);
            o[4 * j + 3] = fmaf(f, v.w, o[4 * j + 3]);
        }
    }
    const size_t row = (size_t)(place.token + r) * a.H + blockIdx.x / blocks;
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const __nv_bfloat162 x = L == 0.0f ? __floats2bfloat162_rn(0.0f, 0.0f) : __floats2bfloat162_rn(o[2 * j] * inv, o[2 * j + 1] * inv);
        w[j] = *reinterpret_cast<const uint32_t *>(&x);
    }
    uint4 *to = reinterpret_cast<uint4 *>(a.out + row * kLatV + 16 * group);
    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (a.lse && group == 0) a.lse[row] = (M + log2f(L)) * kLatLn2;
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs &a, cudaStream_t s)
{
    CUtensorMap mq{}, mkv{}, mr{};
    // without keys nothing is loaded by the last two
    const bool keys = a.S > 0;
    if (!map16x3(&mq, a.q, (uint64_t)a.T, (uint64_t)a.q_stride, (uint64_t)a.H, (uint64_t)a.q_head, kLatK + kLatR, 1, kPrRows) ||
        !map16x3(&mkv, keys ? a.kv : a.q, keys ? (uint64_t)a.S : 1, (uint64_t)a.kv_stride, (uint64_t)a.H, (uint64_t)a.kv_head, kLatK + kLatV, 1,
                 kPrTile) ||
        !map16s(&mr, keys ? a.rope_key : a.q, keys ? (uint64_t)a.S : 1, kLatR, (uint64_t)a.rope_stride, kPrTile))
        return cudaErrorInvalidValue;
    const cudaError_t allowed = once_a_device([] {
        // the shares of setmaxnreg are of the launch's registers: with another count they would never be there
        cudaFuncAttributes fa{};
        for (const void *kernel : {(const void *)prompt_kernel<false>, (const void *)prompt_kernel<true>}) {
            if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs != kPrRegs) return cudaErrorInvalidConfiguration;
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrSmem);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    });
    if (allowed != cudaSuccess) return allowed;
    const int blocks = a.seq_start ? a.T / (2 * kPrRows) + std::min(a.n_seq, a.T)
                                   : a.n_seq == 1 ? (a.T + 2 * kPrRows - 1) / (2 * kPrRows) : a.n_seq;
    // parts of the keys while the blocks leave SMs without one, of four tiles at least by the sequences' average, or as if half of all
    // keys were one sequence's (4 prompts of 55 tokens in all behind up to 2561: 15.7 us, by the average alone 22.4; 12 of 300 behind up to
    // 1000, 3 heads, 13.8 and 19.0; even ones take the same either way); their sums are where the absorbed form has its own
    const int items = blocks * a.H;
    int splits = std::min(std::min(num_sms(), kMaxShares) / items, std::max(a.S / std::min(a.n_seq, a.T) / (4 * kPrTile), a.S / (8 * kPrTile)));
    splits = std::max(1, std::min(splits, kPrMaxSplits));
    const int sorted = splits == 1 && items > num_sms() && a.n_seq <= kPrSorted && blocks <= kPrSorted && (size_t)a.S * a.H * (kLatK + kLatV) * 2 <= kPrSortedBytes;
    float *parts = latent_parts(a.ws);
    PromptPlace *places = reinterpret_cast<PromptPlace *>(a.ws + kCtrOffset + kCtrBytes);
    timing_begin("latent_prompt", s);
    cudaError_t err = launch_pdl(splits > 1 ? prompt_kernel<true> : prompt_kernel<false>, dim3((unsigned)items, (unsigned)splits), dim3(kPrThreads), kPrSmem, s, a, mq, mkv, mr, blocks, sorted, parts, places);
    count_launch();
    timing_end("latent_prompt", s);
    if (err != cudaSuccess || splits == 1) return err;
    timing_begin("latent_prompt_join", s);
    err = launch_pdl(prompt_join_kernel, dim3((unsigned)items, kPrGroups), dim3(kPrBlock), 0, s, a, blocks, splits, (const float *)parts, (const PromptPlace *)places);
    count_launch();
    timing_end("latent_prompt_join", s);
    return err;
}

}  // namespace k3moe
