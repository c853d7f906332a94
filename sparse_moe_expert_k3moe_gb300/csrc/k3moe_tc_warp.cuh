// k3moe_tc_warp.cuh -- more inline-PTX helpers of tensor-core kernels (sm_103a), for the
// operators whose operands also live in tensor memory: MMA issue, commit and tile loads by a
// converged warp, A operands in and stores to tensor memory, prefetches to the L2; and a
// tensor map of a matrix whose rows are slices of wider ones.
#pragma once
#include "k3moe_tc.cuh"

namespace k3moe {
namespace {

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
// The same boxes and ranges brought to the L2 only.
__device__ __forceinline__ void prefetch2d(const CUtensorMap *m, int c0, int c1)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(m), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void prefetch_bulk(const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
// Forms that a converged warp executes whole, one elected lane issuing: descriptors and
// addresses stay uniform over the warp, which makes the issue of a small MMA several times
// cheaper than from inside a single lane's branch (measured 160 clocks apart there for
// 128 x 64 x 16 MMAs that take 32).
// A descriptor's halves: `lo` has the address (and the leading offset), the upper half is a
// constant of the layout, so that one addition makes the next descriptor.  In a cluster a
// shared address holds the block's rank above its low 18 bits, which are all that go in.
constexpr uint32_t kDescSw128 = (1024u >> 4) | (1u << 14) | (2u << 29);      // 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t leading = 16) { return ((addr >> 4) & 0x3FFFu) | ((leading >> 4) << 16); }
template <uint32_t kHi = kDescSw128>
__device__ __forceinline__ void umma_warp(uint32_t dtmem, uint32_t a, uint32_t b, uint32_t id, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(dtmem),
        "r"(a), "r"(b), "r"(id), "r"(acc), "r"(kHi)
        : "memory");
}
__device__ __forceinline__ void mb_expect_tx_warp(uint64_t *b, uint32_t bytes)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(saddr(b)),
        "r"(bytes)
        : "memory");
}
__device__ __forceinline__ void tma2d_warp(void *dst, const CUtensorMap *m, int c0, int c1, uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];\n\t}" ::"r"(saddr(dst)),
        "l"(m), "r"(c0), "r"(c1), "r"(saddr(bar))
        : "memory");
}
// A operand in tensor memory (two 16-bit elements of K a column), B in shared memory.
template <uint32_t kHi = kDescSw128>
__device__ __forceinline__ void umma_ts_warp(uint32_t dtmem, uint32_t atmem, uint32_t b, uint32_t id, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(dtmem),
        "r"(atmem), "r"(b), "r"(id), "r"(acc), "r"(kHi)
        : "memory");
}
__device__ __forceinline__ void umma_commit_warp(uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(saddr(bar))
        : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
        "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld8_nowait(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// 16-bit matrix of `rows` rows of `cols` elements, `stride` elements apart: boxes of 64
// columns x box_rows rows, 128-byte swizzle; what a box has outside reads as zero.
inline bool map16s(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, uint64_t stride,
                   uint32_t box_rows)
{
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {stride * 2};
    const cuuint32_t box[2] = {64u, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// f's result, from the first call on the current device (a kernel's attributes are the
// device's), whichever threads call; f's type tells one use from another.
template <typename F> cudaError_t once_a_device(F f)
{
    constexpr int kMaxDevices = 64;
    static std::once_flag flag[kMaxDevices];
    static cudaError_t result[kMaxDevices];
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::call_once(flag[dev], [&] { result[dev] = f(); });
    return result[dev];
}

}  // namespace
}  // namespace k3moe
