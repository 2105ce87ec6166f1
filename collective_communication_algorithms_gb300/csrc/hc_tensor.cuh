// hc_tensor.cuh -- tensor-core building blocks: matrix instructions whose
// operands lie in shared memory and whose sums lie in tensor memory (TMEM),
// tiled bulk copies, and the descriptors of both.  Internal; not installed.
#pragma once

#include <cuda.h>

#include "hc_ops.cuh"

namespace hc {
namespace {

// ---------------------------------------------------------------------------
// tensor memory: 128 lanes of 512 columns of 32 bits
// ---------------------------------------------------------------------------
// G: blocks that work on a tile together (1, or a cluster of 2, both of which
// then call this).
template <int G>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {
    if constexpr (G == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int G>
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
    if constexpr (G == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}
// 32 columns of the warp's 32 lanes: a thread has its lane's.  The loads and the
// wait for them are one statement, so that nothing that uses them can be moved
// between the two.
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(at)
        : "memory");
}
// 16 columns.
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tensor_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---------------------------------------------------------------------------
// operands in shared memory, written by tiled copies with 128-byte swizzling:
// rows of 128 bytes (64 bf16), eight rows a pattern, tiles on 1024 bytes.
//   along the sum's direction: a row is one m (or n) and 64 k; 8 rows to the
//     next pattern is 1024 bytes; 16 k further on is 32 bytes;
//   across it: a row is one k and 64 m (or n); the next 8 k are 1024 bytes on,
//     the next 64 m are `group` bytes on; 16 k further on is 2048 bytes.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t operand_along(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
__device__ __forceinline__ uint64_t operand_across(uint32_t addr, uint32_t group) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(group >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// bf16 operands, binary32 sums; m x n of one instruction.
__host__ __device__ constexpr uint32_t product_shape(bool a_across, bool b_across, int m, int n) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (a_across ? 1u << 15 : 0u) | (b_across ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 |
           (uint32_t)(m >> 4) << 24;
}
// sums[m][n] (+)= a[m][0..15] b[n][0..15], by one thread.  With G = 2 each block
// holds half of a's m and of b's n at the same places of its shared memory, and
// the sums of its m; a thread of the first block issues.
template <int G>
__device__ __forceinline__ void product16(uint32_t sums, uint64_t a, uint64_t b, uint32_t shape, bool add) {
    if constexpr (G == 1)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(sums),
            "l"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(sums),
            "l"(a), "l"(b), "r"(shape), "r"((uint32_t)add)
            : "memory");
}
// An arrival on `m` (of both blocks, if G = 2 and `both`) once all products
// that this thread issued are done.
template <int G>
__device__ __forceinline__ void products_arrive(uint64_t* m, bool both = true) {
    if constexpr (G == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(m)) : "memory");
    else if (both)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                         smem_addr(m)),
                     "h"((uint16_t)3)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(m)) : "memory");
}

// One thread of a warp that is together here: matrix instructions take their
// operands from registers that a warp shares, which the compiler only keeps
// them in where the warp has not parted.
__device__ __forceinline__ bool elected() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}

// ---------------------------------------------------------------------------
// barriers of the first block of a cluster of two (G = 2), or of the block
// itself, which then uses no cluster instruction
// ---------------------------------------------------------------------------
template <int G>
__device__ __forceinline__ uint32_t first_blocks(const uint64_t* m) {
    uint32_t a = smem_addr(m);
    if constexpr (G > 1) asm("mapa.shared::cluster.u32 %0, %0, 0;" : "+r"(a));
    return a;
}
template <int G>
__device__ __forceinline__ void first_arrive(uint64_t* m) {
    if constexpr (G == 1) mbar_arrive(m);
    else asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(first_blocks<G>(m)) : "memory");
}
// mbar_wait_quick for arrivals from both blocks.
template <int G>
__device__ __forceinline__ bool first_wait(uint64_t* m, unsigned parity, unsigned long long limit_ns) {
    if constexpr (G == 1) return mbar_wait_quick(m, parity, limit_ns);
    unsigned long long t0 = 0;
    for (bool first = true;; first = false) {
        unsigned ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_addr(m)), "r"(parity)
            : "memory");
        if (ok) return true;
        const unsigned long long t = global_ns();
        if (first) t0 = t;
        else if (t - t0 > limit_ns) return false;
    }
}

// ---------------------------------------------------------------------------
// tiled copies; x counts elements along the innermost direction and is a
// multiple of 16 (32 bytes) in every use
// ---------------------------------------------------------------------------
// G = 2: the barrier may be the cluster's first block's (first_blocks).
template <int G>
__device__ __forceinline__ void tile_g2s(void* dst, const CUtensorMap* map, int x, int y, uint32_t m) {
    if constexpr (G == 1)
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                         smem_addr(dst)),
                     "l"(map), "r"(x), "r"(y), "r"(m)
                     : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                smem_addr(dst)),
            "l"(map), "r"(x), "r"(y), "r"(m)
            : "memory");
}
template <int G>
__device__ __forceinline__ void tile_g2s(void* dst, const CUtensorMap* map, int x, int y, int z, uint32_t m) {
    if constexpr (G == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                smem_addr(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(m)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                smem_addr(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(m)
            : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

}  // namespace
}  // namespace hc
