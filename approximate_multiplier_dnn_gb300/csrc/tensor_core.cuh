// Wrappers for the tensor-core kernels of the exact operators: CTA pairs,
// tensor-map copies, and the tcgen05 matrix instructions with their
// tensor-memory accumulators.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "bounded_wait.cuh"

namespace amsim {
namespace tc {

// ------------------------------------------------------------------ CTA pairs
// The kernels run in clusters of two CTAs on neighbouring SMs, which the
// matrix instructions treat as one: rank 0 leads.
__device__ __forceinline__ uint32_t pair_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Address of `p` (an address of this CTA's shared memory) in the leader's.
__device__ __forceinline__ uint32_t leader_addr(const void *p)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
    return r;
}

// All threads of both CTAs; memory written before is seen after.
__device__ __forceinline__ void pair_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrive on a barrier of the pair by its cluster address.
__device__ __forceinline__ void bar_arrive_at(uint32_t addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Box at (x, y) of a 2-D tensor map into this CTA's shared memory; completes on
// a barrier of the pair, given by its cluster address.
__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// A staged box from shared memory to (x, y) of a 2-D tensor map; elements
// outside the tensor are not written.
__device__ __forceinline__ void store_box(const CUtensorMap *map, int x, int y, const void *src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(smem_addr(src))
                 : "memory");
}
__device__ __forceinline__ void stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The thread's committed stores have read their shared memory / are done.
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ------------------------------------------------------------------ tcgen05
// A warp of each CTA of the pair allocates `COLS` columns of its SM's tensor
// memory and writes their address to shared memory; the same warp frees them.
template <int COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "n"(COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

template <int COLS>
__device__ __forceinline__ void tmem_free(uint32_t addr)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand descriptor of a 128-byte swizzled tile (rows of 128
// bytes, atoms of 8 rows): start address, leading and stride byte offsets in
// units of 16 bytes, descriptor version 1, swizzle mode 2.
// K-major operands (64 bf16 of K per row): stride = next 8 rows, leading unused.
// MN-major operands (64 bf16 of M or N per row): stride = next 8 steps of K,
// leading = next 64 rows of M or N.
// The low word alone moves with the address, by 1 per 16 bytes.
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t leading) { return addr >> 4 | leading >> 4 << 16; }
__host__ __device__ constexpr uint32_t desc_high(uint32_t stride) { return stride >> 4 | 1u << 14 | 2u << 29; }

// Instruction descriptor: fp32 accumulator, bf16 A and B, their majors (0 K,
// 1 MN), the M x N shape.
__host__ __device__ constexpr uint32_t instr_desc(int m, int n, int a_mn, int b_mn)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (uint32_t)(n >> 3) << 17 |
           (uint32_t)(m >> 4) << 24;
}

// D (tensor memory of both CTAs) = A B, + D when `acc`; 16 steps of K, one
// issuing thread of the leader.  Each CTA holds its half of A's rows, its half
// of B's columns, and the accumulator of its rows.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_low, uint32_t a_high, uint32_t b_low, uint32_t b_high,
                                    uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_low), "r"(a_high), "r"(b_low), "r"(b_high), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

// `bar` of both CTAs gets one arrival when every matrix instruction issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// 32 accumulator columns of the calling thread's row (its lane of tensor
// memory); the whole warp loads together, so it comes together first.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32])
{
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

// Loads issued before are done; `r` passes through, so that no use of it is
// scheduled above the wait.
__device__ __forceinline__ void tmem_load_wait(uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.wait::ld.sync.aligned;"
        : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
        :
        : "memory");
}

}  // namespace tc
}  // namespace amsim
