// mbarriers with bounded waits, for kernels that wait for asynchronous copies or
// for other warps of their CTA.  Each translation unit that includes this
// header has its own wait status, registered with the library's registry, so
// amsim_device_errors reports a wait that gave up in any of them.
#pragma once

#include "amsim_internal.h"

namespace amsim {
namespace tc {

constexpr unsigned long long kWaitLimitNs = 2000000000ULL;   // 2 s

static __device__ unsigned int g_wait_timeouts;

namespace {
int tu_wait_status(unsigned int *bits, int clear)
{
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_wait_timeouts, sizeof(v)) != cudaSuccess) return AMSIM_ECUDA;
    *bits |= v;
    if (clear && v) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(zero)) != cudaSuccess) return AMSIM_ECUDA;
    }
    return AMSIM_OK;
}
// No wait here is on another CTA's flag: the settable limit has nothing to set.
int tu_flag_wait_limit(long long) { return AMSIM_OK; }
[[maybe_unused]] const bool g_tu_wait_words = register_wait_words(&tu_wait_status, &tu_flag_wait_limit);
}  // namespace

__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool bar_try(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ unsigned long long now_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Wait for the phase of `bar` with parity `parity`; after kWaitLimitNs the
// timeout is recorded, `aborted` set, and every later wait of the thread
// returns at once, so the thread runs to its end.  The timer is read once in
// 1024 polls: a read takes longer than the waits between the roles of a CTA.
static __device__ __noinline__ bool bar_wait_slow(uint64_t *bar, uint32_t parity)
{
    unsigned long long t0 = 0;
    for (uint32_t i = 1; !bar_try(bar, parity); ++i) {
        if (i & 1023) continue;
        const unsigned long long t = now_ns();
        if (!t0) t0 = t;
        if (t - t0 > kWaitLimitNs) {
            atomicOr(&g_wait_timeouts, (unsigned)AMSIM_WAIT_COPY);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, bool &aborted)
{
    if (aborted) return false;
    if (bar_try(bar, parity)) return true;
    aborted = !bar_wait_slow(bar, parity);
    return !aborted;
}

// The same by a whole warp, all of whose lanes get one answer, so that its
// control flow stays uniform.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, bool &aborted)
{
    if (aborted) return false;
    if (__all_sync(0xFFFFFFFFu, bar_try(bar, parity))) return true;
    aborted = !__all_sync(0xFFFFFFFFu, bar_wait_slow(bar, parity));
    return !aborted;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte
// aligned; completes on `bar`.
__device__ __forceinline__ void copy_bytes(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}
// Shared-memory writes of this thread before become visible to copies issued after.
__device__ __forceinline__ void fence_staged() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace tc
}  // namespace amsim
