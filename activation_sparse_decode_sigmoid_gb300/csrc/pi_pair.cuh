// CTAs of a cluster that work on one tile: who is who, barriers, and the end after a failure.
#pragma once

#include <stdint.h>

#include "pi_tc.cuh"

namespace pi {
namespace {

__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// address of the first CTA's copy of a shared-memory object
__device__ __forceinline__ uint32_t in_first(uint32_t addr)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// After a failure: copies and MMAs in flight finish within microseconds; the
// CTA stays for a bounded time that covers them.
__device__ __forceinline__ void linger()
{
    const uint64_t t0 = gtimer();
    while (gtimer() - t0 < 5000000ull) {
    }
}

} // namespace
} // namespace pi
