// gemm_common.cuh -- what the linear layers' kernels share: 2-D TMA loads and thread-block clusters.
#pragma once

#include "device_common.cuh"
#include "ring_end.h"

namespace fdpp {

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// mbar_wait for hand-overs of a few hundred cycles: the clock, whose reading takes as long, is first read
// after 64 tries.
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity)
{
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            const uint64_t now = global_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > FDPP_WAIT_NS) return false;
        }
    }
}

// Barrier of every thread of the cluster; the arrive releases and the wait acquires this
// thread's (and, through them, the CTA's) shared-memory writes at cluster scope.
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Address of the same shared-memory location in cluster member `rank`.
__device__ __forceinline__ uint32_t dsmem_addr(uint32_t saddr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}

__device__ __forceinline__ float4 ld_dsmem_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_dsmem_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// The barriers of a ring's stages, for what is under way when a CTA ends (ring_end.h). bytes: of one CTA's copies.
struct RingBarriers {
    uint32_t bars, bytes;

    __device__ __forceinline__ void announce(uint32_t stage) { mbar_arrive_expect_tx(bars + 8 * stage, bytes); }
    __device__ __forceinline__ void excuse(uint32_t stage)
    {
        asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bars + 8 * stage), "r"(bytes) : "memory");
    }
    __device__ __forceinline__ void landed(uint32_t stage, uint32_t parity)
    {
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(bars + 8 * stage, parity) && global_ns() - t0 < 100000000ull) {
        }
    }
    // the last turn of a ring of `depth` barriers that completed `count` phases in all, whose arrivals are on their way
    __device__ __forceinline__ void arrived(uint32_t count, uint32_t depth)
    {
        for (uint32_t i = ring_last_turn(count, depth); i < count; ++i) landed(i % depth, (i / depth) & 1u);
    }
};

// The producer's last act: every stage that it filled has been used, so that neither copies nor the tensor cores' arrivals
// are under way when the CTA ends (false: the wait ran out).
__device__ __forceinline__ bool ring_used(uint32_t empty, uint32_t issued, uint32_t stages)
{
    for (uint32_t i = ring_last_turn(issued, stages); i < issued; ++i)
        if (!mbar_wait_short(empty + 8 * (i % stages), (i / stages) & 1u)) return false;
    return true;
}

}  // namespace fdpp
