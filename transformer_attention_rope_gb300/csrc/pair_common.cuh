// pair_common.cuh -- inline-PTX building blocks of the kernels on CTA pairs
// (prefill_pair.cu, cache_pair.cu): clusters of two, arrivals on the leader's barriers,
// bounded waits that end together, and tcgen05 with cta_group::2.
#pragma once

#include <stdint.h>

#include "device_common.cuh"

namespace apex {

// ---------------------------------------------------------------- cluster
__device__ __forceinline__ uint32_t cluster_rank()
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

// Arrive on the barrier at the same shared-memory offset in the leader CTA.
// Default (release, CTA-scope) semantics: a cluster-scope release here costs
// about a microsecond per arrival on the softmax critical path.
__device__ __forceinline__ void arrive_leader(uint32_t local_bar)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local_bar), "r"(0));
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}

// Bounded wait on a local barrier (some receive arrivals from the peer CTA).
// On time-out the status word and the CTA's abort flag (shared memory) are
// set and the wait returns; once the flag is set, later waits of the CTA that
// do not complete at once give up at their first timer check, so a broken
// pipeline drains in about one time-out.
__device__ __forceinline__ void pair_wait(uint32_t bar, uint32_t parity, const WaitCtl &wc, volatile uint32_t *abort)
{
    if (mbar_try_wait(bar, parity)) return;
    uint64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return;
        if ((n & 255u) == 0) {
            if (*abort) return;
            const uint64_t now = global_timer_ns();
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > wc.timeout_ns) {
                *abort = 1u;
                report_status(wc.status, kStatusWaitTimeout);
                return;
            }
        }
    }
}

// ---------------------------------------------------------------- tcgen05 over both CTAs
// The mbarrier at this shared-memory offset in each CTA receives one arrival once every
// cta_group::2 operation this thread issued before has completed.
__device__ __forceinline__ void commit_pair(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     bar),
                 "h"((uint16_t)3)
                 : "memory");
}

// D[tmem] (+)= A[smem desc] * B[smem desc], M and B split between the CTAs
__device__ __forceinline__ void mma_ss_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc]
__device__ __forceinline__ void mma_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                            uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

}  // namespace apex
