// The wait of roles that run on whole warps, the halves of a cluster's barrier, and
// copies of 3-D boxes.
#pragma once

#include "ops.cuh"

namespace tmmo {

// Bounded wait of a whole converged warp on an mbarrier phase.  The roles that
// issue copies and MMAs run on whole warps, one elected lane issuing: their
// operands then live in uniform registers, from which the instructions take
// them (from a branch of one lane an MMA took about 140 cycles to issue and a
// copy about 100).
template <bool CLUSTER_SCOPE = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const TcWatch& w)
{
    long long t0 = 0;
    for (;;) {
        const bool done = CLUSTER_SCOPE ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
        if (__all_sync(0xffffffffu, done))
            return true;
        const long long now = clock64();
        if (t0 == 0)
            t0 = now;
        const bool late = now - t0 > w.budget;
        if (late)
            tc_raise(w);
        if (__any_sync(0xffffffffu, late || *w.abort_flag))
            return false;
    }
}

// warp_wait for what may lie any number of K steps ahead: the budget counts anew
// whenever *progress, which the block's copies move on, has changed.
__device__ __forceinline__ bool warp_wait_behind(uint32_t bar, uint32_t parity, const TcWatch& w,
                                                 const volatile int* progress)
{
    long long t0 = clock64();
    int seen = *progress;
    for (;;) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
            return true;
        const long long now = clock64();
        const int at = *progress;
        if (at != seen) {
            seen = at;
            t0 = now;
        }
        const bool late = now - t0 > w.budget;
        if (late)
            tc_raise(w);
        if (__any_sync(0xffffffffu, late || *w.abort_flag))
            return false;
    }
}

// The two halves of cluster_sync(), each by every thread of the cluster.
__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// For a wait that spans `steps` K steps (a whole tile's): a step takes well below
// 2^-18 of the budget.
__device__ __forceinline__ TcWatch patient(TcWatch w, int steps)
{
    w.budget *= 1 + (steps >> 18);
    return w;
}

// tma_load_2d_pair of a 3-D box.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

}  // namespace tmmo
