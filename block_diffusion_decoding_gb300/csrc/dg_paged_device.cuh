// Device helpers of the paged attention kernels, beside those of dg_device.cuh.
#pragma once

#include "dg_device.cuh"

namespace dg {

// mbar_wait with the clock read only once it has lasted: a wait that a few
// polls satisfy, as most in a running pipeline are, pays for those alone.
// CLUSTER: acquires what the other CTA of a pair released.  SLEEP: nanoseconds
// between polls, for roles with time to spare whose polls would take issue
// slots from the others of their SM.
template <bool CLUSTER = false, int SLEEP = 0>
DG_DEVICE bool mbar_wait_poll(uint64_t *bar, uint32_t parity, WsHeader *ws, int where,
                              uint64_t limit_ns = kWaitLimitNs)
{
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        uint32_t ok;
        if (CLUSTER)
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(smem_u32(bar)), "r"(parity)
                : "memory");
        else
            ok = mbar_try_wait(bar, parity) ? 1u : 0u;
        if (ok) return true;
        if (SLEEP > 0) __nanosleep(SLEEP);
        if ((it & 63u) == 0) {
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > limit_ns) {
                report_error(ws, DG_ERR_TIMEOUT, where);
                return false;
            }
        }
    }
}

DG_DEVICE uint64_t policy_evict_normal()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Registers per thread of a warpgroup (4 warps, all of which execute it):
// raised from, or given back to, those the block was launched with.
template <int N>
DG_DEVICE void reg_inc()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
DG_DEVICE void reg_dec()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A barrier of THREADS threads, apart from __syncthreads()'s: those that wait at
// it, and those that only arrive.
template <int THREADS>
DG_DEVICE void start_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

template <int THREADS>
DG_DEVICE void start_arrive()
{
    asm volatile("bar.arrive 1, %0;" ::"n"(THREADS) : "memory");
}

// cluster_sync_all() in two halves.
DG_DEVICE void cluster_arrive_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

DG_DEVICE void cluster_wait_all()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A word of shared memory given by its cluster address.
DG_DEVICE void st_cluster(uint32_t cluster_addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

// True in one lane of a converged warp, the same one every time.  A role whose
// whole warp runs its loop and only issues under this keeps its operands
// uniform over the warp, which is how the tensor instructions take them; a
// role run by one lane alone pays a move and a wait for each operand.
DG_DEVICE bool elect_lane()
{
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}

// 32 lanes x 32 bit, 8 consecutive columns per thread.
DG_DEVICE void tmem_st8(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

}  // namespace dg
