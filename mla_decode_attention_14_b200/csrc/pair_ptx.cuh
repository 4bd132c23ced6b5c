// pair_ptx.cuh -- inline-PTX wrappers for kernels whose two CTAs drive one tensor-core tile
// (cta_group::2): TMEM allocation by both CTAs, MMAs issued by the pair's leader (rank 0), commits
// that arrive in both CTAs, and TMA loads that complete on the leader's barrier.
#pragma once

#include "sm100_ptx.cuh"

namespace mla {
namespace sm100 {

// One warp of EACH CTA of the pair calls these.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst_smem)),
                 "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Bounded waits without a suspend-time hint: with one, a warp was seen to wake up
// to about a thousand cycles after its phase, which the short dependent steps of a pair kernel cannot hide.
// Same contract as mbar_wait (false: *abort was set, or the bound passed and *abort is now set).
__device__ __forceinline__ bool mbar_poll(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (mbar_test(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int k = 0; k < 64; ++k)
            if (mbar_test(bar, parity)) return true;
        if (*abort) return false;
        if (clock64() - t0 > kSpinCycles) {
            *abort = 1;
            return false;
        }
    }
}
// For a whole converged warp: all lanes look at once (by lane 0 with a shuffle, a ready phase took 250 cycles).
__device__ __forceinline__ bool warp_poll(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_poll(bar, parity, abort));
}

// Arrive on a barrier of either CTA given by its shared::cluster address, in order with this thread's own
// accesses. What it announces lies in this CTA's shared memory, written through fence.proxy.async, and is
// read there by the tensor core, so no fence over the cluster goes with it (a release at cluster scope
// measured about 2,000 cycles here, with loads in flight).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// True in one lane of a converged warp. The compiler knows the region behind it to be warp-uniform and
// keeps descriptors in uniform registers; behind `lane == 0` it moves each operand of each MMA there
// (measured: 77 cycles an MMA instead of the tensor core's own 32 for 128 x 128 x 16).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
    return p != 0;
}

// D[tmem of both CTAs] (+)= A B over the pair: each CTA holds half of A's rows and half of B's columns
// at the same shared-memory offsets.
__device__ __forceinline__ void mma_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
// Arrive on the barrier at this offset in BOTH CTAs once every MMA this thread issued has completed.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_addr(bar)), "h"((uint16_t)3) : "memory");
}
// The same for this CTA's barrier alone.
__device__ __forceinline__ void mma_commit_pair_local(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// 3-D tiled TMA load into this CTA's shared memory that completes on `bar`, a shared::cluster address
// in either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;"
        ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}
// Programmatic dependent launch: the kernel may have been put on the GPU before the one ahead of it in the
// stream has ended; here that one has, and its writes are visible. (Such kernels read by plain loads, not
// __ldg: what they read is not constant for as long as they run, only from here on.)
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Brings a box into L2 only.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

}  // namespace sm100
}  // namespace mla
