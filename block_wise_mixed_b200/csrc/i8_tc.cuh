// i8_tc.cuh -- tcgen05 / TMA / cluster helpers of the int8 kernels.
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace mpq {

// As in k_decode.cuh: bounded waits; the wait-test build gives up after 2 ms
// and its producers arm their barriers without issuing a copy.
#ifdef MPQ_WAIT_TEST
constexpr bool kI8WaitTest = true;
constexpr uint64_t I8_WAIT_NS = 2000000ull;
#else
constexpr bool kI8WaitTest = false;
constexpr uint64_t I8_WAIT_NS = 2000000000ull;
#endif

// Shared-memory operand, K-major, 128-byte swizzle: 8-row groups 1024 bytes
// apart, descriptor version 1, layout type 2.
__device__ __forceinline__ uint64_t i8_smem_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(1024u >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// Instruction descriptors, both operands K-major: s8 x s8 -> s32, and
// fp16 x fp16 -> fp32.
__host__ __device__ constexpr uint32_t i8_idesc(int M, int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t f16_idesc(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// KIND 0: i8, 1: f16.  PAIR: the two SMs of a cluster.
template <bool PAIR, int KIND>
__device__ __forceinline__ void i8_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
#define MPQ_I8_MMA(GROUP, K)                                                      \
    asm volatile(                                                                 \
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                         \
        "tcgen05.mma.cta_group::" GROUP ".kind::" K " [%0], %1, %2, %3, p;\n\t}"  \
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory")
    if (PAIR) {
        if (KIND == 0) MPQ_I8_MMA("2", "i8");
        else MPQ_I8_MMA("2", "f16");
    } else {
        if (KIND == 0) MPQ_I8_MMA("1", "i8");
        else MPQ_I8_MMA("1", "f16");
    }
#undef MPQ_I8_MMA
}

// One lane of the (converged) warp.  The MMA warp runs its loop as a whole and
// only issues from this lane, so that stages, phases and descriptors stay
// warp-uniform values: issued from a single-lane branch, each instruction's
// operands were moved over one by one and a stage took some 870 cycles.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}

// The four MMAs over 128 bytes of the contraction (32 bytes each) of operand
// tiles at shared addresses a and b.
template <bool PAIR, int KIND>
__device__ __forceinline__ void i8_mma4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
    const uint64_t da = i8_smem_desc(a), db = i8_smem_desc(b);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)   // 32 bytes = 2 units of the address field
        i8_mma<PAIR, KIND>(d, da + 2 * kk, db + 2 * kk, idesc, kk > 0 || accumulate ? 1u : 0u);
}

// Arrive on `bar` (PAIR: on the barrier at the same address in both CTAs)
// when the MMAs issued so far by this thread are done.
template <bool PAIR>
__device__ __forceinline__ void i8_commit(uint64_t* bar) {
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                     : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void i8_tmem_alloc(uint32_t* dst, uint32_t cols) {
    if (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <bool PAIR>
__device__ __forceinline__ void i8_tmem_free(uint32_t addr, uint32_t cols) {
    if (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void i8_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void i8_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 8 / 16 / 32 consecutive 32-bit columns of the warp's 32 lanes, completed by
// i8_tmem_wait().
__device__ __forceinline__ void i8_tmem_ld8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void i8_tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void i8_tmem_ld32(uint32_t taddr, uint32_t* r) {
    i8_tmem_ld16(taddr, r);
    i8_tmem_ld16(taddr + 16u, r + 16);
}
__device__ __forceinline__ void i8_tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Cluster of two.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// Arrive on a barrier of either CTA.  What it announces is the arriving CTA's
// own shared memory or TMEM, already made visible to the tensor cores by a
// proxy fence or tcgen05 fence, so no cluster-wide release is asked for: that
// costs a memory barrier of several hundred cycles on every arrival.
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same for data that the peer reads itself (after a wait with CLUSTER).
__device__ __forceinline__ void cluster_arrive_release(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A shared address of this CTA in the CTA of the given rank, and a load there.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t cluster_load(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Waits for the phase of the given parity, for at most about I8_WAIT_NS;
// false when that ran out.  The clock is read only after a while of polling:
// reading it first cost the MMA thread some 300 cycles a stage.  CLUSTER:
// arrivals may come from the peer CTA.
template <bool CLUSTER = false>
__device__ __forceinline__ bool i8_wait(uint64_t* bar, uint32_t parity) {
    uint64_t t0 = 0;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
            uint32_t ok;
            if (CLUSTER)
                asm volatile(
                    "{\n\t.reg .pred p;\n\t"
                    "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                    "selp.u32 %0, 1, 0, p;\n\t}"
                    : "=r"(ok)
                    : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)
                    : "memory");
            else
                ok = mbar_try_wait_sleep(bar, parity, 100000u);
            if (ok) return true;
        }
        const uint64_t t = global_timer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > I8_WAIT_NS) return false;
    }
}

// i8_wait by a whole warp: the same answer in every lane.
template <bool CLUSTER = false>
__device__ __forceinline__ bool i8_wait_warp(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, i8_wait<CLUSTER>(bar, parity));
}

// Tensor-map copies global -> own shared memory.  PAIR: completes on a
// barrier of either CTA of the cluster (bar: shared::cluster address).
template <bool PAIR>
__device__ __forceinline__ void i8_tma_load(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    if (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void i8_tma_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

__device__ __forceinline__ uint32_t i8_load_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// After an abort: gives copies and arrivals in flight, which no barrier of
// this CTA tracks any more, time to land before the memory is given up.
__device__ __forceinline__ void i8_settle() {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {}
}

}  // namespace mpq
