// PTX of the orthogonalisation's tensor-core kernels (tc.cu has its own): mbarriers with bounded
// waits, fences, tensor memory, and tcgen05.mma on fp16 operands in 128-byte swizzled shared memory.
//
// Every wait is bounded: a kernel whose wait runs out sets a bit of the device's error word,
// stops, waits (bounded) for what it has in flight and frees its tensor memory.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace mk {

constexpr unsigned long long kWaitNs = 1000000000ull;  // 1 s bound on every wait
// bits of the error word, as the MTTKRP's kernels set them
constexpr uint32_t kStatusTimeoutTma = 1u << 0;
constexpr uint32_t kStatusTimeoutMma = 1u << 2;
constexpr uint32_t kStatusTimeoutEpi = 1u << 3;
constexpr uint32_t kStatusTimeoutDrain = 1u << 4;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ unsigned long long gtimer() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ uint32_t mbar_try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok;
}

// Blocking probe: the thread is suspended (no issue slots used) until the phase
// completes or about kSuspendNs elapse.
constexpr uint32_t kSuspendNs = 20000;

__device__ __forceinline__ uint32_t mbar_try_wait_suspend(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return ok;
}

// Wait for the phase of `bar` with the given parity; false if the CTA was aborted or the wait
// exceeded kWaitNs (then the CTA is aborted and `code` recorded).  The clock is first read after
// one suspension has run out, so a wait that ends within the first one costs no timer read.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                             uint32_t* status, uint32_t code) {
    if (mbar_try_wait(bar, parity)) return true;
    unsigned long long t0 = 0;
    bool timing = false;
    while (true) {
        if (mbar_try_wait_suspend(bar, parity)) return true;
        if (*abort_flag) return false;
        if (!timing) {
            t0 = gtimer();
            timing = true;
        } else if (gtimer() - t0 > kWaitNs) {
            *abort_flag = 1;
            atomicOr(status, code);
            return false;
        }
    }
}

// The same whatever the abort flag (for work in flight).
__device__ __forceinline__ bool wait_drain(uint64_t* bar, uint32_t parity, uint32_t* status) {
    unsigned long long t0 = 0;
    bool timing = false;
    while (!mbar_try_wait_suspend(bar, parity)) {
        if (!timing) {
            t0 = gtimer();
            timing = true;
        } else if (gtimer() - t0 > kWaitNs) {
            atomicOr(status, kStatusTimeoutDrain);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// K-major, 128-byte swizzle descriptor: 8-row groups of 128-byte rows, 1024
// bytes apart (high word; the low word is the start address >> 4 and LBO = 1)
constexpr uint64_t kDescSw128Hi = ((uint64_t)1 << 16)            // leading byte offset (unused)
                                | ((uint64_t)(1024 >> 4) << 32)  // stride byte offset: 8 rows x 128 B
                                | ((uint64_t)1 << 46)            // descriptor version
                                | ((uint64_t)2 << 61);           // 128-byte swizzle

__device__ __forceinline__ uint32_t sdesc128_lo(uint32_t saddr) {
    return (uint32_t)kDescSw128Hi | ((saddr & 0x3FFFFu) >> 4);
}

// MN-major operand: 64-row parts of M (128 bytes, contiguous in memory) x 64 contraction
// indices, 8 KB apart, which is the canonical MN-major layout with a 128-byte swizzle: 8-row
// groups of K 1024 bytes apart (stride offset), the 64-row parts of M 8192 bytes apart (leading
// offset); a slice of 16 contraction indices advances the start address by 16 rows (2048 bytes).
constexpr uint32_t kDescMnLo = (uint32_t)((8192 >> 4) << 16);   // leading byte offset: M halves

__device__ __forceinline__ uint32_t sdesc128mn_lo(uint32_t saddr) { return kDescMnLo | ((saddr & 0x3FFFFu) >> 4); }

// D (+)= A B of fp16 operands by the low words of their descriptors, on one CTA or a pair; issued
// by the lane whose `leader` is not 0
template <int kCtas>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc, uint32_t leader) {
    if constexpr (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
            "mov.b64 da, {%1, %3};\n\t"
            "mov.b64 db, {%2, %3};\n\t"
            "setp.ne.b32 p, %5, 0;\n\t"
            "setp.ne.b32 e, %6, 0;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, p;\n\t}\n" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"((uint32_t)(kDescSw128Hi >> 32)), "r"(idesc), "r"(acc), "r"(leader));
    else
        asm volatile(
            "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
            "mov.b64 da, {%1, %3};\n\t"
            "mov.b64 db, {%2, %3};\n\t"
            "setp.ne.b32 p, %5, 0;\n\t"
            "setp.ne.b32 e, %6, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}\n" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"((uint32_t)(kDescSw128Hi >> 32)), "r"(idesc), "r"(acc), "r"(leader));
}

// arrive on `bar` (of both CTAs) when that lane's MMAs so far are done
template <int kCtas>
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t leader) {
    if constexpr (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
            "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}\n" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3), "r"(leader)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
            "r"(leader)
            : "memory");
}

// Registers of the warpgroup's threads: up only within what the block was launched with.
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace mk
