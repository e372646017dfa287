// tensor.cuh -- inline-PTX wrappers for the fifth-generation tensor cores on sm_103a: tensor memory,
// tcgen05.mma with its descriptors, tiled TMA loads, and mbarrier waits that end.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "../ptx.cuh"
#include "spec_verify.h"

namespace spec {
namespace context {

// ---- tensor memory: 128 lanes x 512 columns of 32 bits
__device__ __forceinline__ void tmem_alloc(uint32_t to, uint32_t columns) {  // one whole warp
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The warp's loads are done; `r` is named so that nothing that uses it moves ahead of this.
__device__ __forceinline__ void wait_loads(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), 
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), 
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), 
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void wait_loads(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), 
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes, a lane a thread.
__device__ __forceinline__ void tmem_load32(uint32_t (&r)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// ---- tcgen05.mma, kind::f16, one CTA: D[128 x n] (fp32, tensor memory) (+)= A[128 x 16] B[16 x n]
// The low word of a shared-memory operand in rows of 128 bytes, swizzled over 8 rows (1024 bytes); `lead`: bytes
// between groups of 64 columns of an operand whose rows run along the product's inner axis.  A step of
// 16 bytes is 1.
__device__ __forceinline__ uint32_t operand(uint32_t at, uint32_t lead) { return (at & 0x3ffff) >> 4 | lead >> 4 << 16; }
__device__ __forceinline__ uint64_t descriptor(uint32_t low) {
    constexpr uint32_t kHigh = 1024 >> 4 | 1u << 14 | 2u << 29;  // 1024 bytes between groups of 8 rows; version; swizzle
    return static_cast<uint64_t>(kHigh) << 32 | low;
}
// `type`: 0 fp16, 1 bf16; `rows_inner`: B's rows run along the inner axis (its columns are contiguous).
__host__ __device__ constexpr uint32_t instruction(uint32_t type, uint32_t n, bool rows_inner) {
    return 1u << 4 | type << 7 | type << 10 | (rows_inner ? 1u << 16 : 0u) | n >> 3 << 17 | 128u >> 4 << 24;
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(instr), "r"(static_cast<uint32_t>(add))
        : "memory");
}
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t instr, bool add) {  // A from tensor memory
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(instr), "r"(static_cast<uint32_t>(add))
        : "memory");
}
// The barrier gets an arrival when every mma that this thread has issued is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// ---- TMA and barriers
__device__ __forceinline__ void tma_load3(uint32_t to, const CUtensorMap *map, int x, int y, int z, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(to),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_load4(uint32_t to, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(to),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint64_t policy_evict_normal() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}
__device__ __forceinline__ void arrive(uint32_t bar, uint32_t n = 1) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
// What generic stores wrote to shared memory is there for the tensor cores and TMA.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#ifdef SPEC_TEST_HOOKS
constexpr int kWaitTries = SPEC_SPIN_LIMIT;  // test builds: 25 ms
#else
constexpr int kWaitTries = 1 << 20;  // each suspends the thread for 1.5 us: 1.6 s, far beyond any wait that ends
#endif

// (mbar_try_wait takes no hint of a time to suspend for: with one of a microsecond the thread slept past the phase's end.)

// A thread waits for a barrier's phase; false after kWaitTries, or once another of the CTA has given up.  Nothing spins
// for ever: on false the caller leaves its loop.
__device__ __forceinline__ bool wait_alone(uint32_t bar, uint32_t parity, volatile int *gave_up, uint32_t *status) {
    bool done = ptx::mbar_try_wait(bar, parity);
    for (int i = 1; !done && i < kWaitTries; ++i) {
        if ((i & 63) == 0 && *gave_up) return false;
        done = ptx::mbar_try_wait(bar, parity);
    }
    if (!done) {
        *gave_up = 1;
        atomicOr(status, SPEC_DEV_TIMEOUT);
    }
    return done;
}
// The same for a whole warp, which sleeps between its tries where it is not in a hurry: warps that ask all the time
// take shared memory's ports from those that work.
template <bool HURRY>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int *gave_up, uint32_t *status) {
    bool done = ptx::mbar_try_wait(bar, parity);
    for (int i = 1; !done && i < kWaitTries; ++i) {
        if ((i & 63) == 0 && *gave_up) break;
        if (!HURRY) __nanosleep(100);
        done = ptx::mbar_try_wait(bar, parity);
    }
    done = __all_sync(0xffffffffu, done);
    if (!done && !*gave_up) {
        *gave_up = 1;
        atomicOr(status, SPEC_DEV_TIMEOUT);
    }
    return done;
}

}  // namespace context
}  // namespace spec
