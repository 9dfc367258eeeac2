// PTX building blocks of the tensor-core kernels (sm_100a): mbarriers with
// bounded waits, TMA tile loads, TMEM allocation and the tcgen05 matrix
// instructions, with the descriptors they take.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fpstok {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// The loading and the issuing warp run as whole warps with the same values in
// every lane, and single-thread instructions elect one lane themselves: TMA
// and tcgen05 operands live in uniform registers, which the compiler can only
// use where it sees that a warp agrees.  Issued from inside a one-lane branch
// a product took 80 cycles of its warp.
#define FPS_ELECT ".reg .pred elected;\n\telect.sync _|elected, 0xffffffff;\n\t"

// A value that every lane of the warp holds alike.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// ---------------------------------------------------------------- mbarriers

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// By a whole warp: one arrival.
__device__ __forceinline__ void mbar_arrive_one(uint32_t bar) {
  asm volatile("{\n\t" FPS_ELECT "@elected mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("{\n\t" FPS_ELECT "@elected mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
               "r"(bytes)
               : "memory");
}
// A poll sleeps in hardware for up to kWaitNs; polled without that, the waits
// took half of the softmax warps' issue slots.
constexpr uint32_t kWaitNs = 20000;
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kWaitNs)
      : "memory");
  return ok != 0;
}

// Every wait ends: after so many polls as `polls` says, or once another warp of
// the block has given up, it returns false and the caller leaves its loop.
struct WaitState {
  int gave_up, polls;
};
// Of one lane.  Lanes may end with different answers, and what follows a wait
// is for whole warps (TMEM reads and writes, ballots), so only mbar_wait_warp
// calls it.
__device__ __forceinline__ bool mbar_wait_lane(uint32_t bar, uint32_t parity, volatile WaitState* state) {
#pragma unroll 1
  for (int i = 0; !mbar_try(bar, parity); ++i)
    if (i >= state->polls || state->gave_up) {
      state->gave_up = 1;
      return false;
    }
  return true;
}

// By a whole warp, with the same answer for every lane.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile WaitState* state) {
  return __all_sync(0xffffffffu, mbar_wait_lane(bar, parity, state));
}

// After a wait gave up: for what is still in flight and ends on `bar`, whether
// or not the other waits do.
__device__ __forceinline__ void mbar_land_warp(uint32_t bar, uint32_t parity, volatile WaitState* state) {
  volatile WaitState own;
  own.gave_up = 0;
  own.polls = state->polls;
  mbar_wait_warp(bar, parity, &own);
}

// ---------------------------------------------------------------- TMA

// By a whole warp: one box.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile("{\n\t" FPS_ELECT
               "@elected cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
               "%4, %5}], [%2];\n\t}" ::"r"(dst),
               "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Generic writes to shared memory before, reads of them by TMA or the tensor core after.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---------------------------------------------------------------- TMEM

// By one whole warp; the base address is written to *slot.
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes, one lane per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// The wait for loaded values, with the registers as operands: no use of them
// moves before it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
        "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
        "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld8(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}

// ---------------------------------------------------------------- matrix instructions

// Shared-memory operand in 128-byte swizzled panels: rows of 128 bytes (64
// 16-bit values), 8-row groups 1024 bytes apart, panels of 64 values
// `panel_bytes` apart.  The low word of its descriptor holds the address and
// the panel stride in units of 16 bytes, so a step adds bytes / 16 to it: 2
// for 16 values along the rows (K-major), 128 for 16 rows (MN-major); the
// high word is the same for all.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr, uint32_t panel_bytes) {
  return (addr >> 4) | ((panel_bytes >> 4) << 16);
}

// Instruction descriptor: 16-bit operands, float32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t mma_desc(bool bf16, bool a_mn, bool b_mn, int n, int m = 128) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D[tmem] (+)= A B over 64 values of the sum, by a whole warp with one
// election for its four instructions: A and B in shared memory (low descriptor
// words), each along its rows (2 per step) or across them (128 per step).
template <int kA, int kB>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t" FPS_ELECT ".reg .pred p, t;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "@elected tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t"
      "add.s64 x, x, %6;\n\tadd.s64 y, y, %7;\n\t"
      "@elected tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, x, %6;\n\tadd.s64 y, y, %7;\n\t"
      "@elected tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t"
      "add.s64 x, x, %6;\n\tadd.s64 y, y, %7;\n\t"
      "@elected tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, t;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(kDescHigh), "n"(kA), "n"(kB)
      : "memory");
}
// The same with A as 32 columns of 16-bit pairs in TMEM and B across its rows.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t" FPS_ELECT ".reg .pred p, t;\n\t.reg .b64 y;\n\t.reg .b32 x;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "setp.eq.u32 t, 0, 0;\n\tmov.b64 y, {%2, %5};\n\tmov.b32 x, %1;\n\t"
      "@elected tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\t"
      "add.s64 y, y, 128;\n\tadd.u32 x, x, 8;\n\t"
      "@elected tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
      "add.s64 y, y, 128;\n\tadd.u32 x, x, 8;\n\t"
      "@elected tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t"
      "add.s64 y, y, 128;\n\tadd.u32 x, x, 8;\n\t"
      "@elected tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, t;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(kDescHigh)
      : "memory");
}
constexpr uint32_t kRun = 64 * 128 >> 4;  // 64 rows on, in descriptor units

// Arrives on `bar` once every tcgen05 operation this warp issued before is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("{\n\t" FPS_ELECT
               "@elected tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
               : "memory");
}

}  // namespace fpstok
