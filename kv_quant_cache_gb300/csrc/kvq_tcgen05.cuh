// kvq_tcgen05.cuh -- the fifth-generation tensor-core primitives that the
// tiled attention kernel uses: tensor-memory allocation and access, shared
// memory and instruction descriptors, the matrix instruction with its first
// operand in shared or in tensor memory, completion on an mbarrier, and
// bounded waits.  Inline PTX for sm_103a.
#pragma once

#include <stdint.h>

#include "kvq_tma.cuh"

namespace kvq {
namespace tc {

// ---- waits -------------------------------------------------------------------
// No wait is endless: after `polls` polls (of the launch; one at least) or
// kClocks cycles the waiter raises the CTA's `dead` flag and returns false, and
// every other waiter of the CTA that polls sees the flag.  (The cycle counter, not
// the nanosecond timer: a read of that one takes longer than most waits.)
constexpr uint32_t kPolls = 1u << 24;      // unless kvq_set_tile_wait_limit says otherwise
constexpr long long kClocks = 2000000000;  // about 1 s

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* dead,
                                     uint32_t polls) {
  if (tma::mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t i = 1; i < polls; ++i) {
    if (tma::mbar_test(bar, parity)) return true;
    if ((i & 63u) == 0 && (*dead || clock64() - t0 > kClocks)) break;
  }
  *dead = 1;
  return false;
}

// The same by a whole warp, which stays converged.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* dead,
                                          uint32_t polls) {
  return __all_sync(kFullMask, wait(bar, parity, dead, polls));
}

// What a role that gives up still has in flight: waits until it has landed,
// bounded by the same clock whatever the launch's limit.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  for (uint32_t i = 1; i < kPolls && !tma::mbar_test(bar, parity); ++i) {
    if ((i & 63u) == 0 && clock64() - t0 > kClocks) break;
  }
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---- tensor memory -------------------------------------------------------------
// One warp allocates all 512 columns of the SM and later frees them.
__device__ __forceinline__ void alloc512(uint32_t smem_slot) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_slot)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc512(uint32_t tmem) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 lanes x 32 columns of 32 bits: thread l of the warp gets (puts) lane
// 32 (warp % 4) + l, columns c .. c + 31.
__device__ __forceinline__ void ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// 32 lanes x 16 (8) columns, as ld32.
__device__ __forceinline__ void ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ld8(uint32_t (&r)[8], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// By the number of columns.
__device__ __forceinline__ void ld(uint32_t (&r)[32], uint32_t addr) { ld32(r, addr); }
__device__ __forceinline__ void ld(uint32_t (&r)[16], uint32_t addr) { ld16(r, addr); }
__device__ __forceinline__ void ld(uint32_t (&r)[8], uint32_t addr) { ld8(r, addr); }

// ---- descriptors -----------------------------------------------------------------
// Shared-memory matrix of 128-byte rows with the 128-byte swizzle, base
// 1024-byte aligned.  Groups of 8 rows are 1024 bytes apart.  Where the rows
// run along the product's inner dimension ("k rows": the operand's outer
// dimension is contiguous, 64 values to a row), blocks of 64 outer values are
// `block` bytes apart; where the inner dimension is contiguous `block` is not
// used (1).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t block) {
  uint64_t d = (addr >> 4) & 0x3fff;
  d |= (uint64_t)((block >> 4) & 0x3fff) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version of this architecture
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}

// bf16 x bf16 -> fp32, M = 128; k_rows_b: the second operand's rows run along
// the inner dimension (k_rows_a: the first's).
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, bool k_rows_b,
                                                         bool k_rows_a = false) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((k_rows_a ? 1u : 0u) << 15) |
         ((k_rows_b ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// D[tmem] (+)= A B, one K = 16 step.  The whole warp calls, converged, and one
// elected lane issues (always the same one, which commit() relies on): the
// operands then are warp-uniform for the compiler.  Issued from a branch of
// one lane instead, each instruction took about 75 cycles to prepare, longer
// than it takes to run.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// Arrives on `bar` once all matrix instructions issued so far are done.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar)
      : "memory");
}

}  // namespace tc
}  // namespace kvq
