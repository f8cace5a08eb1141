// nvfp4_tc.cuh -- building blocks of the tcgen05 kernels: bounded mbarrier
// waits, shared-memory operand descriptors, tensor-memory loads and the even
// split of a step sequence over the CTAs.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace nvfp4 {

// A wait suspends the thread (no spinning) for up to kTcSuspendNs per try,
// and gives up after kTcTries tries (about 2 s): far beyond any legitimate
// wait, which lasts a few microseconds.
constexpr uint32_t kTcSuspendNs = 1000000u;
constexpr int kTcTries = 2000;

__device__ __forceinline__ uint32_t tc_smem(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Byte offset of 16-byte chunk `c` (0..7) of row `r` in a K-major tile with
// the 128-byte swizzle: rows of 128 bytes, chunk index XOR (row mod 8).
__device__ __forceinline__ uint32_t sw128(uint32_t r, uint32_t c) { return r * 128u + ((c ^ (r & 7u)) << 4); }

// Shared-memory matrix descriptor of a K-major, 128-byte-swizzled operand:
// start address >> 4 (bits 0-13), leading byte offset 16 (unused by this
// layout), stride byte offset 1024 (8 rows of 128 bytes, bits 32-45),
// descriptor version 1 (bits 46-47), swizzle mode 128 bytes (bits 61-63).
__device__ __forceinline__ uint64_t tc_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void mbar_init(uint32_t mb, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(mb), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t mb) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(mb) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t mb, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mb), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t mb, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(mb), "r"(parity), "n"(kTcSuspendNs) : "memory");
  return done != 0;
}

__device__ __forceinline__ bool mbar_test(uint32_t mb, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(mb), "r"(parity) : "memory");
  return done != 0;
}

// Bounded wait for the phase of `parity`; gives up early once another role of
// the CTA has raised `fail`, and raises it itself when the limit (about 2 s)
// runs out.  SLEEP_NS = 0: suspending tries, for the waits on the critical
// path; otherwise the warp sleeps that long between tests, which keeps
// waiting warps that are off the critical path from taking issue slots from
// the dequantizing ones.
template <int SLEEP_NS = 0>
__device__ __forceinline__ bool tc_wait(uint32_t mb, uint32_t parity, volatile int *fail) {
  if (mbar_test(mb, parity)) return true;
  constexpr int kTries = SLEEP_NS ? 2000000000 / SLEEP_NS : kTcTries;
  for (int it = 0; it < kTries; ++it) {
    if (SLEEP_NS) {
      __nanosleep(SLEEP_NS);
      if (mbar_test(mb, parity)) return true;
    } else if (mbar_try(mb, parity)) {
      return true;
    }
    if (*fail) return false;
  }
  *fail = 1;
  return false;
}

// The first wait of a CTA's MMA thread under the test hook: gives up after
// `tries` tries (0: at once) and raises `fail`.
__device__ __forceinline__ bool tc_wait_tries(uint32_t mb, uint32_t parity, volatile int *fail, int tries) {
  for (int it = 0; it < tries; ++it)
    if (mbar_try(mb, parity)) return true;
  *fail = 1;
  return false;
}

// The same wait without the early exit: used after a failure to let this
// CTA's own copies and MMAs in flight finish before it leaves.
__device__ __forceinline__ void tc_drain(uint32_t mb, uint32_t parity) {
  for (int it = 0; it < kTcTries && !mbar_try(mb, parity); ++it) {
  }
}

// Tiles of the work sequence: CTA c covers steps [c T / G, (c+1) T / G); the
// CTA holding step g is floor(((g+1) G - 1) / T).
__host__ __device__ __forceinline__ int64_t tc_first_step(int64_t c, int64_t T, int64_t G) { return c * T / G; }
__host__ __device__ __forceinline__ int64_t tc_cta_of(int64_t g, int64_t T, int64_t G) { return ((g + 1) * G - 1) / T; }

// 16 consecutive fp32 columns of tensor memory, one lane per thread (the
// warp's 32 lanes); the caller waits with tcgen05.wait::ld.
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
               "%12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                 "=r"(r[15])
               : "r"(taddr));
}

}  // namespace nvfp4
