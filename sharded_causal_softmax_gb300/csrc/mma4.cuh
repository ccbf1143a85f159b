// Pieces of warp-specialised tensor-core kernels beside ptx.cuh: MMAs issued
// four k-steps at a time, register moves between warpgroups, a barrier test
// that never waits.
#pragma once

#include "ptx.cuh"

namespace sca {

// Registers a thread of the warpgroup from here on (all its warps execute it).
template <int N>
SCA_INLINE void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
SCA_INLINE void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// Four k-steps of one product, issued by one elected lane of the converged
// warp: A from tensor memory (8 columns a step) or shared memory (AS a
// step), B from shared memory (BS a step; descriptor units of 16 bytes).
// One election and one set of adds (in a descriptor's lower word, which holds
// the address) for four MMAs: with one each, the warp
// took about 130 clk an MMA to issue, twice what the tensor pipe needs.
template <int BS>
SCA_INLINE void umma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3, l, l1, l2, l3, h;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 {l, h}, %2;\n\tadd.s32 l1, l, %5;\n\tadd.s32 l2, l, %6;\n\tadd.s32 l3, l, %7;\n\t"
      "mov.b64 b1, {l1, h};\n\tmov.b64 b2, {l2, h};\n\tmov.b64 b3, {l3, h};\n\t"
      "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accum), "n"(BS), "n"(2 * BS), "n"(3 * BS)
      : "memory");
}
template <int AS, int BS>
SCA_INLINE void umma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b1, b2, b3, a1, a2, a3;\n\t.reg .b32 l, l1, l2, l3, h;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 {l, h}, %2;\n\tadd.s32 l1, l, %5;\n\tadd.s32 l2, l, %6;\n\tadd.s32 l3, l, %7;\n\t"
      "mov.b64 b1, {l1, h};\n\tmov.b64 b2, {l2, h};\n\tmov.b64 b3, {l3, h};\n\t"
      "mov.b64 {l, h}, %1;\n\tadd.s32 l1, l, %8;\n\tadd.s32 l2, l, %9;\n\tadd.s32 l3, l, %10;\n\t"
      "mov.b64 a1, {l1, h};\n\tmov.b64 a2, {l2, h};\n\tmov.b64 a3, {l3, h};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum), "n"(BS), "n"(2 * BS), "n"(3 * BS), "n"(AS), "n"(2 * AS), "n"(3 * AS)
      : "memory");
}

// One arrival for the whole warp, after everything its lanes did before (each
// lane having fenced its own writes for the proxies that read them).  A
// hundred lanes arriving one by one on one barrier are as many atomic
// operations in a row on one word: 300 to 500 clk of latency at each hand-over.
SCA_INLINE void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

SCA_INLINE uint32_t globaltimer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}

// mbar_wait in fewer instructions: the role warps' loops run once per tile
// between the other warps' long straight-line code, so that they mostly wait
// for instructions.  Gives up as mbar_wait does, by setting *abort; the kernel
// reports that once, at its end (report_abort).
SCA_INLINE bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = globaltimer_lo();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_lo() - t0 > static_cast<uint32_t>(kWaitLimitNs)) *abort = 1;
    if (*abort) return false;
  }
  return true;
}
SCA_INLINE bool wait_all_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort));
}
SCA_INLINE void report_abort(const volatile int* abort, int* status) {
  if (threadIdx.x == 0 && *abort) report(status, SCA_ERR_TIMEOUT);
}

// has the phase with this parity completed? (never waits)
SCA_INLINE bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

SCA_INLINE void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace sca
