// Roles of whole warps in a warp-specialised kernel: an elected lane, bounded waits on
// barriers, copies into rings.
#pragma once

#include "moe_sm100.cuh"

namespace moe {
namespace sm100 {

// One lane of a converged warp, the same one each time. Roles run as whole warps and elect a
// lane around what it issues: the compiler then keeps addresses and descriptors in uniform
// registers (four MMAs and a commit of one thread in a divergent branch issue in 275
// cycles, elected in 165).
MOE_DEV bool elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
// Barriers by their 32-bit shared-memory addresses: the roles' loops are bound by their own
// instructions, and generic pointers cost several of them each time.
MOE_DEV bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// Whether the phase is complete, without any waiting.
MOE_DEV bool test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// try_wait for one that will wait: asleep until the phase completes or some 20 us have passed, instead of taking turns
// from the warps that work.
MOE_DEV bool try_wait_asleep(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(bar), "r"(parity), "r"(20000u) : "memory");
  return ok != 0;
}
// Bounded: about two seconds, after which every role winds down and the error word is set.
static __device__ __noinline__ bool slow_wait(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
  const long long t0 = clock64();
  while (!__all_sync(0xFFFFFFFFu, try_wait_asleep(bar, parity))) {
    if (__any_sync(0xFFFFFFFFu, *abort != 0)) return false;
    if (__any_sync(0xFFFFFFFFu, clock64() - t0 > 4000000000LL)) {
      set_error(err, kDevTimeout);
      *abort = 1;
      return false;
    }
  }
  return true;
}
// The same for a role that has no registers left for a call, nor time for a vote: each lane waits by itself. Lanes may
// give up apart, so that nobody stops here: a role goes on to its end with whatever there is, and after the first wait
// that ran out (or an abort elsewhere) no other one waits.
MOE_DEV void lane_wait(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
  if (!try_wait(bar, parity)) {
    const long long t0 = clock64();
#pragma unroll 1
    while (!try_wait_asleep(bar, parity) && !*abort)
      if (clock64() - t0 > 4000000000LL) {
        set_error(err, kDevTimeout);
        *abort = 1;
      }
  }
  __syncwarp();
}
// A wait by a whole warp, which goes on or gives up as one.
MOE_DEV bool warp_wait(uint32_t bar, uint32_t parity, int* err, volatile int* abort) {
  if (__all_sync(0xFFFFFFFFu, try_wait(bar, parity))) return true;
  return slow_wait(bar, parity, err, abort);
}
MOE_DEV void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
MOE_DEV void expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(bar), "r"(bytes) : "memory");
}
MOE_DEV void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}
MOE_DEV void load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(bar) : "memory");
}
MOE_DEV void load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}

// After an abort: the copies of a ring's last stages land before the CTA exits.
MOE_DEV void land(uint64_t* full, int stages, uint32_t issued, int* err, volatile int* abort) {
  if ((threadIdx.x & 31) || !*abort) return;
  for (uint32_t q = issued > (uint32_t)stages ? issued - stages : 0; q < issued; ++q)
    mbar_wait(&full[q % stages], (q / stages) & 1, err, abort, 20000000LL, false);
}

}  // namespace sm100
}  // namespace moe
