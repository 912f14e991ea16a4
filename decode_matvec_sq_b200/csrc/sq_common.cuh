// sq_common.cuh -- device helpers shared by the kernels of libsq (sm_100a).
//
// Thin wrappers over PTX: shared-memory mbarriers with a wall-clock bound on
// every wait, programmatic dependent launch control, status reporting and a
// few load / bit helpers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/sq.h"

namespace sq {

// Every spin on an mbarrier gives up after this long and reports SQ_ERR_TIMEOUT.
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count)
               : "memory");
}

// Makes initialised mbarriers visible to the async (TMA) proxy.
__device__ __forceinline__ void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Waits for the phase with the given parity to complete, at most limit_ns.
// false = ran out of time.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity,
                                          uint64_t limit_ns = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_ns() - t0 > limit_ns) return false;
  }
  return true;
}

// Programmatic dependent launch: wait for the preceding grid (and its memory),
// and allow the next grid in the stream to begin launching.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void set_status(int32_t* st, int32_t code) {
  if (st) atomicExch(st, code);
}

__device__ __forceinline__ int4 ldg_nc_v4(const void* p) {
  int4 v;
  asm volatile("ld.global.nc.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Four sign/mask bits (bit i = channel i) -> four bytes of 0 or 1.
__device__ __forceinline__ int expand_nibble(uint32_t bits) {
  return (int)(((bits & 0xFu) * 0x00204081u) & 0x01010101u);
}

// v = hi + lo for tf32 products: hi rounded to tf32's 11 bits, half a step away from
// zero, lo the exact rest, of which the tensor cores read 11 bits.  A value that would round
// to infinity (from 2^128 - 2^116 on) takes the largest finite hi: the bits grow with
// the magnitude, so a minimum for either sign does it.  (The adapters' shrink kernel on
// binary32 weights takes 19.4 us so, 20.4 with a saturating cvt, 19.9 with a clamp before it.)
// An infinity then has an infinite lo, a NaN a NaN.
__device__ __forceinline__ void cut_tf32(float v, uint32_t& hi, uint32_t& lo) {
  const uint32_t up = (uint32_t)__viaddmin_s32(__float_as_int(v), 0x1000, 0x7F7FFFFF);  // positive
  hi = min(up, 0xFF7FFFFFu) & 0xFFFFE000u;                                              // negative
  lo = __float_as_uint(v - __uint_as_float(hi));
}
__device__ __forceinline__ void cut_tf32(float v, float& hi, float& lo) {
  uint32_t h, l;
  cut_tf32(v, h, l);
  hi = __uint_as_float(h);
  lo = __uint_as_float(l);
}

}  // namespace sq
