// kda_tc.cuh -- helpers of the kernels whose warps take different roles around tcgen05
// products (softmax attention, the state-space scan).
#pragma once

#include "kda.h"
#include "kda_common.cuh"

namespace kda {

// A bounded wait that also gives up when another role has (ctl->abort, in shared memory).
template <class Ctl>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Ctl* ctl, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait_sleep(bar, parity, kSleepHintNs)) {
    if (*reinterpret_cast<volatile int*>(&ctl->abort)) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
      atomicCAS(err, 0, static_cast<int>(KDA_ERR_TIMEOUT));
      return false;
    }
  }
  return true;
}

// The same for a whole warp: true if every lane's wait ended.
template <class Ctl>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Ctl* ctl, int* err) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, ctl, err));
}

template <int REGS>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void regs_give() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// True in one lane of the warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(p));
  return p != 0;
}

// One K = 16 step, bf16: D (tmem, fp32) (+)= A * B with B in shared memory and A in
// shared memory (ss) or tensor memory (ts).  A descriptor is a low word (address
// and leading offset) plus a constant step, and a high word; putting it together
// inside keeps 16 steps' descriptors from being held in registers (or spilled).
template <uint32_t STEP_A, uint32_t STEP_B>
__device__ __forceinline__ void mma_ss_step(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "add.u32 x, %1, %2;\n\t"
      "add.u32 y, %3, %4;\n\t"
      "mov.b64 a, {x, %5};\n\t"
      "mov.b64 b, {y, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %6, p;\n\t}\n" ::"r"(d),
      "r"(a_lo), "n"(STEP_A), "r"(b_lo), "n"(STEP_B), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
template <uint32_t STEP_A, uint32_t STEP_B>
__device__ __forceinline__ void mma_ts_step(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t hi,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "add.u32 x, %1, %2;\n\t"
      "add.u32 y, %3, %4;\n\t"
      "mov.b64 b, {y, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %6, p;\n\t}\n" ::"r"(d),
      "r"(a_tmem), "n"(STEP_A), "r"(b_lo), "n"(STEP_B), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Pairs of fp32 in one operation (same rate per value, half the issue slots).
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 pair(const uint32_t& lo, const uint32_t& hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpair(f2 x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ void unpair(f2 x, uint32_t& lo, uint32_t& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(x));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace kda
