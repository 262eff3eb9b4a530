// linear.cuh -- device helpers of linear attention's kernels.
#pragma once

#include "delta.cuh"
#include "linear.h"

namespace vssm {

// The waits of a role of a CTA: as wait_or_stop, in a loop that takes little
// code, of which these kernels' many roles have much: instructions that have to
// be fetched again cost the walk more than any other stall.  After one that has
// run out (ok is false then) the role waits for nothing any more.
// A try sleeps until the phase is over, or for about a microsecond.
__device__ __forceinline__ bool mbar_sleep_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0;
}

static __device__ __noinline__ bool lin_wait(const LinArgs& a, volatile int* stop, uint64_t* bar, uint32_t parity, bool forced) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_sleep_wait(bar, parity)) {
      if (!forced) return true;
      break;
    }
    if (i & 15) continue;
    if (*stop) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > a.wait_ns) break;
  }
  *stop = 1;
  atomicOr(a.status, kStatusTmaTimeout);
  return false;
}

struct LinWaiter {
  const LinArgs& a;
  volatile int* stop;
  bool ok = true;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity, bool forced = false) {
    if (ok && (forced || !mbar_try_wait(bar, parity))) ok = lin_wait(a, stop, bar, parity, forced);
  }
};

// Whether this is the lane of a warp that issues for it: the same one whenever all lanes ask.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// As umma (and with A in tensor memory, its rows in the lanes, two bf16 to a
// column), for a warp that goes through it together; the elected lane issues.
// Operands and predicate then come from the uniform registers that the
// instruction takes them from: a step takes 60 to 80 cycles to issue, with a lane
// picked by its number 95, and by a branch for it 110.
__device__ __forceinline__ void umma_one(uint32_t tmem_d, uint64_t desc_a, uint64_t desc_b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(desc_a), "l"(desc_b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_ta_one(uint32_t tmem_d, uint32_t tmem_a, uint64_t desc_b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(desc_b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Running sums of g, whose differences enter exp, as sums of two floats (48
// bits); doubles took the one warp that makes the gates longer than all else
// in a chunk (GB300 has two FP64 units an SM).
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
  const float hi = s + e;
  return Pair{hi, e - (hi - s)};
}
__device__ __forceinline__ Pair over_ln2(Pair a) {
  constexpr float kLog2eRest = (float)(1.44269504088896340736 - (double)kLog2e);
  const float p = a.hi * kLog2e;
  const float e = fmaf(a.hi, kLog2e, -p) + fmaf(a.hi, kLog2eRest, a.lo * kLog2e);
  const float hi = p + e;
  return Pair{hi, e - (hi - p)};
}
// 2^x to the MUFU's 2^-22; outside a float's range the power is 0 or infinite by itself.
__device__ __forceinline__ float exp2_of(Pair x) {
  const float p = ex2(x.hi);
  return x.hi > -126.0f && x.hi < 128.0f ? fmaf(p, x.lo * 0.6931471805599453f, p) : p;
}

// exp of either is 0; -inf would leave inf - inf
__device__ __forceinline__ float clamp_g(float g) { return g < -256.0f ? -256.0f : g; }

// The sum of g before a lane's four tokens of a chunk of 128, and over all of them, that one over ln 2.
__device__ __forceinline__ Pair running_sums(const float (&g)[4], int lane, Pair& last) {
  Pair incl{0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) incl = add(incl, Pair{clamp_g(g[i]), 0.0f});
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const Pair v{__shfl_up_sync(0xffffffffu, incl.hi, o), __shfl_up_sync(0xffffffffu, incl.lo, o)};
    if (lane >= o) incl = add(v, incl);
  }
  last = over_ln2(Pair{__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)});
  Pair before{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
  if (lane == 0) before = Pair{0.0f, 0.0f};
  return before;
}
__device__ __forceinline__ Pair minus(Pair a) { return Pair{-a.hi, -a.lo}; }

}  // namespace vssm
