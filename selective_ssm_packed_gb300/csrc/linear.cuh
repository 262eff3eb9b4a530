// linear.cuh -- device helpers of linear attention's kernels.
#pragma once

#include "delta.cuh"
#include "linear.h"

namespace vssm {

struct LinWaiter {
  const LinArgs& a;
  volatile int* stop;
  bool ok = true;
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity, bool forced = false) {
    ok = ok && wait_or_stop(a, stop, bar, parity, forced);
  }
};

// Like umma, A in tensor memory: its rows in the lanes, two bf16 to a column.
__device__ __forceinline__ void umma_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t desc_b, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
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

// A chunk's running sums of g over ln 2, a lane's tokens, and the sum over all.
template <int kPer>
struct GateSums {
  Pair G[kPer], last;
  __device__ __forceinline__ GateSums(const float (&g)[kPer], int lane) {
    Pair incl{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float v = g[i] < -256.0f ? -256.0f : g[i];  // exp of either is 0; -inf would leave inf - inf
      G[i] = incl = add(incl, Pair{v, 0.0f});
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Pair v{__shfl_up_sync(0xffffffffu, incl.hi, o), __shfl_up_sync(0xffffffffu, incl.lo, o)};
      if (lane >= o) incl = add(v, incl);
    }
    last = over_ln2(Pair{__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)});
    Pair before{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
    if (lane == 0) before = Pair{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kPer; ++i) G[i] = over_ln2(add(before, G[i]));
  }
};
__device__ __forceinline__ Pair minus(Pair a) { return Pair{-a.hi, -a.lo}; }

}  // namespace vssm
