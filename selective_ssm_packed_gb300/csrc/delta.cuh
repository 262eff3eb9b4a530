// delta.cuh -- device helpers of the chunked gated delta rule's kernels.
#pragma once

#include <atomic>

#include "delta.h"
#include "umma.cuh"

namespace vssm {

template <IO kIO> struct IoType { using type = float; };
template <> struct IoType<IO::BF16> { using type = __nv_bfloat16; };

// exp(x) with the error of x * log2(e) carried along, that of the product's
// rounding and that of kLog2e's own: the MUFU's 2^-22 remains, at every x whose
// exponential is a normal number.
__device__ __forceinline__ float exp_f(float x) {
  constexpr float kLog2eRest = (float)(1.44269504088896340736 - (double)kLog2e);
  const float t = x * kLog2e;
  const float r = fmaf(x, kLog2e, -t) + x * kLog2eRest;
  const float p = ex2(t);
  // outside, the power is 0 or infinite by itself, and r, where t is, means nothing
  return t > -126.0f && t < 128.0f ? fmaf(p, r * 0.6931471805599453f, p) : p;
}

// 8 consecutive io values from floats (16-byte aligned).
__device__ __forceinline__ void st_io8(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void st_io8(__nv_bfloat16* p, const float* v) {
  uint32_t t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    t[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(t[0], t[1], t[2], t[3]);
}

// Writes 8 values as chunk `chunk` of row `row` of NT images term_bytes apart
// (shared or global memory).
template <int NT, int kRowBytes>
__device__ __forceinline__ void put_chunk(uint8_t* image, int term_bytes, int row, int chunk, const float2* v) {
  uint32_t t[4][NT];
#pragma unroll
  for (int i = 0; i < 4; ++i) split_pair<NT>(v[i], t[i]);
  const uint32_t o = image_chunk<kRowBytes>(row, chunk);
#pragma unroll
  for (int i = 0; i < NT; ++i)
    *reinterpret_cast<uint4*>(image + i * term_bytes + o) = make_uint4(t[0][i], t[1][i], t[2][i], t[3][i]);
}

// kPairs pairs of this thread's row, columns from chunk0 * 8.
template <int NT, int kRowBytes, int kPairs>
__device__ __forceinline__ void put_row(uint8_t* image, int term_bytes, int row, int chunk0, const float2 (&v)[kPairs]) {
#pragma unroll
  for (int c = 0; c < kPairs / 4; ++c) put_chunk<NT, kRowBytes>(image, term_bytes, row, chunk0 + c, v + 4 * c);
}

// x * 0 added up: not 0 once any x is NaN or infinite.
template <int kPairs>
__device__ __forceinline__ float2 trace_row(const float2 (&v)[kPairs], float2 z) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) z = fma2(v[i], splat2(0.0f), z);
  return z;
}

template <int kPairs>
__device__ __forceinline__ void scale_row(float2 (&v)[kPairs], float f) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) v[i] = mul2(v[i], splat2(f));
}

// 16 bytes of io values as pairs (4 of bf16, 2 of float).
__device__ __forceinline__ void unpack(uint4 q, float2 (&v)[4]) {
  v[0] = make_float2(bf16_lo(q.x), bf16_hi(q.x));
  v[1] = make_float2(bf16_lo(q.y), bf16_hi(q.y));
  v[2] = make_float2(bf16_lo(q.z), bf16_hi(q.z));
  v[3] = make_float2(bf16_lo(q.w), bf16_hi(q.w));
}
__device__ __forceinline__ void unpack(uint4 q, float2 (&v)[2]) {
  v[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
  v[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
}

// N lanes (four or two), N chunks each: lane j's chunk i becomes lane i's chunk
// j.  A warp reads or writes 32 rows of 16 N bytes with it N lanes to a row,
// 32 / N rows an instruction; a lane to a row would touch 32 lines with every
// instruction (the forward walk spent more time on that than on its products).
template <int N>
__device__ __forceinline__ void transpose(uint4 (&q)[N], int lane) {
#pragma unroll
  for (int o = N / 2; o >= 1; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int a = 0; a < N; ++a) {
      if (a & o) continue;
      const uint4 give = up ? q[a] : q[a + o];
      uint4 got;
      got.x = __shfl_xor_sync(0xffffffffu, give.x, o);
      got.y = __shfl_xor_sync(0xffffffffu, give.y, o);
      got.z = __shfl_xor_sync(0xffffffffu, give.z, o);
      got.w = __shfl_xor_sync(0xffffffffu, give.w, o);
      if (up) q[a] = got; else q[a + o] = got;
    }
  }
}

// 32 rows of 16 N bytes, row i of a warp at base + i * stride (in T); `rows` of
// them exist and `cols` values of each.  Lane l gets (or gives) row l, once
// transposed.
template <typename T, int N>
__device__ __forceinline__ void load_rows(const T* base, int64_t stride, int rows, int cols, int lane, uint4 (&q)[N]) {
  constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = (lane & ~(N - 1)) + i, c = (lane & (N - 1)) * kPer;
    q[i] = make_uint4(0, 0, 0, 0);
    if (r < rows && c < cols) q[i] = *reinterpret_cast<const uint4*>(base + r * stride + c);
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_rows(T* base, int64_t stride, int rows, int cols, int lane, uint4 (&q)[N]) {
  constexpr int kPer = 16 / (int)sizeof(T);
  transpose(q, lane);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = (lane & ~(N - 1)) + i, c = (lane & (N - 1)) * kPer;
    if (r < rows && c < cols) *reinterpret_cast<uint4*>(base + r * stride + c) = q[i];
  }
}

// Eight pairs as 16-byte chunks of io values (two of bf16, four of float).
__device__ __forceinline__ void pack(const float2 (&v)[8], uint4* q, __nv_bfloat16) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[4 * i + j].x, v[4 * i + j].y);
      t[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    q[i] = make_uint4(t[0], t[1], t[2], t[3]);
  }
}
__device__ __forceinline__ void pack(const float2 (&v)[8], uint4* q, float) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = make_uint4(__float_as_uint(v[2 * i].x), __float_as_uint(v[2 * i].y), __float_as_uint(v[2 * i + 1].x),
                      __float_as_uint(v[2 * i + 1].y));
}

// A thread's part of a tile's row in the walks: where at most two walks share a
// CTA they have two threads to a row, 16 columns each, otherwise one.
template <int kWalks>
constexpr int walk_threads() { return kWalks <= 2 ? 256 * kWalks : 128 * kWalks; }  // of a CTA

template <typename T, int kWalks>
struct WalkRow {
  static constexpr int kThreads = walk_threads<kWalks>() / kWalks, kHalves = kThreads / 128;
  static constexpr int kCols = kDeltaTile / kHalves, kSteps = kCols / 16;  // steps of 16 columns: two chunks of an image's row
  static constexpr int kBytes = kCols * (int)sizeof(T), kPiece = kBytes < 64 ? kBytes : 64;  // as io values, in pieces
  static constexpr int kParts = kBytes / kPiece, kChunks = kPiece / 16, kWide = kPiece / (int)sizeof(T);
  static constexpr int kPer = 16 / (int)sizeof(T);
  typedef uint4 Raw[kParts][kChunks];
  // f(k, pair 8 u + k of the row) for k < 8
  template <typename F>
  static __device__ __forceinline__ void each(const Raw& raw, int u, F f) {
#pragma unroll
    for (int i = 0; i < 16 / kPer; ++i) {
      const int at = u * (16 / kPer) + i;
      float2 w[kPer / 2];
      unpack(raw[at / kChunks][at % kChunks], w);
#pragma unroll
      for (int j = 0; j < kPer / 2; ++j) f(i * (kPer / 2) + j, w[j]);
    }
  }
  static __device__ __forceinline__ void put(Raw& raw, int u, const float2 (&v)[8]) {
    const int at = u * (16 / kPer);
    pack(v, raw[at / kChunks] + at % kChunks, T());
  }
  // the warp's 32 rows from base on, of which `rows` exist and `cols` columns
  static __device__ __forceinline__ void load(const T* base, int64_t stride, int64_t rows, int cols, int lane, Raw& raw) {
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      load_rows(base + kWide * i, stride, (int)min((int64_t)32, rows), cols - kWide * i, lane, raw[i]);
  }
  static __device__ __forceinline__ void store(T* base, int64_t stride, int64_t rows, int cols, int lane, Raw& raw) {
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      store_rows(base + kWide * i, stride, (int)min((int64_t)32, rows), cols - kWide * i, lane, raw[i]);
  }
};

// A thread's wait for a phase of `bar`; false once it has run out of time, which
// it then says in the status word and to the CTA's other threads, who give up
// theirs (*stop, a word in shared memory, 0 at first).  The timer is read once
// in 64 tries.  forced: a test's wait, which counts as run out once it is over.
__device__ __forceinline__ bool wait_or_stop(const DeltaArgs& a, volatile int* stop, uint64_t* bar, uint32_t parity,
                                             bool forced = false) {
  if (!forced && mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
      if (!mbar_try_wait(bar, parity)) continue;
      if (!forced) return true;
      t0 = 1;  // long ago
      break;
    }
    if (*stop) return false;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > a.wait_ns) break;
  }
  *stop = 1;
  atomicOr(a.status, kStatusTmaTimeout);
  return false;
}
__device__ __forceinline__ bool forced_here(const DeltaArgs& a) { return (long long)blockIdx.x == a.force_timeout_cta; }

// The waits of one thread of a CTA.  After one that has run out the thread
// waits for nothing and, by `ok`, asks for no copy, issues no product and
// arrives nowhere, so that what others wait for stays out and every wait of the
// CTA ends; it still takes part in the barriers, up to one at which all threads
// leave together, by a vote or by one thread's word from before an earlier
// barrier (the forward walk's way: a vote in every chunk cost a walk alone on
// its SM 3%, where this costs 1.5%).  What the CTA has asked for is then waited
// for (drain_copies, and a commit behind the products) before its memory is
// given back.
struct Waiter {
  const DeltaArgs& a;
  volatile int* stop;
  bool ok = true;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity, bool forced = false) {
    return ok = ok && wait_or_stop(a, stop, bar, parity, forced);
  }
};

// Barrier `id` over `count` threads; whether all of them are ok.
__device__ __forceinline__ bool vote(int id, int count, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(count), "r"(ok ? 1u : 0u)
      : "memory");
  return all != 0;
}

// Waits, with a limit, for all `count` copies that were asked for on `bar`.
__device__ __forceinline__ void drain_copies(uint64_t* bar, int64_t count) {
  if (count > 0) mbar_wait(bar, (uint32_t)(count - 1) & 1, kCopyDrainNs);
}

template <typename P>
__device__ __forceinline__ P* align1024(P* p) {
  return reinterpret_cast<P*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~(uintptr_t)1023);
}

// Lets kernel f (one per call site: `done` is that site's own) use `bytes` of
// shared memory, once per device.
inline cudaError_t set_smem(const void* f, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

}  // namespace vssm
